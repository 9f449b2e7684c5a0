// The gated delta rule, as its kernels see it. Per head (query and key group
// g = h / (H / G)), with the state S [N][P]:
//   a_t = e^{g_t},  e_t = v_t - a_t S_{t-1}^T k_t,
//   S_t = a_t S_{t-1} + beta_t k_t e_t^T,  y_t = scale S_t^T q_t
// States are kept [P][N] in memory, as the scan's are.
#pragma once
#include <hip/hip_runtime.h>

#include "common.hpp"

namespace bm {

constexpr int kDeltaChunk = 64;   // tokens between kept states

// One direction of a problem (validated). Units are rows of the batch or
// packed sequences; a reversed direction takes a unit's tokens from its end.
struct DeltaArgs {
    const void *q, *k;         // [tok][G][N]
    const void *v;             // [tok][H][P]; walking back: float, the gradient of y
    const float *g, *beta;     // [tok][H]
    float scale;
    int units, L, H, P, N, G;  // L: tokens of a row (packed: of all)
    bool reverse, add;         // add: y += instead of y =
    const int32_t *cu;         // device offsets [units + 1] of packed sequences, or nullptr
    const float *init;         // [units][H][P][N] or nullptr (zeros); walking back: its gradient
    float *last;               // the same, written at the end, or nullptr
    float *y;                  // [tok][H][P]: y; for the gradient [tok][H][P rounded up]: e, walking back
                               // z = d loss / d (beta e)
    float *states;             // [slot][H][N][P rounded up]: chunks' incoming states; walking back: gradients
                               // of what they leave
};

// What the gradient reads beside a direction's inputs, and writes.
struct DeltaGradArgs {
    const float *dy;                 // [tok][H][P]
    const float *e, *z;              // [tok][H][P rounded up]
    const float *enter, *leave;      // [slot][H][N][P rounded up]: incoming states, gradients of the outgoing
    const float *gates;              // the preparing kernel's (delta_gates)
    float *dq, *dk, *dv, *dg, *dbeta;
    float *parts;                    // [delta_grad_parts - 1][dq, dk][tok][G][N]
};

// A unit's chunk c is kept in slot first_slot + c. Packed units' slots are
// given out without a table: floor(x) + ceil(y) <= floor(x + y) + 1.
__host__ __device__ inline long long delta_slots(int units, int L, bool packed) {
    return packed ? (long long)L / kDeltaChunk + units
                  : (long long)units * ((L + kDeltaChunk - 1) / kDeltaChunk);
}
struct DeltaUnit {
    long long start, slot;
    int len;
};
__device__ __forceinline__ DeltaUnit delta_unit(const DeltaArgs &a, int u) {
    DeltaUnit d;
    if (a.cu) {
        d.start = a.cu[u];
        d.len = a.cu[u + 1] - a.cu[u];
        d.slot = d.start / kDeltaChunk + u;
    } else {
        d.start = (long long)u * a.L;
        d.len = a.L;
        d.slot = (long long)u * ((a.L + kDeltaChunk - 1) / kDeltaChunk);
    }
    return d;
}
// the unit whose chunk a slot keeps, and the chunk (past its end if the slot is
// not used)
__device__ __forceinline__ DeltaUnit delta_slot(const DeltaArgs &a, long long slot, int &chunk) {
    int u;
    if (a.cu) {
        int lo = 0, hi = a.units;   // slot of unit lo <= slot < slot of unit hi
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if ((long long)a.cu[mid] / kDeltaChunk + mid <= slot) lo = mid;
            else hi = mid;
        }
        u = lo;
    } else {
        u = (int)(slot / ((a.L + kDeltaChunk - 1) / kDeltaChunk));
    }
    const DeltaUnit d = delta_unit(a, u);
    chunk = (int)(slot - d.slot);
    return d;
}
__device__ __forceinline__ long long delta_token(const DeltaUnit &d, bool reverse, int i) {
    return d.start + (reverse ? d.len - 1 - i : i);
}

// delta_seq.hip: y and the last state, token by token
hipError_t launch_delta_seq(const DeltaArgs &a, bool bf16, hipStream_t s);
// delta_chunk.hip: the same by chunks, of one or both directions (a[0] forward,
// a[1] reverse, each with its workspace); e and the chunks' incoming states; z and
// the gradients of the outgoing (with the workspace that the call before filled)
size_t delta_chunk_workspace(const DeltaArgs &a, bool grad);
hipError_t launch_delta_chunked(const DeltaArgs *a, int ndir, bool bf16, void *const *ws, hipStream_t s);
hipError_t launch_delta_keep(const DeltaArgs *a, int ndir, bool bf16, void *const *ws, hipStream_t s);
hipError_t launch_delta_back(const DeltaArgs *a, int ndir, bool bf16, void *const *ws, hipStream_t s);
const float *delta_gates(const DeltaArgs &a, void *ws);
// delta_grad.hip, and the bytes of e or z, and of the kept states or their gradients
size_t delta_rows_bytes(const DeltaArgs &a);
size_t delta_parts_bytes(const DeltaArgs &a);
size_t delta_states_bytes(const DeltaArgs &a);
hipError_t launch_delta_grad(const DeltaArgs *a, const DeltaGradArgs *o, int ndir, bool bf16, hipStream_t s);

// A walk keeps one CU a head and unit busy: where both directions' fit on the 256
// CUs they go side by side, each with arrays of its own (a[1].y is not a[0].y then,
// and is added to it). One after the other the 66 heads of eleven packed
// sequences took 73 us, side by side 38.
inline bool delta_apart(int units, int H) { return 2LL * units * H <= 256; }

}  // namespace bm
