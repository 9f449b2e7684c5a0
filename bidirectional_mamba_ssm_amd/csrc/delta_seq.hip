// The gated delta rule token by token, in fp32, for every type, head size and
// length: the forward recurrence (delta.hpp), the same keeping what its
// gradient needs, and the gradient's walk back. With dS the gradient of S_t
// and do_t = scale dy_t, from the last token to the first:
//   z_t = (dS + q_t do_t^T)^T k_t            (the gradient of beta_t e_t)
//   dS <- a_t (dS + q_t do_t^T - beta_t k_t z_t^T)
// Columns of S never meet: a wave holds 16 of them, eight lanes to a pair of
// columns, N / 8 rows in registers a lane. Both products with the incoming state
// (k and q forward, k backward) are reduced over the eight lanes by DPP, then the
// update follows; y_t = scale (a_t S_{t-1}^T q_t + (q_t . k_t) beta_t e_t) so that
// no product waits for the update. Queries, keys and the third input are
// staged in LDS as fp32, kTile tokens at a time, the next tile's loads under way
// meanwhile.
#include "delta.hpp"
#include "internal.hpp"
#include "rows.hpp"

namespace bm {
namespace {

constexpr int kTile = 16;
enum { FWD, KEEP, BACK };

// 16 bytes of queries or keys as floats
__device__ __forceinline__ void widen(float *to, rvec r, uint16_t) {
#pragma unroll
    for (int j = 0; j < 8; ++j) to[j] = Lane<uint16_t>::get(r, j);
}
__device__ __forceinline__ void widen(float *to, rvec r, float) {
#pragma unroll
    for (int j = 0; j < 4; ++j) to[j] = __uint_as_float(r[j]);
}
__device__ __forceinline__ float as_float(uint16_t v) { return bf2f(v); }
__device__ __forceinline__ float as_float(float v) { return v; }

template <typename T, int N, int W, int MODE>
__global__ __launch_bounds__(64 * W) void k_delta_seq(DeltaArgs a, int blocks) {
    using X = typename std::conditional<MODE == BACK, float, T>::type;   // the third input's type
    constexpr int kThreads = 64 * W, V = 16 / sizeof(T), R = N / 8, kCols = 16 * W;
    constexpr int kVecs = 2 * kTile * N / V, kPer = (kVecs + kThreads - 1) / kThreads;
    __shared__ __attribute__((aligned(16))) float qk[2][2][kTile][N];
    __shared__ float third[2][kTile][kCols];
    __shared__ float gate[2][2][kTile];   // e^g, beta
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int part = lane & 7, pair = lane >> 3;
    const int block = blockIdx.x % blocks, h = blockIdx.x / blocks % a.H, u = blockIdx.x / blocks / a.H;
    const int p0 = block * kCols, p = p0 + 16 * wave + 2 * pair, grp = h / (a.H / a.G);
    const DeltaUnit at = delta_unit(a, u);
    const bool own0 = p < a.P, own1 = p + 1 < a.P;
    float s0[R], s1[R];
    const size_t state = (((size_t)u * a.H + h) * a.P + p) * N + part * R;
#pragma unroll
    for (int j = 0; j < R; ++j) {
        s0[j] = a.init && own0 ? a.init[state + j] : 0.f;
        s1[j] = a.init && own1 ? a.init[state + N + j] : 0.f;
    }
    rvec nqk[kPer];
    X nthird[4];
    float ngate = 0.f;
    // the tokens of tile t in the order they are walked
    auto token = [&](int i) {
        const int k = min(i, at.len - 1);
        return delta_token(at, a.reverse, MODE == BACK ? at.len - 1 - k : k);
    };
    auto fetch = [&](int t) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = tid + kThreads * i;
            if (kVecs % kThreads == 0 || e < kVecs) {
                const int which = e / (kTile * N / V), r = e % (kTile * N / V), tok = r / (N / V), c = r % (N / V) * V;
                const T *src = (const T *)(which ? a.k : a.q);
                nqk[i] = Lane<T>::load(src + ((size_t)token(t + tok) * a.G + grp) * N + c);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = tid + kThreads * i, tok = e / kCols, c = min(p0 + e % kCols, a.P - 1);
            nthird[i] = ((const X *)a.v)[((size_t)token(t + tok) * a.H + h) * a.P + c];
        }
        if (tid < 2 * kTile) {
            const float *src = tid < kTile ? a.g : a.beta;
            ngate = src[(size_t)token(t + tid % kTile) * a.H + h];
        }
    };
    auto stash = [&](int buf) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = tid + kThreads * i;
            if (kVecs % kThreads == 0 || e < kVecs) widen(&qk[buf][0][0][0] + e * V, nqk[i], T());
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = tid + kThreads * i;
            (&third[buf][0][0])[e] = as_float(nthird[i]);
        }
        if (tid < 2 * kTile) (&gate[buf][0][0])[tid] = tid < kTile ? expf(ngate) : ngate;
    };
    if (at.len > 0) {
        fetch(0);
        stash(0);
    }
    for (int t = 0, buf = 0; t < at.len; t += kTile, buf ^= 1) {
        __syncthreads();
        if (t + kTile < at.len) fetch(t + kTile);
        const int n = min(kTile, at.len - t);
        for (int i = 0; i < n; ++i) {
            const int step = t + i, pos = MODE == BACK ? at.len - 1 - step : step;
            if (MODE != FWD) {
                // the state before a chunk's first token, the gradient after its last
                const bool edge = MODE == KEEP ? pos % kDeltaChunk == 0
                                               : pos % kDeltaChunk == kDeltaChunk - 1 || step == 0;
                if (edge) {
                    float *to = a.states + (((size_t)(at.slot + pos / kDeltaChunk) * a.H + h) * a.P + p) * N + part * R;
#pragma unroll
                    for (int j = 0; j < R; ++j) {
                        if (own0) to[j] = s0[j];
                        if (own1) to[N + j] = s1[j];
                    }
                }
            }
            float kf[R], qf[R];
#pragma unroll
            for (int j = 0; j < R; ++j) {
                qf[j] = qk[buf][0][i][part * R + j];
                kf[j] = qk[buf][1][i][part * R + j];
            }
            const float decay = gate[buf][0][i], beta = gate[buf][1][i];
            const float x0 = third[buf][i][16 * wave + 2 * pair], x1 = third[buf][i][16 * wave + 2 * pair + 1];
            float k0 = 0.f, k1 = 0.f, q0 = 0.f, q1 = 0.f, dot = 0.f;
#pragma unroll
            for (int j = 0; j < R; ++j) {
                k0 = fmaf(kf[j], s0[j], k0);
                k1 = fmaf(kf[j], s1[j], k1);
                if (MODE == FWD) {
                    q0 = fmaf(qf[j], s0[j], q0);
                    q1 = fmaf(qf[j], s1[j], q1);
                }
                if (MODE != KEEP) dot = fmaf(qf[j], kf[j], dot);
            }
            k0 = group_total<8>(k0);
            k1 = group_total<8>(k1);
            if (MODE != KEEP) dot = group_total<8>(dot);
            float o0, o1;
            if constexpr (MODE == BACK) {
                const float d0 = a.scale * x0, d1 = a.scale * x1;
                o0 = fmaf(dot, d0, k0);
                o1 = fmaf(dot, d1, k1);
                const float w0 = -beta * o0, w1 = -beta * o1;
#pragma unroll
                for (int j = 0; j < R; ++j) {
                    s0[j] = decay * fmaf(kf[j], w0, fmaf(qf[j], d0, s0[j]));
                    s1[j] = decay * fmaf(kf[j], w1, fmaf(qf[j], d1, s1[j]));
                }
            } else {
                const float e0 = fmaf(-decay, k0, x0), e1 = fmaf(-decay, k1, x1);
                const float w0 = beta * e0, w1 = beta * e1;
                o0 = e0;
                o1 = e1;
                if (MODE == FWD) {
                    q0 = group_total<8>(q0);
                    q1 = group_total<8>(q1);
                    o0 = a.scale * fmaf(dot, w0, decay * q0);
                    o1 = a.scale * fmaf(dot, w1, decay * q1);
                }
#pragma unroll
                for (int j = 0; j < R; ++j) {
                    s0[j] = fmaf(kf[j], w0, decay * s0[j]);
                    s1[j] = fmaf(kf[j], w1, decay * s1[j]);
                }
            }
            if (part < 2) {
                const bool own = part ? own1 : own0;
                if (own) {
                    float *y = a.y + ((size_t)delta_token(at, a.reverse, pos) * a.H + h) * a.P + p + part;
                    const float o = part ? o1 : o0;
                    *y = MODE == FWD && a.add ? *y + o : o;
                }
            }
        }
        if (t + kTile < at.len) stash(buf ^ 1);
    }
    if (!a.last) return;
#pragma unroll
    for (int j = 0; j < R; ++j) {
        if (own0) a.last[state + j] = s0[j];
        if (own1) a.last[state + N + j] = s1[j];
    }
}

template <typename T, int N, int MODE>
hipError_t launch_n(const DeltaArgs &a, hipStream_t s) {
    static const char *const names[] = {"delta_seq", "delta_seq_keep", "delta_seq_back"};
    // four waves share their queries and keys where that leaves workgroups for
    // every CU
    const long long heads = (long long)a.units * a.H;
    const int wide = (a.P + 63) / 64, narrow = (a.P + 15) / 16;
    if (a.P > 16 && heads * wide >= 512)
        BM_LAUNCH(names[MODE], (k_delta_seq<T, N, 4, MODE>), dim3((unsigned)(heads * wide)), dim3(256), 0, s, a, wide);
    else
        BM_LAUNCH(names[MODE], (k_delta_seq<T, N, 1, MODE>), dim3((unsigned)(heads * narrow)), dim3(64), 0, s, a,
                  narrow);
    return hipGetLastError();
}
template <typename T, int MODE>
hipError_t launch_t(const DeltaArgs &a, hipStream_t s) {
    switch (a.N) {
        case 16: return launch_n<T, 16, MODE>(a, s);
        case 32: return launch_n<T, 32, MODE>(a, s);
        case 64: return launch_n<T, 64, MODE>(a, s);
        case 128: return launch_n<T, 128, MODE>(a, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_delta_seq(const DeltaArgs &a, bool bf16, hipStream_t s) {
    return bf16 ? launch_t<uint16_t, FWD>(a, s) : launch_t<float, FWD>(a, s);
}
hipError_t launch_delta_keep(const DeltaArgs &a, bool bf16, hipStream_t s) {
    return bf16 ? launch_t<uint16_t, KEEP>(a, s) : launch_t<float, KEEP>(a, s);
}
hipError_t launch_delta_back(const DeltaArgs &a, bool bf16, hipStream_t s) {
    return bf16 ? launch_t<uint16_t, BACK>(a, s) : launch_t<float, BACK>(a, s);
}

}  // namespace bm
