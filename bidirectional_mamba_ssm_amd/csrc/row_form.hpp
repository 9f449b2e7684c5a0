// How the row norms (layer_norm.hip, rms_norm.hip) hold a row in registers:
// NV 16-byte vectors a lane, over the lanes of a part of a wave, of a wave or
// of several waves of a workgroup.
//
// The last vector of a row whose length is no multiple of it starts at C - V
// instead: it overlaps its neighbour, its first `skip` elements count in no
// sum, and its stores repeat the neighbour's values. No load leaves the row.
#pragma once
#include "internal.hpp"
#include "rows.hpp"

namespace bm {
namespace {

constexpr int kMaxWaves = 8;   // of a row

// Where a lane's vectors lie in a row of C channels shared by `waves` waves:
// vector k starts at channel c[k]. has[k] is false for a lane past the end (it
// reads the row's last vector again). In vector kt (-1: none) some lane's
// first `skip` elements belong to the vector before.
template <int V, int NV>
struct Place {
    int c[NV];
    bool has[NV];
    int kt, skip;
    float count;   // elements of this wave
    __device__ __forceinline__ Place(int C, int t, int lanes) {
        kt = C % V ? C / (V * lanes) : -1;
        skip = 0;
        int n = 0;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int at = (k * lanes + t) * V;
            c[k] = min(at, C - V);
            has[k] = at < C;
            if (at < C && at != c[k]) skip = at - c[k];
            const int first = (k * lanes + (t & ~63)) * V;
            n += max(0, min(64 * V, C - first));
        }
        count = (float)n;
    }
    // v's element j of vector k counts: all do but the overlapped ones
    __device__ __forceinline__ float own(int k, int j, float v) const { return k == kt && j < skip ? 0.f : v; }
};

template <int V>
__device__ __forceinline__ void load_w(const float *p, int c, float none, float *v) {
    if (p) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            const rvec r = *(const u4_a4 *)(p + c + 4 * i);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[4 * i + j] = __uint_as_float(r[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = none;
    }
}

template <int G>
__device__ __forceinline__ float lanes_total(float v) {
    if constexpr (G == 0 || G == 64) return wave_total(v);
    else return group_total<G>(v);
}

// How a row is held: G lanes of one wave or (G = 0) `waves` waves, nv vectors
// a lane. Rows of up to 256 channels take the fewest lanes, 8 elements each
// (kernel times, bf16: 60 000 x 64 5.6 us, with residual and checkpoint 8.9,
// their gradient 12.4; a wave a row 16.8, 26.9 and 21.8; 60 000 x 128 13.3 and
// 16.0 for 27.2 and 23.4); wider ones `lane` elements a lane, or the fewest
// that kMaxWaves waves can do with.
struct Form {
    int nv, waves, G;
};
template <typename T>
Form row_form(int C, int lane) {
    const int V = 16 / (int)sizeof(T);
    Form f;
    f.nv = 1;
    f.waves = 1;
    f.G = 64;
    if (C <= 256) {
        f.nv = 8 / V;
        f.G = C <= 64 ? 8 : C <= 128 ? 16 : 32;
        return f;
    }
    const int units = (C + 64 * V - 1) / (64 * V);          // vectors of a row, in waves
    while (f.nv * V < lane && f.nv < units) f.nv *= 2;
    while (f.nv * kMaxWaves < units) f.nv *= 2;
    f.waves = (units + f.nv - 1) / f.nv;
    if (f.waves > 1) f.G = 0;
    return f;
}
}  // namespace
}  // namespace bm
