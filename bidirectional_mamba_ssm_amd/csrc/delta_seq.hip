// The gated delta rule token by token, in fp32, for every type, head size and
// length (delta.hpp): what decoding and short blocks run.
// Columns of S never meet: a wave holds 16 of them, eight lanes to a pair of
// columns, N / 8 rows in registers a lane. Both products with the incoming state
// are reduced over the eight lanes by DPP, then the update follows;
// y_t = scale (a_t S_{t-1}^T q_t + (q_t . k_t) beta_t e_t) so that no product
// waits for the update. Queries, keys and values are staged in LDS as fp32, kTile
// tokens at a time, the next tile's loads under way meanwhile. One token is bound
// by its states' way through HBM: 64 x 32 heads of 128 x 128 61 us, 270 MB at
// 4.4 TB/s (a copy moves 5.1); a block by its chain of tokens, 0.4 us each.
#include "delta.hpp"
#include "internal.hpp"
#include "rows.hpp"

namespace bm {
namespace {

constexpr int kTile = 16;

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

// R consecutive entries of a column, 16 bytes at a time
template <int R>
__device__ __forceinline__ void load_state(bool given, const float *p, float *s) {
    constexpr int V = R < 4 ? R : 4;
    typedef float vec __attribute__((ext_vector_type(V)));
#pragma unroll
    for (int j = 0; j < R; j += V) {
        vec v = 0.f;
        if (given) v = *(const vec *)(p + j);
#pragma unroll
        for (int e = 0; e < V; ++e) s[j + e] = v[e];
    }
}
template <int R>
__device__ __forceinline__ void store_state(bool wanted, float *p, const float *s) {
    constexpr int V = R < 4 ? R : 4;
    typedef float vec __attribute__((ext_vector_type(V)));
#pragma unroll
    for (int j = 0; j < R; j += V) {
        vec v;
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = s[j + e];
        if (wanted) *(vec *)(p + j) = v;
    }
}

template <typename T, int N, int W>
__global__ __launch_bounds__(64 * W) void k_delta_seq(DeltaArgs a, int blocks) {
    constexpr int kThreads = 64 * W, V = 16 / sizeof(T), R = N / 8, kCols = 16 * W;
    constexpr int kVecs = 2 * kTile * N / V, kPer = (kVecs + kThreads - 1) / kThreads;
    __shared__ __attribute__((aligned(16))) float qk[2][2][kTile][N];
    __shared__ float vs[2][kTile][kCols];
    __shared__ float gate[2][2][kTile];   // e^g, beta
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int part = lane & 7, pair = lane >> 3;
    const int block = blockIdx.x % blocks, h = blockIdx.x / blocks % a.H, u = blockIdx.x / blocks / a.H;
    const int p0 = block * kCols, p = p0 + 16 * wave + 2 * pair, grp = h / (a.H / a.G);
    const DeltaUnit at = delta_unit(a, u);
    const bool own0 = p < a.P, own1 = p + 1 < a.P;
    float s0[R], s1[R];
    const size_t state = (((size_t)u * a.H + h) * a.P + p) * N + part * R;
    load_state<R>(a.init && own0, a.init + state, s0);
    load_state<R>(a.init && own1, a.init + state + N, s1);
    rvec nqk[kPer];
    T nv[4];
    float ngate = 0.f;
    // the tokens of tile t in the order they are walked
    auto token = [&](int i) { return delta_token(at, a.reverse, min(i, at.len - 1)); };
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
            nv[i] = ((const T *)a.v)[((size_t)token(t + tok) * a.H + h) * a.P + c];
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
            (&vs[buf][0][0])[e] = as_float(nv[i]);
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
            float kf[R], qf[R];
#pragma unroll
            for (int j = 0; j < R; ++j) {
                qf[j] = qk[buf][0][i][part * R + j];
                kf[j] = qk[buf][1][i][part * R + j];
            }
            const float decay = gate[buf][0][i], beta = gate[buf][1][i];
            const float x0 = vs[buf][i][16 * wave + 2 * pair], x1 = vs[buf][i][16 * wave + 2 * pair + 1];
            float k0 = 0.f, k1 = 0.f, q0 = 0.f, q1 = 0.f, dot = 0.f;
#pragma unroll
            for (int j = 0; j < R; ++j) {
                k0 = fmaf(kf[j], s0[j], k0);
                k1 = fmaf(kf[j], s1[j], k1);
                q0 = fmaf(qf[j], s0[j], q0);
                q1 = fmaf(qf[j], s1[j], q1);
                dot = fmaf(qf[j], kf[j], dot);
            }
            k0 = group_total<8>(k0);
            k1 = group_total<8>(k1);
            q0 = group_total<8>(q0);
            q1 = group_total<8>(q1);
            dot = group_total<8>(dot);
            const float w0 = beta * fmaf(-decay, k0, x0), w1 = beta * fmaf(-decay, k1, x1);
            const float o0 = a.scale * fmaf(dot, w0, decay * q0), o1 = a.scale * fmaf(dot, w1, decay * q1);
#pragma unroll
            for (int j = 0; j < R; ++j) {
                s0[j] = fmaf(kf[j], w0, decay * s0[j]);
                s1[j] = fmaf(kf[j], w1, decay * s1[j]);
            }
            if (part < 2) {
                const bool own = part ? own1 : own0;
                if (own) {
                    float *y = a.y + ((size_t)delta_token(at, a.reverse, t + i) * a.H + h) * a.P + p + part;
                    const float o = part ? o1 : o0;
                    *y = a.add ? *y + o : o;
                }
            }
        }
        if (t + kTile < at.len) stash(buf ^ 1);
    }
    store_state<R>(a.last && own0, a.last + state, s0);
    store_state<R>(a.last && own1, a.last + state + N, s1);
}

template <typename T, int N>
hipError_t launch_n(const DeltaArgs &a, hipStream_t s) {
    // four waves share their queries and keys where that leaves two workgroups for
    // every CU (256 heads of 128 x 128: one token 13.3 us, 14.2 with a wave each, 16
    // tokens 21.0 and 27.1; 128 heads 9.6 and 9.4, 16.1 and 15.9)
    const long long heads = (long long)a.units * a.H;
    const int wide = (a.P + 63) / 64, narrow = (a.P + 15) / 16;
    if (a.P > 16 && heads * wide >= 512)
        BM_LAUNCH("delta_seq", (k_delta_seq<T, N, 4>), dim3((unsigned)(heads * wide)), dim3(256), 0, s, a, wide);
    else
        BM_LAUNCH("delta_seq", (k_delta_seq<T, N, 1>), dim3((unsigned)(heads * narrow)), dim3(64), 0, s, a, narrow);
    return hipGetLastError();
}
template <typename T>
hipError_t launch_t(const DeltaArgs &a, hipStream_t s) {
    switch (a.N) {
        case 16: return launch_n<T, 16>(a, s);
        case 32: return launch_n<T, 32>(a, s);
        case 64: return launch_n<T, 64>(a, s);
        case 128: return launch_n<T, 128>(a, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_delta_seq(const DeltaArgs &a, bool bf16, hipStream_t s) {
    return bf16 ? launch_t<uint16_t>(a, s) : launch_t<float>(a, s);
}

}  // namespace bm
