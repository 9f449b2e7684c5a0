// Layer norm of the residual stream in front of a mixer block, and its
// gradient. Per row (token) of C channels:
//   h = x + residual (rounded to the dtype), mu = mean h,
//   var = mean (h - mu)^2, rstd = (var + eps)^-1/2,
//   out = (h - mu) rstd w + b
// and, with xh = (h - mu) rstd, g = dout w, dsum the gradient that reaches h
// along the residual path:
//   dh = rstd (g - mean g - xh mean(g xh)) + dsum
//   dw = sum_rows dout xh,  db = sum_rows dout
// h may be read back from its 8-bit checkpoint (rows.hpp), which the forward
// pass can write as it goes.
//
// Both are streams bounded by HBM. A row lives in the registers of 64 to 512
// lanes (32 elements each at most, 16-byte vectors), so every array is
// read or written once; the sums over a row are DPP lane moves, and LDS only
// where a row has more than one wave. dw and db are summed in registers over
// the rows a workgroup walks, then over the workgroups in a fixed order by a
// second launch (col_sum.hip): no atomics, the same bits every time.
//
// The last vector of a row whose length is no multiple of it starts at C - V
// instead: it overlaps its neighbour, its first `skip` elements count in no
// sum, and its stores repeat the neighbour's values. No load leaves the row.
#include "internal.hpp"
#include "rows.hpp"

namespace bm {
namespace {

// sums of N values over the TPR lanes of a row; `part` has 2 * TPR/64 * N
// floats, its halves used in turn (`flip`), so one barrier a sum is enough
template <int TPR, int N>
__device__ __forceinline__ void row_totals(float (&v)[N], float *part, int &flip) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_total(v[i]);
    if constexpr (TPR > 64) {
        constexpr int NW = TPR / 64;
        const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
        float *p = part + flip * NW * N;
        flip ^= 1;
        if (lane == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) p[wave * N + i] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) s += p[w * N + i];
            v[i] = s;
        }
    }
}

// Where a lane's vectors lie in a row of C channels: vector k starts at
// channel c[k]; its elements below skip[k] belong to the vector before
// (V: the lane has none).
template <int V, int NV, int TPR>
struct Place {
    int c[NV], skip[NV];
    uint32_t full;   // bit k: every lane of the wave has all of vector k
    __device__ __forceinline__ Place(int C) {
        const int t = threadIdx.x & (TPR - 1);
        full = 0;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int at = (k * TPR + t) * V;
            c[k] = min(at, C - V);
            skip[k] = min(at - c[k], V);
            if (__all(skip[k] == 0)) full |= 1u << k;
        }
    }
};

template <typename T, int E, int TPR, bool RES, bool CK>
__global__ __launch_bounds__(TPR > 64 ? TPR : 256) void k_layer_norm(LnArgs a) {
    using L = Lane<T>;
    constexpr int V = L::V, NV = E / V;
    __shared__ float part[TPR > 64 ? 2 * TPR / 64 : 1];
    const int C = a.C;
    const Place<V, NV, TPR> at(C);
    const int slot = TPR > 64 ? 0 : threadIdx.x >> 6;
    constexpr int RPW = TPR > 64 ? 1 : 4;
    const float n = (float)C;
    int flip = 0;
    for (long long row = (long long)blockIdx.x * RPW + slot; row < a.rows; row += (long long)gridDim.x * RPW) {
        const T *x = (const T *)a.x + row * C;
        rvec r[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) r[k] = L::load(x + at.c[k]);
        if constexpr (RES) {
            const T *s = (const T *)a.res + row * C;
            rvec q[NV];
#pragma unroll
            for (int k = 0; k < NV; ++k) q[k] = L::load(s + at.c[k]);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                float h[V];
#pragma unroll
                for (int j = 0; j < V; ++j) h[j] = L::get(r[k], j) + L::get(q[k], j);
                r[k] = L::pack(h);   // the stream is kept in its dtype, and the norm sees what is kept
            }
        }
        float m[1] = {0.f};
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (at.full >> k & 1) {
#pragma unroll
                for (int j = 0; j < V; ++j) m[0] += L::get(r[k], j);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) m[0] += j >= at.skip[k] ? L::get(r[k], j) : 0.f;
            }
        }
        row_totals<TPR>(m, part, flip);
        const float mean = m[0] / n;   // exact for a constant row whose sum is
        float q[1] = {0.f};
#pragma unroll
        for (int k = 0; k < NV; ++k) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float d = L::get(r[k], j) - mean;
                const float dd = (at.full >> k & 1) || j >= at.skip[k] ? d : 0.f;
                q[0] = fmaf(dd, dd, q[0]);
            }
        }
        row_totals<TPR>(q, part, flip);
        const float rstd = 1.0f / sqrtf(q[0] / n + a.eps);
        T *out = (T *)a.out + row * C;
        T *sum = (T *)a.sum + row * C;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const bool ok = at.skip[k] < V;
            float o[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                o[j] = (L::get(r[k], j) - mean) * rstd;
                if (a.w) o[j] *= a.w[at.c[k] + j];
                if (a.b) o[j] += a.b[at.c[k] + j];
            }
            if (ok) {
                L::store(out + at.c[k], L::pack(o));
                if constexpr (RES) L::store(sum + at.c[k], r[k]);
            }
            if constexpr (CK) {
                uint32_t top = 0;
#pragma unroll
                for (int j = 0; j < V; ++j)
                    top = max(top, j >= at.skip[k] ? abs_bits(L::get(r[k], j)) : 0u);
                const int e = (int)(block_max<32 / V>(top) >> 23);
                int8_t *cq = a.q + row * C;
                int code[V];
#pragma unroll
                for (int j = 0; j < V; ++j) code[j] = act8_code(L::get(r[k], j), e);
                if (at.skip[k] == 0) {
                    Bytes<V>::store(cq + at.c[k], Bytes<V>::pack(code));
                } else {
                    // the overlapped elements may lie in another block
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        if (j >= at.skip[k]) cq[at.c[k] + j] = (int8_t)code[j];
                }
                const int c0 = at.c[k] + at.skip[k];
                if (ok && (c0 & 31) == 0) a.scale[row * ((C + 31) / 32) + c0 / 32] = (uint8_t)e;
            }
        }
        if ((threadIdx.x & (TPR - 1)) == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
    }
}

template <typename T, int E, int TPR, bool Q8, bool DSUM>
__global__ __launch_bounds__(TPR > 64 ? TPR : 256) void k_layer_norm_bwd(LnBwdArgs a) {
    using L = Lane<T>;
    constexpr int V = L::V, NV = E / V;
    __shared__ float part[TPR > 64 ? 4 * TPR / 64 : 1];
    const int C = a.C;
    const Place<V, NV, TPR> at(C);
    const int slot = TPR > 64 ? 0 : threadIdx.x >> 6;
    constexpr int RPW = TPR > 64 ? 1 : 4;
    const float inv = 1.0f / (float)C;
    const int nblk = (C + 31) / 32;
    int flip = 0;
    float w[NV][V], dw[NV][V], db[NV][V];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            w[k][j] = a.w ? a.w[at.c[k] + j] : 1.f;
            dw[k][j] = db[k][j] = 0.f;
        }
    for (long long row = (long long)blockIdx.x * RPW + slot; row < a.rows; row += (long long)gridDim.x * RPW) {
        const float mean = a.mean[row], rstd = a.rstd[row];
        const T *dout = (const T *)a.dout + row * C;
        const T *ds = (const T *)a.dsum + row * C;
        rvec g[NV], s[DSUM ? NV : 1], x[Q8 ? 1 : NV];
        typename Bytes<V>::type q[Q8 ? NV : 1];
        uint32_t e[Q8 ? NV : 1];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            g[k] = L::load(dout + at.c[k]);
            if constexpr (Q8) {
                q[k] = Bytes<V>::load((const int8_t *)a.x + row * C + at.c[k]);
                // the block of the lane's own elements; overlapped ones are not used
                e[k] = a.xscale[row * nblk + min(at.c[k] + at.skip[k], C - 1) / 32];
            } else {
                x[k] = L::load((const T *)a.x + row * C + at.c[k]);
            }
            if constexpr (DSUM) s[k] = L::load(ds + at.c[k]);
        }
        auto xhat = [&](int k, int j) {
            float v;
            if constexpr (Q8) v = (float)Bytes<V>::get(q[k], j) * act8_unit(e[k]);
            else v = L::get(x[k], j);
            return (v - mean) * rstd;
        };
        float t[2] = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < NV; ++k) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float d = L::get(g[k], j);
                const float xh = xhat(k, j);
                db[k][j] += d;
                dw[k][j] = fmaf(d, xh, dw[k][j]);
                const float gw = (at.full >> k & 1) || j >= at.skip[k] ? d * w[k][j] : 0.f;
                t[0] += gw;
                t[1] = fmaf(gw, xh, t[1]);
            }
        }
        row_totals<TPR>(t, part, flip);
        const float m1 = t[0] * inv, m2 = t[1] * inv;
        T *dx = (T *)a.dx + row * C;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float o[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                o[j] = rstd * (fmaf(L::get(g[k], j), w[k][j], -m1) - xhat(k, j) * m2);
                if constexpr (DSUM) o[j] += L::get(s[k], j);
            }
            if (Q8 ? at.skip[k] == 0 : at.skip[k] < V) {
                L::store(dx + at.c[k], L::pack(o));
            } else if (Q8 && at.skip[k] < V) {
                const rvec p = L::pack(o);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    if (j < at.skip[k]) continue;
                    if constexpr (sizeof(T) == 2)
                        dx[at.c[k] + j] = (T)(p[j >> 1] >> (16 * (j & 1)));
                    else
                        dx[at.c[k] + j] = __uint_as_float(p[j]);
                }
            }
        }
    }
    if (!a.part) return;
    // this workgroup's share of dw | db; several waves of one row each hold
    // other channels, four waves of four rows the same ones (added in order)
    float *out = a.part + (size_t)blockIdx.x * 2 * C;
    if constexpr (TPR == 64) {
        __shared__ float sum[2 * E * 64];
        const int lane = threadIdx.x & 63;
        for (int s = 0; s < 4; ++s) {
            if (slot == s) {
#pragma unroll
                for (int k = 0; k < NV; ++k)
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const int i = (k * V + j) * 64 + lane;
                        if (s > 0) {
                            dw[k][j] += sum[i];
                            db[k][j] += sum[E * 64 + i];
                        }
                        if (s < 3) {
                            sum[i] = dw[k][j];
                            sum[E * 64 + i] = db[k][j];
                        }
                    }
            }
            __syncthreads();
        }
        if (slot != 3) return;
    }
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (j >= at.skip[k]) {
                out[at.c[k] + j] = dw[k][j];
                out[C + at.c[k] + j] = db[k][j];
            }
}

// lanes and elements per lane of a row: the fewest that hold it
#define BM_ROW_FORMS(DO) DO(8, 64) DO(16, 64) DO(32, 64) DO(32, 128) DO(32, 256) DO(32, 512)

template <typename T, bool RES, bool CK>
hipError_t launch_fwd(const LnArgs &a, hipStream_t s) {
#define DO(E, TPR)                                                                              \
    if (a.C <= E * TPR) {                                                                       \
        const long long per = TPR > 64 ? 1 : 4, wgs = (a.rows + per - 1) / per;                  \
        const dim3 grid((unsigned)(wgs < 4096 ? wgs : 4096));                                    \
        BM_LAUNCH("layer_norm", (k_layer_norm<T, E, TPR, RES, CK>), grid,                        \
                  dim3(TPR > 64 ? TPR : 256), 0, s, a);                                          \
        return hipGetLastError();                                                               \
    }
    BM_ROW_FORMS(DO)
#undef DO
    return hipErrorInvalidValue;
}

template <typename T, bool Q8, bool DSUM>
hipError_t launch_b(const LnBwdArgs &a, int wgs, hipStream_t s) {
#define DO(E, TPR)                                                                              \
    if (a.C <= E * TPR) {                                                                       \
        BM_LAUNCH("layer_norm_bwd", (k_layer_norm_bwd<T, E, TPR, Q8, DSUM>), dim3((unsigned)wgs),  \
                  dim3(TPR > 64 ? TPR : 256), 0, s, a);                                          \
        return hipGetLastError();                                                               \
    }
    BM_ROW_FORMS(DO)
#undef DO
    return hipErrorInvalidValue;
}

template <typename T>
hipError_t launch_fwd_t(const LnArgs &a, hipStream_t s) {
    if (a.res) return a.q ? launch_fwd<T, true, true>(a, s) : launch_fwd<T, true, false>(a, s);
    return a.q ? launch_fwd<T, false, true>(a, s) : launch_fwd<T, false, false>(a, s);
}
template <typename T>
hipError_t launch_b_t(const LnBwdArgs &a, int wgs, hipStream_t s) {
    if (a.xscale) return a.dsum ? launch_b<T, true, true>(a, wgs, s) : launch_b<T, true, false>(a, wgs, s);
    return a.dsum ? launch_b<T, false, true>(a, wgs, s) : launch_b<T, false, false>(a, wgs, s);
}

}  // namespace

hipError_t launch_layer_norm(const LnArgs &a, bool bf16, hipStream_t s) {
    if (a.rows == 0) return hipSuccess;
    return bf16 ? launch_fwd_t<uint16_t>(a, s) : launch_fwd_t<float>(a, s);
}

// workgroups of the gradient: each leaves one row of 2 C partial sums
int layer_norm_bwd_wgs(long long rows, int C) {
    const long long per = C > 2048 ? 1 : 4, wgs = (rows + per - 1) / per;
    return (int)(wgs < 512 ? wgs : 512);
}

hipError_t launch_layer_norm_bwd(const LnBwdArgs &a, bool bf16, hipStream_t s) {
    const int wgs = layer_norm_bwd_wgs(a.rows, a.C);
    if (a.rows > 0) {
        hipError_t e = bf16 ? launch_b_t<uint16_t>(a, wgs, s) : launch_b_t<float>(a, wgs, s);
        if (e != hipSuccess) return e;
    }
    if (!a.dw && !a.db) return hipSuccess;
    const ColSum c{a.part, wgs, a.C, 1, 1, a.dw, a.db};
    return launch_col_sum(&c, 1, s);
}

}  // namespace bm
