// RMS norm of the residual stream in front of a mixer block, to the dtype or
// straight to the 8-bit rows that the integer product reads (linear8.hip).
// Per row (token) of C channels:
//   h = x + residual (rounded to the dtype), rstd = (mean h^2 + eps)^-1/2,
//   o = h rstd w
//   8-bit rows: top = max |o|, scale = top / 127, q = round(o 127 / top)
// with 127 / top and the product each rounded to fp32 and round() to the
// nearest integer, ties to even. A row with top < 2^-100 stands for zeros
// (scale 0); one that holds an infinity or a NaN has a NaN for its scale and
// zeros for q. Without the norm (rows8_pack) o is x.
//
// A stream bounded by HBM: the row stays in registers from its one read to its
// one write (rows laid over the lanes as row_form.hpp says), the next row's
// loads are under way meanwhile. max |o| is rstd max |h w| up to the rounding
// of the two products, so one exchange over a row's waves gives both the sum
// and the largest magnitude: o is taken as (h w) rstd, whose rounding keeps
// the order of magnitudes, and its largest is exactly round(max |h w| rstd).
// A row whose mean square leaves fp32 (values from 1e19, or tiny ones with no eps to
// speak of) is taken once more from its registers, times a power of two.
//
// Measured (bf16, residual, 8-bit rows alone): 131 072 x 2048 350 us, 1.88 GB at 5.4
// TB/s (a copy of that size moves 5.1); 8192 x 4096 36 us, 6.5 TB/s, some of it out of
// the last-level cache; 64 x 2560 3.6 us. To bf16 alone: 131 072 x 2048 396 us, 5.4 TB/s.
#include <type_traits>

#include "row_form.hpp"

namespace bm {
namespace {

constexpr int kRows = 4;   // waves of a workgroup where a row has at most one

// largest over the lanes of a row within a wave, the same in each of them
template <int G>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
    v = max(v, dpp<0xB1>(v));
    v = max(v, dpp<0x4E>(v));
    v = max(v, dpp<0x141>(v));
    if constexpr (G != 8) v = max(v, dpp<0x140>(v));
    if constexpr (G == 0 || G > 16) v = max(v, (uint32_t)__shfl_xor((int)v, 16));
    if constexpr (G == 0 || G > 32) v = max(v, (uint32_t)__shfl_xor((int)v, 32));
    return v;
}

template <typename T, int NV, int G, bool NORM, bool RES, bool OUT, bool Q8>
__global__ __launch_bounds__(G == 0 ? 64 * kMaxWaves : 64 * kRows) void k_rms_norm(RmsArgs a) {
    using L = Lane<T>;
    constexpr int V = L::V;
    constexpr bool MULTI = G == 0;
    constexpr int kShare = MULTI ? 1 : 64 / G;   // rows of a wave
    __shared__ float2 part[MULTI ? 3 : 1][MULTI ? kMaxWaves : 1];
    const int C = a.C;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t = MULTI ? threadIdx.x : threadIdx.x & (G - 1), lanes = MULTI ? blockDim.x : G;
    const Place<V, NV> at(C, t, lanes);
    const float inv = 1.0f / (float)C;
    float w[NV][V];
#pragma unroll
    for (int k = 0; k < NV; ++k) load_w<V>(a.w, at.c[k], 1.f, w[k]);
    const long long step = (long long)gridDim.x * (MULTI ? 1 : kRows * kShare);
    long long row = (long long)blockIdx.x * (MULTI ? 1 : kRows * kShare) + (MULTI ? 0 : wave * kShare);
    if (kShare > 1) row += (threadIdx.x & 63) / (MULTI ? 64 : G);
    rvec nx[NV], nr[RES ? NV : 1];
    auto fetch = [&](long long r) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            nx[k] = L::load((const T *)a.x + r * C + at.c[k]);
            if constexpr (RES) nr[k] = L::load((const T *)a.res + r * C + at.c[k]);
        }
    };
    constexpr bool kAhead = NV * V <= 16;   // wider lanes have no registers for it
    if (kAhead && row < a.rows) fetch(row);
    for (int flip = 0; row < a.rows; row += step, flip ^= 1) {
        if (!kAhead) fetch(row);
        rvec r[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            r[k] = nx[k];
            if constexpr (RES) {
                float h[V];
#pragma unroll
                for (int j = 0; j < V; ++j) h[j] = L::get(nx[k], j) + L::get(nr[k], j);
                r[k] = L::pack(h);   // the stream is kept in its dtype, and the norm sees what is kept
            }
        }
        if (kAhead && row + step < a.rows) fetch(row + step);
        float o[NV][V];
        float ss;
        uint32_t top;
        // h w of the lane's elements, and the row's sum of h^2 and largest |h w|, with h
        // times `by` (a power of two, 1 in the first pass)
        auto pass = [&](auto first, float by) {
            constexpr bool kFirst = decltype(first)::value;
            auto value = [&](int k, int j) { return kFirst ? L::get(r[k], j) : L::get(r[k], j) * by; };
            ss = 0.f;
            top = 0;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                float s = 0.f;
                uint32_t m = 0;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float h = value(k, j);
                    if constexpr (NORM) s = fmaf(h, h, s);
                    o[k][j] = NORM ? h * w[k][j] : h;
                    if constexpr (Q8) m = max(m, abs_bits(o[k][j]));
                }
                if (NORM && k == at.kt) {
                    s = 0.f;
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const float h = at.own(k, j, value(k, j));
                        s = fmaf(h, h, s);
                    }
                }
                // lanes past the row's end hold its last vector again
                ss += at.has[k] ? s : 0.f;
                top = max(top, m);
            }
            if constexpr (NORM) ss = lanes_total<G>(ss);
            if constexpr (Q8) top = lanes_max<G>(top);
            if constexpr (MULTI) {
                // the second pass has a place of its own, which the next row's barrier frees
                float2 *const p = part[kFirst ? flip : 2];
                if ((t & 63) == 0) p[wave] = make_float2(ss, __uint_as_float(top));
                __syncthreads();
                ss = 0.f;
                top = 0;
                for (int i = 0; i < (lanes >> 6); ++i) {
                    ss += p[i].x;
                    top = max(top, __float_as_uint(p[i].y));
                }
            }
        };
        pass(std::true_type(), 1.f);
        float rstd = 1.f, by = 1.f;   // of h times `by`
        if constexpr (NORM) {
            float mean = fmaf(ss, inv, a.eps);
            // Squares that overflow, or underflow where eps lets them count: once more,
            // with the row scaled to where they do neither
            if (!(mean >= 0x1p-100f && mean < __builtin_inff())) {
                by = mean < 1.f ? 0x1p100f : 0x1p-80f;
                // (the compiler would keep the first pass's values for it: of 2048 channels
                // to 8 bits 110 registers and 361 us, so 94 and 354)
#pragma unroll
                for (int k = 0; k < NV; ++k) asm volatile("" : "+v"(r[k]));
                pass(std::false_type(), by);
                mean = fmaf(ss, inv, a.eps * by * by);
            }
            rstd = 1.0f / sqrtf(mean);
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int j = 0; j < V; ++j) o[k][j] *= rstd;
        }
        float unit = 0.f, scale = 0.f;   // 127 / top and top / 127
        bool none = false;               // no finite largest magnitude
        if constexpr (Q8) {
            const float m = NORM ? __uint_as_float(top) * rstd : __uint_as_float(top);
            none = !(m < __builtin_inff());
            if (m >= 0x1p-100f) {
                unit = 127.0f / m;
                scale = m / 127.0f;
            }
            if (none) scale = __uint_as_float(0x7fc00000u);
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (!at.has[k]) continue;
            if constexpr (OUT) L::store((T *)a.out + row * C + at.c[k], L::pack(o[k]));
            if constexpr (RES) L::store((T *)a.sum + row * C + at.c[k], r[k]);
            if constexpr (Q8) {
                uint32_t code[V];
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float v = __builtin_amdgcn_fmed3f(rintf(o[k][j] * unit), -127.f, 127.f);
                    code[j] = none ? 0u : (uint32_t)(int)v;
                }
                Bytes<V>::store(a.q + row * C + at.c[k], Bytes<V>::pack(code));
            }
        }
        if (t == 0) {
            if constexpr (NORM) {
                if (a.rstd) a.rstd[row] = rstd * by;
            }
            if constexpr (Q8) a.scale[row] = scale;
        }
    }
}

template <typename T, bool NORM, bool RES, bool OUT, bool Q8>
hipError_t launch(const RmsArgs &a, hipStream_t s) {
    const Form f = row_form<T>(a.C, 16);
    const long long per = f.G ? kRows * (64 / f.G) : 1, wgs = (a.rows + per - 1) / per;
    // two turns a workgroup, more only if that makes a grid beyond the largest
    const long long half = (wgs + 1) / 2, most = 1 << 20;
    const dim3 grid((unsigned)(wgs < 2048 ? wgs : half < 2048 ? 2048 : half < most ? half : most));
    const dim3 block(64 * (f.G ? kRows : f.waves));
#define GO(NV, G_)                                                                                       \
    if (f.nv == NV && f.G == G_) {                                                                       \
        BM_LAUNCH(NORM ? "rms_norm" : "rows8_pack", (k_rms_norm<T, NV, G_, NORM, RES, OUT, Q8>), grid,    \
                  block, 0, s, a);                                                                       \
        return hipGetLastError();                                                                        \
    }
    constexpr int N8 = 8 * sizeof(T) / 16;   // vectors that make 8 elements
    GO(N8, 8) GO(N8, 16) GO(N8, 32)
    GO(N8, 64) GO(2 * N8, 64) GO(2 * N8, 0) GO(4 * N8, 0)
#undef GO
    return hipErrorInvalidValue;
}

template <typename T>
hipError_t launch_t(const RmsArgs &a, hipStream_t s) {
    if (!a.norm) return launch<T, false, false, false, true>(a, s);
    if (!a.q) return a.res ? launch<T, true, true, true, false>(a, s) : launch<T, true, false, true, false>(a, s);
    if (!a.out) return a.res ? launch<T, true, true, false, true>(a, s) : launch<T, true, false, false, true>(a, s);
    return a.res ? launch<T, true, true, true, true>(a, s) : launch<T, true, false, true, true>(a, s);
}

}  // namespace

hipError_t launch_rms_norm(const RmsArgs &a, bool bf16, hipStream_t s) {
    if (a.rows == 0) return hipSuccess;
    return bf16 ? launch_t<uint16_t>(a, s) : launch_t<float>(a, s);
}

}  // namespace bm
