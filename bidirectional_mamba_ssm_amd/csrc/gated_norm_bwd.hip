// Gradient of the gated RMS norm (epilogue.hip). With s = silu(z), v = y s,
// r = (mean over the group of v^2 + eps)^-1/2 and g = dout w:
//   dv = r (g - v r^2 mean(g v)),  dy = dv s,
//   dz = dv y sig(z) (1 + z (1 - sig(z))),  dw = sum over rows of dout v r
// y and z may be read back from 8-bit checkpoints (rows.hpp).
//
// A stream bounded by HBM: y, z and dout are read once, dy and dz written
// once. One workgroup of four waves per token at a time, laid out like the
// forward kernel: lane l of wave w holds channels 1024k + 256w + 4l .. +3 of
// pass k, so a group (a multiple of 256 channels) is a run of whole (pass,
// wave) chunks. Both sums a row needs, of v^2 and of g v, come from one walk
// over the registers and cost one barrier. dw stays in registers over the
// rows a workgroup walks and is joined by col_sum.hip.
#include "internal.hpp"
#include "rows.hpp"

namespace bm {
namespace {

constexpr int kThreads = 256;

typedef uint32_t w2 __attribute__((ext_vector_type(2)));

// four channels of one lane: fp32, bf16 or 8-bit
template <typename T> struct Quad;
template <> struct Quad<float> {
    rvec r;
    __device__ __forceinline__ void load(const void *p, const uint8_t *, size_t row, int C, int c) {
        r = *(const rvec *)((const float *)p + row * C + c);
    }
    __device__ __forceinline__ float get(int j) const { return __uint_as_float(r[j]); }
    __device__ __forceinline__ static void store(float *p, const float *v) {
        *(float4 *)p = make_float4(v[0], v[1], v[2], v[3]);
    }
};
template <> struct Quad<uint16_t> {
    w2 r;
    __device__ __forceinline__ void load(const void *p, const uint8_t *, size_t row, int C, int c) {
        r = *(const w2 *)((const uint16_t *)p + row * C + c);
    }
    __device__ __forceinline__ float get(int j) const {
        return __uint_as_float((j & 1) ? (r[j >> 1] & 0xffff0000u) : (r[j >> 1] << 16));
    }
    __device__ __forceinline__ static void store(uint16_t *p, const float *v) {
        const rf2 a = {v[0], v[1]}, b = {v[2], v[3]};
        w2 o;
        o[0] = __builtin_bit_cast(uint32_t, __builtin_convertvector(a, rbf2));
        o[1] = __builtin_bit_cast(uint32_t, __builtin_convertvector(b, rbf2));
        *(w2 *)p = o;
    }
};
template <> struct Quad<int8_t> {
    uint32_t r;
    uint32_t e;
    __device__ __forceinline__ void load(const void *p, const uint8_t *scale, size_t row, int C, int c) {
        r = *(const uint32_t *)((const int8_t *)p + row * C + c);
        e = scale[row * (C / 32) + c / 32];
    }
    __device__ __forceinline__ float get(int j) const { return (float)Bytes<4>::get(r, j) * act8_unit(e); }
};

template <typename T, typename TY, typename TZ, int KP>
__global__ __launch_bounds__(kThreads) void k_gated_norm_bwd(EpiBwdArgs a) {
    __shared__ float2 part[2][KP * 4];
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const int C = a.C, nq = a.gs / 256, groups = C / a.gs;
    const float inv = 1.0f / (float)a.gs;
    float w[KP][4], dw[KP][4];
#pragma unroll
    for (int k = 0; k < KP; ++k) {
        const int c = 1024 * k + 4 * tid;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            w[k][j] = c < C ? a.w[c + j] : 0.f;
            dw[k][j] = 0.f;
        }
    }
    int buf = 0;
    for (size_t row = blockIdx.x; row < (size_t)a.rows; row += gridDim.x, buf ^= 1) {
        Quad<TY> y[KP];
        Quad<TZ> z[KP];
        Quad<T> d[KP];
#pragma unroll
        for (int k = 0; k < KP; ++k) {
            // lanes past the last channel read the last four again
            const int c = min(1024 * k + 4 * tid, C - 4);
            y[k].load(a.y, a.yscale, row, C, c);
            z[k].load(a.z, a.zscale, row, C, c);
            d[k].load(a.dout, nullptr, row, C, c);
        }
        float v[KP][4], sg[KP][4];
#pragma unroll
        for (int k = 0; k < KP; ++k) {
            float vv = 0.f, gv = 0.f;
            const bool ok = 1024 * k + 256 * wave < C;   // whole chunks of 256
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float zj = z[k].get(j);
                sg[k][j] = __builtin_amdgcn_rcpf(1.0f + __expf(-zj));
                v[k][j] = y[k].get(j) * (zj * sg[k][j]);
                vv = fmaf(v[k][j], v[k][j], vv);
                gv = fmaf(d[k].get(j) * w[k][j], v[k][j], gv);
            }
            vv = wave_total(vv);
            gv = wave_total(gv);
            if (lane == 0) part[buf][4 * k + wave] = ok ? make_float2(vv, gv) : make_float2(0.f, 0.f);
        }
        __syncthreads();
        // lane g adds up group g's chunks; every wave does so for itself
        float gv2 = 0.f, ggv = 0.f;
        if (lane < groups)
            for (int q = 0; q < nq; ++q) {
                const float2 p = part[buf][lane * nq + q];
                gv2 += p.x;
                ggv += p.y;
            }
        const float r_l = 1.0f / sqrtf(gv2 * inv + a.eps);
        const float m_l = ggv * inv * r_l * r_l;
        float *dy = a.dy + row * C;
        T *dz = (T *)a.dz + row * C;
#pragma unroll
        for (int k = 0; k < KP; ++k) {
            const int chunk = 4 * k + wave;
            const int c = 1024 * k + 4 * tid;
            if (256 * chunk >= C) break;
            const int g = chunk / nq;
            const float r = __shfl(r_l, g), m = __shfl(m_l, g);
            float oy[4], oz[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float dj = d[k].get(j), zj = z[k].get(j), s = sg[k][j];
                dw[k][j] = fmaf(dj, v[k][j] * r, dw[k][j]);
                const float dv = r * (dj * w[k][j] - v[k][j] * m);
                oy[j] = dv * (zj * s);
                oz[j] = dv * y[k].get(j) * (s * (1.0f + zj * (1.0f - s)));
            }
            Quad<float>::store(dy + c, oy);
            Quad<T>::store(dz + c, oz);
        }
    }
    if (!a.part) return;
    float *out = a.part + (size_t)blockIdx.x * C;
#pragma unroll
    for (int k = 0; k < KP; ++k) {
        const int c = 1024 * k + 4 * tid;
        if (c < C) Quad<float>::store(out + c, dw[k]);
    }
}

template <typename T, typename TY, typename TZ>
hipError_t launch_t(const EpiBwdArgs &a, int wgs, hipStream_t s) {
    const dim3 grid((unsigned)wgs);
#define GO(KP) BM_LAUNCH("gated_norm_bwd", (k_gated_norm_bwd<T, TY, TZ, KP>), grid, dim3(kThreads), 0, s, a)
    if (a.C <= 1024) GO(1);
    else if (a.C <= 2048) GO(2);
    else if (a.C <= 4096) GO(4);
    else GO(8);
#undef GO
    return hipGetLastError();
}

template <typename T>
hipError_t launch_d(const EpiBwdArgs &a, int wgs, hipStream_t s) {
    if (a.yscale) return a.zscale ? launch_t<T, int8_t, int8_t>(a, wgs, s) : launch_t<T, int8_t, T>(a, wgs, s);
    return a.zscale ? launch_t<T, float, int8_t>(a, wgs, s) : launch_t<T, float, T>(a, wgs, s);
}

}  // namespace

int gated_norm_bwd_wgs(long long rows) { return (int)(rows < 1024 ? rows : 1024); }

hipError_t launch_gated_norm_bwd(const EpiBwdArgs &a, bool bf16, hipStream_t s) {
    const int wgs = gated_norm_bwd_wgs(a.rows);
    if (a.rows > 0) {
        hipError_t e = bf16 ? launch_d<uint16_t>(a, wgs, s) : launch_d<float>(a, wgs, s);
        if (e != hipSuccess) return e;
    }
    if (!a.dw) return hipSuccess;
    const ColSum c{a.part, wgs, a.C, 1, 0, a.dw, nullptr};
    return launch_col_sum(&c, 1, s);
}

}  // namespace bm
