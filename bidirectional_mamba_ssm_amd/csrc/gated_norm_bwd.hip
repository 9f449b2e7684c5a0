// Gradient of the gated RMS norm (epilogue.hip). With s = silu(z), v = y s,
// r = (mean over the group of v^2 + eps)^-1/2 and g = dout w:
//   dv = r (g - v r^2 mean(g v)),  dy = dv s,
//   dz = dv y sig(z) (1 + z (1 - sig(z))),  dw = sum over rows of dout v r
// y and z may be read back from 8-bit checkpoints (rows.hpp).
//
// A stream bounded by HBM: y, z and dout are read once, dy and dz written
// once. A row of n chunks of 256 channels is held by W waves, KP chunks each
// (chunk k W + wave, four channels a lane), R rows at a time by a workgroup
// of up to 8 or 16 waves; a group is a run of whole chunks. Both sums that a row
// needs, of v^2 and of g v, come from one walk over the registers and cost
// one barrier, and the next row's loads are under way meanwhile. dw stays in
// registers over the rows that a workgroup walks and is joined by col_sum.hip.
//
// Measured (bf16): 8192 x 4096, one group, 90 us, 470 MB at 5.2 TB/s, and 5 us
// for the sums; 3001 x 5120, groups of 1280, both checkpoints, 34 us, 155 MB at
// 4.5 TB/s. Four chunks a wave need 210 registers, so that 5-wave workgroups
// took two rounds (44 us); loads of eight passes for five chunks 62.
#include "internal.hpp"
#include "rows.hpp"

namespace bm {
namespace {

// waves of a workgroup at most, with KP chunks a wave
constexpr int kWaves(int kp) { return kp == 1 ? 8 : 16; }

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
    uint32_t r, e;
    __device__ __forceinline__ void load(const void *p, const uint8_t *scale, size_t row, int C, int c) {
        r = *(const uint32_t *)((const int8_t *)p + row * C + c);
        e = scale[row * (C / 32) + c / 32];
    }
    __device__ __forceinline__ float get(int j) const {
        float v[4];
        values4(r, act8_unit(e), v);
        return v[j];
    }
};

template <typename T, typename TY, typename TZ, int KP>
__global__ __launch_bounds__(64 * kWaves(KP)) void k_gated_norm_bwd(EpiBwdArgs a, int W, int R) {
    __shared__ float2 part[2][kWaves(KP) * KP];
    __shared__ float sum[KP == 1 ? 4 * 256 : 1];   // joins dw where R > 1 (then W <= 4 and KP = 1)
    const int wave_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int sub = wave_all / W, wave = wave_all - sub * W, lane = threadIdx.x & 63;
    const int C = a.C, n = C / 256, nq = a.gs / 256, groups = C / a.gs;
    const float inv = 1.0f / (float)a.gs;
    // lanes of a chunk past the last one read the last one again, and store nothing
    int at[KP];
    float w[KP][4], dw[KP][4];
#pragma unroll
    for (int k = 0; k < KP; ++k) {
        at[k] = 256 * min(k * W + wave, n - 1) + 4 * lane;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            w[k][j] = a.w[at[k] + j];
            dw[k][j] = 0.f;
        }
    }
    struct Row {
        Quad<TY> y[KP];
        Quad<TZ> z[KP];
        Quad<T> d[KP];
    };
    auto fetch = [&](Row &o, long long row) {
#pragma unroll
        for (int k = 0; k < KP; ++k) {
            o.y[k].load(a.y, a.yscale, row, C, at[k]);
            o.z[k].load(a.z, a.zscale, row, C, at[k]);
            o.d[k].load(a.dout, nullptr, row, C, at[k]);
        }
    };
    // all waves make the same turns (the barrier); one without a row reads the
    // last one and uses nothing of it
    const long long step = (long long)gridDim.x * R, last = a.rows - 1;
    long long base = (long long)blockIdx.x * R;
    Row next;
    fetch(next, min(base + sub, last));
    for (int buf = 0; base < a.rows; base += step, buf ^= 1) {
        const long long row = base + sub;
        const bool live = row < a.rows;
        const Row r = next;
        fetch(next, min(row + step, last));
        float v[KP][4], gate[KP][4], slope[KP][4];
#pragma unroll
        for (int k = 0; k < KP; ++k) {
            float vv = 0.f, gv = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float z = r.z[k].get(j), y = r.y[k].get(j);
                const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-z));
                gate[k][j] = z * s;
                slope[k][j] = y * (s * fmaf(z, 1.0f - s, 1.0f));
                v[k][j] = y * gate[k][j];
                vv = fmaf(v[k][j], v[k][j], vv);
                gv = fmaf(r.d[k].get(j) * w[k][j], v[k][j], gv);
            }
            vv = wave_total(vv);
            gv = wave_total(gv);
            if (lane == 0 && k * W + wave < n) part[buf][sub * n + k * W + wave] = make_float2(vv, gv);
        }
        __syncthreads();
        if (!live) continue;
        // lane g adds up group g's chunks; every wave does so for itself
        float vv = 0.f, gv = 0.f;
        if (lane < groups)
            for (int q = 0; q < nq; ++q) {
                const float2 p = part[buf][sub * n + lane * nq + q];
                vv += p.x;
                gv += p.y;
            }
        const float r_l = 1.0f / sqrtf(vv * inv + a.eps);
        const float m_l = gv * inv * r_l * r_l;
#pragma unroll
        for (int k = 0; k < KP; ++k) {
            const int chunk = k * W + wave;
            if (chunk >= n) break;
            const int g = chunk / nq;
            const float rg = __shfl(r_l, g), m = __shfl(m_l, g);
            float oy[4], oz[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float d = r.d[k].get(j);
                dw[k][j] = fmaf(d, v[k][j] * rg, dw[k][j]);
                const float dv = rg * (d * w[k][j] - v[k][j] * m);
                oy[j] = dv * gate[k][j];
                oz[j] = dv * slope[k][j];
            }
            Quad<float>::store(a.dy + row * C + at[k], oy);
            Quad<T>::store((T *)a.dz + row * C + at[k], oz);
        }
    }
    if (!a.part) return;
    if constexpr (KP == 1) {
        for (int s = 0; s < R && R > 1; ++s) {   // the R rows' sums, in order
            if (sub == s) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float *p = sum + (j * W + wave) * 64 + lane;
                    if (s > 0) dw[0][j] += *p;
                    if (s < R - 1) *p = dw[0][j];
                }
            }
            __syncthreads();
        }
        if (sub != R - 1) return;
    }
#pragma unroll
    for (int k = 0; k < KP; ++k)
        if (k * W + wave < n) Quad<float>::store(a.part + (size_t)blockIdx.x * C + at[k], dw[k]);
}

// How a row is held: a chunk a wave up to 8 chunks, two beyond; rows of up to 4
// chunks share a workgroup (20 000 x 1024 from checkpoints: 39 us, one row a
// workgroup 54). All workgroups are resident at once (16 waves a CU), and walk
// the rows.
struct Form {
    int kp, waves, rows, wgs;
};
Form row_form(long long rows, int C) {
    const int n = C / 256;
    Form f;
    f.kp = n <= kWaves(1) ? 1 : 2;
    f.waves = (n + f.kp - 1) / f.kp;
    f.rows = f.waves > 4 ? 1 : kWaves(1) / f.waves;
    const long long wgs = (rows + f.rows - 1) / f.rows, most = f.waves > 8 ? 256 : 512;
    f.wgs = (int)(wgs < most ? wgs : most);
    return f;
}

template <typename T, typename TY, typename TZ>
hipError_t launch_t(const EpiBwdArgs &a, hipStream_t s) {
    const Form f = row_form(a.rows, a.C);
    const dim3 grid((unsigned)f.wgs), block(64 * f.waves * f.rows);
#define GO(KP)                                                                                             \
    BM_LAUNCH("gated_norm_bwd", (k_gated_norm_bwd<T, TY, TZ, KP>), grid, block, 0, s, a, f.waves, f.rows)
    if (f.kp == 1) GO(1);
    else GO(2);
#undef GO
    return hipGetLastError();
}

template <typename T>
hipError_t launch_d(const EpiBwdArgs &a, hipStream_t s) {
    if (a.yscale) return a.zscale ? launch_t<T, int8_t, int8_t>(a, s) : launch_t<T, int8_t, T>(a, s);
    return a.zscale ? launch_t<T, float, int8_t>(a, s) : launch_t<T, float, T>(a, s);
}

}  // namespace

// workgroups, each of which leaves a row of partial sums
int gated_norm_bwd_wgs(long long rows, int C) { return row_form(rows, C).wgs; }

hipError_t launch_gated_norm_bwd(const EpiBwdArgs &a, bool bf16, hipStream_t s) {
    if (a.rows > 0) {
        hipError_t e = bf16 ? launch_d<uint16_t>(a, s) : launch_d<float>(a, s);
        if (e != hipSuccess) return e;
    }
    if (!a.dw) return hipSuccess;
    const ColSum c{a.part, gated_norm_bwd_wgs(a.rows, a.C), a.C, 1, 0, a.dw, nullptr};
    return launch_col_sum(&c, 1, s);
}

}  // namespace bm
