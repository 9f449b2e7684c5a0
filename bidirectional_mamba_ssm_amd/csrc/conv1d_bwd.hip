// Gradient of the short convolution (conv1d.hip) of both directions. In scan
// positions p (token p forward, token L-1-p reverse) both directions are the
// same causal filter u_p = b + sum_k w_k in_{p-(W-1)+k}; given the output's
// gradient dout (fp32, as bimamba_ssd_bwd leaves it):
//   du_p = dout_p act'(u_p),   act' = sig(u) (1 + u (1 - sig(u))) for SiLU
//   din_p = sum_k w_k du_{p+(W-1)-k},
//   dw_k = sum_p du_p in_{p-(W-1)+k},   db = sum_p du_p
// terms across a row's or a packed sequence's ends left out. The input may be
// read from its 8-bit checkpoint (rows.hpp).
//
// A stream bounded by HBM: input and dout read once, din written once. A lane
// owns four adjacent channels and walks a run of positions with the last W-1
// inputs and du in registers: u_p and du_p are computed as p comes in, and
// din_{p-(W-1)}, whose last term du_p is, goes out. A run starts W-1
// positions early with its inputs and ends W-1 late with its du; four waves
// of a workgroup take adjacent runs. Rows are loaded kBatch positions ahead.
// The inner batches ask nothing and never wait for their own stores. dw and db
// stay in the lane's registers over the run, are joined over the
// workgroup through LDS and over workgroups by col_sum.hip.
//
// Measured (8 x 1024 tokens, 4352 channels, width 4, bf16, SiLU, both
// directions): 119 us, 571 MB at 4.8 TB/s, and 5 us for the sums; from the
// checkpoint 107 us, 502 MB at 4.7; packed, 32 sequences, 124; 128 rows of 64
// tokens, where half of a workgroup's waves have no run, 127 and 7; 2500 packed
// tokens of 96 channels in fp32 10 us. Tests in every batch 131; the inner
// batches' code shared with a store under a branch, which made each batch wait
// for the stores of the one before, 138. The arithmetic (432 vector
// instructions for 16 elements a lane) would take 60.
#include <type_traits>

#include "conv_seqs.hpp"
#include "internal.hpp"
#include "rows.hpp"

namespace bm {
namespace {

constexpr int kWaves = 4;
constexpr int kBatch = 4;   // positions loaded and worked on together, >= W - 1

typedef uint32_t w2 __attribute__((ext_vector_type(2)));

// VEC channels of one row of the input
template <typename T, bool Q8, int VEC> struct In;
template <> struct In<float, false, 4> {
    rvec r;
    __device__ __forceinline__ void load(const void *p, const uint8_t *, size_t row, int ch, int, int c) {
        r = *(const rvec *)((const float *)p + row * ch + c);
    }
    __device__ __forceinline__ void values(float *v) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = __uint_as_float(r[j]);
    }
};
template <> struct In<uint16_t, false, 4> {
    w2 r;
    __device__ __forceinline__ void load(const void *p, const uint8_t *, size_t row, int ch, int, int c) {
        r = *(const w2 *)((const uint16_t *)p + row * ch + c);
    }
    __device__ __forceinline__ void values(float *v) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = __uint_as_float((j & 1) ? (r[j >> 1] & 0xffff0000u) : (r[j >> 1] << 16));
    }
};
template <typename T> struct In<T, false, 1> {
    T r;
    __device__ __forceinline__ void load(const void *p, const uint8_t *, size_t row, int ch, int, int c) {
        r = ((const T *)p)[row * ch + c];
    }
    __device__ __forceinline__ void values(float *v) const { v[0] = Elem<T>::load(&r, 0); }
};
template <typename T> struct In<T, true, 4> {
    uint32_t r, e;
    __device__ __forceinline__ void load(const void *p, const uint8_t *scale, size_t row, int ch, int nblk, int c) {
        r = *(const uint32_t *)((const int8_t *)p + row * ch + c);
        e = scale[row * nblk + c / 32];
    }
    __device__ __forceinline__ void values(float *v) const { values4(r, act8_unit(e), v); }
};
template <typename T> struct In<T, true, 1> {
    int r;
    uint32_t e;
    __device__ __forceinline__ void load(const void *p, const uint8_t *scale, size_t row, int ch, int nblk, int c) {
        r = ((const int8_t *)p)[row * ch + c];
        e = scale[row * nblk + c / 32];
    }
    __device__ __forceinline__ void values(float *v) const { v[0] = (float)r * act8_unit(e); }
};

template <int VEC>
__device__ __forceinline__ void load_grad(const float *p, float (&v)[VEC]) {
    if constexpr (VEC == 4) {
        const float4 q = *(const float4 *)p;
        v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
    } else {
        v[0] = *p;
    }
}
template <int VEC>
__device__ __forceinline__ void store_in(float *p, const float (&v)[VEC]) {
    if constexpr (VEC == 4) *(float4 *)p = make_float4(v[0], v[1], v[2], v[3]);
    else *p = v[0];
}
template <int VEC>
__device__ __forceinline__ void store_in(uint16_t *p, const float (&v)[VEC]) {
    if constexpr (VEC == 4) {
        const rf2 a = {v[0], v[1]}, b = {v[2], v[3]};
        w2 o;
        o[0] = __builtin_bit_cast(uint32_t, __builtin_convertvector(a, rbf2));
        o[1] = __builtin_bit_cast(uint32_t, __builtin_convertvector(b, rbf2));
        *(w2 *)p = o;
    } else {
        *p = __builtin_bit_cast(uint16_t, (__bf16)v[0]);
    }
}

template <typename T, bool Q8, int VEC, int W, bool PACKED>
__global__ __launch_bounds__(64 * kWaves) void k_conv_bwd(ConvBwdArgs a) {
    constexpr int H = W - 1, N = H + kBatch;
    __shared__ float join[kWaves][VEC * (W + 1)][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // workgroup -> (row and direction, tile of runs, channel slab). Workgroups
    // go round robin over the 8 XCDs; each takes one stretch of the work, so
    // that adjacent tiles meet in one L2.
    const int per = (int)((gridDim.x + 7) / 8);
    const int work = (int)(blockIdx.x % 8) * per + (int)(blockIdx.x / 8);
    if (work >= a.wgs) return;
    const int slab = work % a.slabs;
    const int rest = work / a.slabs;
    const int tile = rest % a.tiles, unit = rest / a.tiles;
    const bool rev = unit % a.ndir != 0;
    const int b = unit / a.ndir;
    const ConvBwdDir d = rev ? a.dir[1] : a.dir[0];
    const int L = a.L, ch = a.ch, nblk = (ch + 31) / 32;
    const int cv = slab * 64 + lane;
    const bool chan_ok = cv < a.nvec;
    const int c0 = (chan_ok ? cv : a.nvec - 1) * VEC;   // lanes past the end store nothing

    float w[VEC][W], bias[VEC], aw[VEC][W], ab[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
#pragma unroll
        for (int k = 0; k < W; ++k) {
            w[j][k] = d.weight[(size_t)(c0 + j) * W + k];
            aw[j][k] = 0.f;
        }
        bias[j] = d.bias ? d.bias[c0 + j] : 0.f;
        ab[j] = 0.f;
    }
    // dout array of the lane: x, B or C
    const float *g;
    int gs;
    if (c0 < a.hp) {
        g = d.dx + c0; gs = a.hp;
    } else if (c0 < a.hp + a.gn) {
        g = d.dB + (c0 - a.hp); gs = a.gn;
    } else {
        g = d.dC + (c0 - a.hp - a.gn); gs = a.gn;
    }
    const size_t row0 = (size_t)b * L;
    const int p0 = (tile * kWaves + wave) * a.run;
    const int p1 = min(p0 + a.run, L);
    auto token = [&](int p) { return rev ? L - 1 - p : p; };

    if (p0 < L) {
        float win[N][VEC], du[N][VEC];
        In<T, Q8, VEC> next[kBatch];
        float gnext[kBatch][VEC];
        auto fetch = [&](int p) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int t = token(min(p + i, L - 1));   // positions past the end: zeroed when used
                next[i].load(d.xbc, d.xscale, row0 + t, ch, nblk, c0);
                load_grad<VEC>(g + (row0 + t) * gs, gnext[i]);
            }
        };
        // where the window of the batch from p has sequence starts
        StartBits starts;
        if constexpr (PACKED) starts = StartBits(a.packed, p0 - H, L, rev);
        auto window = [&](int p) -> uint32_t { return PACKED ? starts.from(p - p0, N) : 0u; };
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const int p = p0 - H + i;
            In<T, Q8, VEC> v;
            v.load(d.xbc, d.xscale, row0 + token(max(p, 0)), ch, nblk, c0);
            v.values(win[i]);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                if (p < 0) win[i][j] = 0.f;
                du[i][j] = 0.f;
            }
        }
        // kBatch positions from p. EDGE: some of them lie past the run's or the
        // row's end, some outputs before the run, or sequences meet (`first`);
        // elsewhere nothing is asked.
        auto batch = [&](int p, auto edge, uint32_t first) {
            constexpr bool EDGE = decltype(edge)::value;
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                next[i].values(win[H + i]);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    du[H + i][j] = gnext[i][j];
                    // a row past the end was read from the last one
                    if (EDGE && p + i >= L) win[H + i][j] = 0.f;
                }
            }
            if (!EDGE || p + kBatch < p1 + H) fetch(p + kBatch);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const bool own = !EDGE || p + i < p1, live = !EDGE || p + i < L;
                const int s = p + i - H;
                float o[VEC];
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    float tap[W];
                    float u = bias[j];
#pragma unroll
                    for (int k = 0; k < W; ++k) {
                        // no start among window positions i + k + 1 .. i + H
                        const bool same = !PACKED || !EDGE || !(first >> (i + k + 1) & ((1u << (H - k)) - 1));
                        tap[k] = same ? win[i + k][j] : 0.f;
                        u = fmaf(w[j][k], tap[k], u);
                    }
                    const float sg = __builtin_amdgcn_rcpf(1.0f + __expf(-u));
                    const float slope = sg * fmaf(u, 1.0f - sg, 1.0f);
                    float v = du[H + i][j] * (a.act ? slope : 1.0f);
                    // a position past the end has no gradient, whatever its slope
                    if (!live) v = 0.f;
                    du[H + i][j] = v;
                    // another run's position counts there: its taps may be
                    // infinite, and a zero times that is no zero
                    if (own) {
                        ab[j] += v;
#pragma unroll
                        for (int k = 0; k < W; ++k) aw[j][k] = fmaf(v, tap[k], aw[j][k]);
                    }
                    o[j] = 0.f;
#pragma unroll
                    for (int k = 0; k < W; ++k) {
                        // no start among window positions i + 1 .. i + k
                        const bool same = !PACKED || !EDGE || !(first >> (i + 1) & ((1u << k) - 1));
                        o[j] = fmaf(w[j][H - k], same ? du[i + k][j] : 0.f, o[j]);
                    }
                }
                // lanes past the last channel vector hold its very values
                if (!EDGE || (s >= p0 && s < p1))
                    store_in<VEC>((T *)d.dxbc + (row0 + token(s)) * ch + c0, o);
            }
#pragma unroll
            for (int i = 0; i < H; ++i)
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    win[i][j] = win[kBatch + i][j];
                    du[i][j] = du[kBatch + i][j];
                }
        };
        fetch(p0);
        int p = p0;
        do {
            batch(p, std::true_type(), window(p));
            p += kBatch;
            // Loads and stores share a counter. With everything arrived here,
            // each turn of the inner loop waits for the loads of the turn
            // before and leaves that turn's stores, which come after them, alone.
            __builtin_amdgcn_s_waitcnt(0x0f70);   // vmcnt(0)
            for (; p + kBatch <= p1 && window(p) == 0; p += kBatch) batch(p, std::false_type(), 0u);
        } while (p < p1 + H);
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
#pragma unroll
        for (int k = 0; k < W; ++k) join[wave][k * VEC + j][lane] = aw[j][k];
        join[wave][W * VEC + j][lane] = ab[j];
    }
    __syncthreads();
    // wave v joins taps v, v + 4 (tap W is the bias)
    float *part = d.part + (size_t)(b * a.tiles + tile) * (W + 1) * ch;
    for (int k = wave; k <= W; k += kWaves) {
        float o[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            o[j] = 0.f;
#pragma unroll
            for (int v = 0; v < kWaves; ++v) o[j] += join[v][k * VEC + j][lane];
        }
        if (chan_ok) store_in<VEC>(part + (size_t)k * ch + c0, o);
    }
}

template <typename T, bool Q8, int VEC, int W>
hipError_t launch_w(const ConvBwdArgs &a, hipStream_t s) {
    const dim3 grid((unsigned)((a.wgs + 7) / 8 * 8));
    if (a.packed.seq || a.packed.count) BM_LAUNCH("conv1d_bwd_packed", (k_conv_bwd<T, Q8, VEC, W, true>), grid, dim3(64 * kWaves), 0, s, a);
    else BM_LAUNCH("conv1d_bwd", (k_conv_bwd<T, Q8, VEC, W, false>), grid, dim3(64 * kWaves), 0, s, a);
    return hipGetLastError();
}
template <typename T, bool Q8, int VEC>
hipError_t launch_v(const ConvBwdArgs &a, hipStream_t s) {
    switch (a.W) {
        case 2: return launch_w<T, Q8, VEC, 2>(a, s);
        case 3: return launch_w<T, Q8, VEC, 3>(a, s);
        case 4: return launch_w<T, Q8, VEC, 4>(a, s);
    }
    return hipErrorInvalidValue;
}
template <typename T>
hipError_t launch_t(const ConvBwdArgs &a, bool vec, hipStream_t s) {
    if (a.dir[0].xscale) return vec ? launch_v<T, true, 4>(a, s) : launch_v<T, true, 1>(a, s);
    return vec ? launch_v<T, false, 4>(a, s) : launch_v<T, false, 1>(a, s);
}

// Positions a wave walks: 32, or fewer where that leaves the chip short of
// waves (a run repeats W - 1 rows at either end; 8 x 1024 tokens of 4352
// channels: 32 122 us, 64 131, 96 145, 16 125; 2500 x 96: 8 8.6 us, 16 11.4,
// 16384 x 96, 2048 waves of 16: 14, of 8: 16.5).
int run_length(int batch, int L, int slabs, int ndir) {
    int run = 32;
    auto waves = [&] { return (long long)((L + run - 1) / run) * slabs * batch * ndir; };
    while (run > 16 && waves() < 2048) run /= 2;
    if (waves() < 1024) run /= 2;
    return run;
}
int tiles_of(int L, int run) { return (L + run * kWaves - 1) / (run * kWaves); }
int slabs_of(int hp, int gn, int *nvec) {
    *nvec = (hp + 2 * gn) / (conv_vectorized(true, hp, gn) ? 4 : 1);
    return (*nvec + 63) / 64;
}

}  // namespace

size_t conv_bwd_part(int batch, int L, int hp, int gn, int W, int ndir) {
    int nvec;
    const int slabs = slabs_of(hp, gn, &nvec);
    return (size_t)batch * tiles_of(L, run_length(batch, L, slabs, ndir)) * (W + 1) * (hp + 2 * gn);
}

hipError_t launch_conv_bwd(ConvBwdArgs a, bool bf16, hipStream_t s) {
    a.slabs = slabs_of(a.hp, a.gn, &a.nvec);
    a.run = run_length(a.batch, a.L, a.slabs, a.ndir);
    a.tiles = tiles_of(a.L, a.run);
    a.wgs = a.slabs * a.tiles * a.batch * a.ndir;
    if (a.L > 0) {
        const bool vec = conv_vectorized(bf16, a.hp, a.gn);
        hipError_t e = bf16 ? launch_t<uint16_t>(a, vec, s) : launch_t<float>(a, vec, s);
        if (e != hipSuccess) return e;
    }
    ColSum sets[2];
    for (int i = 0; i < a.ndir; ++i)
        sets[i] = ColSum{a.dir[i].part, a.batch * a.tiles, a.ch, a.W, 1, a.dir[i].dw, a.dir[i].db};
    return launch_col_sum(sets, a.ndir, s);
}

}  // namespace bm
