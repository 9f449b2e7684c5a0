// The short convolution (conv1d.hip) of both directions from 8-bit
// checkpoints of its input (rows.hpp): what a training step's backward pass
// rebuilds the scan's inputs with. In scan positions p (token p forward, token
// L-1-p reverse) both directions are the same causal filter
//   u_p = b + sum_k w_k in_{p-(W-1)+k},  out_p = silu(u_p) or u_p.
//
// A stream bounded by HBM: 1 + 1/32 bytes of every element read, its output
// written once. A lane owns VEC adjacent channels and walks a run of positions
// with the last W-1 inputs, decoded once, in registers; rows are loaded
// kBatch positions ahead, and a run starts W-1 positions early.
//
// At 8 x 1024 tokens of 4352 channels, width 4, bf16, SiLU, both directions:
// 44 us, 216 MB at 4.9 TB/s, where launches follow one another for long, 49
// where the clock has just risen from idle (the convolution from bf16 input: 54
// us, 285 MB); 8192 packed tokens, 32 sequences, 49 us.
// Its arithmetic alone takes some 35 us (212 vector instructions for 16
// elements a lane, 32 of them exp and rcp at a quarter of the rate), so what
// it spends elsewhere shows: pointers that walk with the rows instead of a
// product each, no test of the activation, a window that is not moved, 62 ->
// 43 us together with the walk itself (the bf16 kernel's form, with a decoding
// load, took 62). 8 channels a lane need 180 registers and ran 66 us; runs of
// 16 or 64 positions 50.
#include <type_traits>

#include "conv_seqs.hpp"
#include "internal.hpp"
#include "rows.hpp"

namespace bm {
namespace {

constexpr int kWaves = 4;
constexpr int kBatch = 4;   // positions loaded and worked on together, >= W - 1

template <int VEC> struct Codes {
    typename Bytes<VEC>::type r;
    uint32_t e;
    __device__ __forceinline__ void load(const int8_t *q, const uint8_t *scale) {
        r = Bytes<VEC>::load(q);
        e = *scale;
    }
    __device__ __forceinline__ void values(float *v) const { Bytes<VEC>::values(r, act8_unit(e), v); }
};
template <> struct Codes<1> {
    int r;
    uint32_t e;
    __device__ __forceinline__ void load(const int8_t *q, const uint8_t *scale) {
        r = *q;
        e = *scale;
    }
    __device__ __forceinline__ void values(float *v) const { v[0] = (float)r * act8_unit(e); }
};

typedef uint32_t u2_a8 __attribute__((ext_vector_type(2)));

template <typename T, int VEC>
__device__ __forceinline__ void store_out(T *p, const float *v) {
    if constexpr (VEC == 1) {
        if constexpr (sizeof(T) == 2) *p = __builtin_bit_cast(uint16_t, (__bf16)v[0]);
        else *p = v[0];
    } else if constexpr (VEC * sizeof(T) == 8) {
        const rf2 lo = {v[0], v[1]}, hi = {v[2], v[3]};
        *(u2_a8 *)p = u2_a8{__builtin_bit_cast(uint32_t, __builtin_convertvector(lo, rbf2)),
                            __builtin_bit_cast(uint32_t, __builtin_convertvector(hi, rbf2))};
    } else {
#pragma unroll
        for (int i = 0; i < VEC / Lane<T>::V; ++i) Lane<T>::store(p + i * Lane<T>::V, Lane<T>::pack(v + i * Lane<T>::V));
    }
}

template <typename T, int VEC, int W, bool PACKED, bool ACT>
__global__ __launch_bounds__(64 * kWaves) void k_conv_act8(ConvAct8Args a) {
    constexpr int H = W - 1, N = H + kBatch;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // as in conv1d_bwd.hip: one stretch of the work for each XCD
    const int per = (int)((gridDim.x + 7) / 8);
    const int work = (int)(blockIdx.x % 8) * per + (int)(blockIdx.x / 8);
    if (work >= a.wgs) return;
    const int slab = work % a.slabs;
    const int rest = work / a.slabs;
    const int tile = rest % a.tiles, unit = rest / a.tiles;
    const bool rev = unit % a.ndir != 0;
    const int b = unit / a.ndir;
    const ConvAct8Dir d = rev ? a.dir[1] : a.dir[0];
    const int L = a.L, ch = a.ch, nblk = (ch + 31) / 32;
    const int p0 = (tile * kWaves + wave) * a.run;
    const int p1 = min(p0 + a.run, L);
    if (p0 >= L) return;
    // lanes past the last channel vector repeat it, with the same results
    const int c0 = min(slab * 64 + lane, a.nvec - 1) * VEC;

    float w[VEC][W], bias[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
#pragma unroll
        for (int k = 0; k < W; ++k) w[j][k] = d.weight[(size_t)(c0 + j) * W + k];
        bias[j] = d.bias ? d.bias[c0 + j] : 0.f;
    }
    // output array of the lane: x, B or C
    T *o;
    long long os;
    if (c0 < a.hp) {
        o = (T *)d.x + c0; os = a.hp;
    } else if (c0 < a.hp + a.gn) {
        o = (T *)d.B + (c0 - a.hp); os = a.gn;
    } else {
        o = (T *)d.C + (c0 - a.hp - a.gn); os = a.gn;
    }
    const size_t row0 = (size_t)b * L;
    auto token = [&](int p) { return rev ? L - 1 - p : p; };
    // walks with the positions: a product a row and lane would cost more
    o += (long long)(row0 + token(p0)) * os;
    if (rev) os = -os;

    float win[8][VEC];   // a ring where batches come in pairs
    Codes<VEC> next[kBatch];
    // so do the rows to load next
    const long long qs = rev ? -ch : ch, ss = rev ? -nblk : nblk;
    const int8_t *q = d.q + (long long)(row0 + token(p0)) * ch + c0;
    const uint8_t *sc = d.scale + (long long)(row0 + token(p0)) * nblk + c0 / 32;
    auto fetch = [&](int p) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            next[i].load(q, sc);
            // past the end the last row again, which is not used
            const bool more = p + i + 1 < L;
            q += more ? qs : 0;
            sc += more ? ss : 0;
        }
    };
    // where the window of the batch from p has sequence starts
    StartBits starts;
    if constexpr (PACKED) starts = StartBits(a.packed, p0 - H, L, rev);
    auto window = [&](int p) -> uint32_t { return PACKED ? starts.from(p - p0, N) : 0u; };
#pragma unroll
    for (int i = 0; i < H; ++i) {
        const int p = p0 - H + i;
        Codes<VEC> v;
        const size_t t = row0 + token(max(p, 0));
        v.load(d.q + t * ch + c0, d.scale + t * nblk + c0 / 32);
        v.values(win[i]);
#pragma unroll
        for (int j = 0; j < VEC; ++j)
            if (p < 0) win[i][j] = 0.f;
    }
    // The batch from p, its window in the ring from slot AT on. EDGE: the run
    // ends in this batch or the next, or sequences meet in its window; elsewhere
    // nothing is asked.
    auto batch = [&](int p, auto edge, auto slot, uint32_t first) {
        constexpr bool EDGE = decltype(edge)::value;
        constexpr int AT = decltype(slot)::value;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) next[i].values(win[(AT + H + i) & 7]);
        if (!EDGE || p + kBatch < p1) fetch(p + kBatch);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            float v[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                float u = bias[j];
#pragma unroll
                for (int k = 0; k < W; ++k) {
                    // no start among window positions i + k + 1 .. i + H
                    const bool same = !PACKED || !EDGE || !(first >> (i + k + 1) & ((1u << (H - k)) - 1));
                    u = fmaf(w[j][k], same ? win[(AT + i + k) & 7][j] : 0.f, u);
                }
                v[j] = ACT ? u * __builtin_amdgcn_rcpf(1.0f + __expf(-u)) : u;
            }
            if (!EDGE || p + i < p1) store_out<T, VEC>(o, v);
            o += os;
        }
    };
    using Even = std::integral_constant<int, 0>;
    using Odd = std::integral_constant<int, kBatch>;
    fetch(p0);
    int p = p0;
    auto back = [&] {   // the last H inputs to the window's start
#pragma unroll
        for (int i = 0; i < H; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) win[i][j] = win[kBatch + i][j];
        p += kBatch;
    };
    do {
        batch(p, std::true_type(), Even(), window(p));
        back();
        __builtin_amdgcn_s_waitcnt(0x0f70);   // vmcnt(0): as in conv1d_bwd.hip
        if constexpr (PACKED) {
            for (; p + 2 * kBatch <= p1 && window(p) == 0;) {
                batch(p, std::false_type(), Even(), 0u);
                back();
            }
        } else {
            // two batches go once round the ring, and nothing is moved (with
            // sequences as well it takes registers that cost a wave: 50 -> 53 us)
            for (; p + 3 * kBatch <= p1; p += 2 * kBatch) {
                batch(p, std::false_type(), Even(), 0u);
                batch(p + kBatch, std::false_type(), Odd(), 0u);
            }
        }
    } while (p < p1);
}

template <typename T, int VEC, int W>
hipError_t launch_w(const ConvAct8Args &a, hipStream_t s) {
    const dim3 grid((unsigned)((a.wgs + 7) / 8 * 8));
#define GO(PACKED, ACT) \
    BM_LAUNCH("conv1d_act8", (k_conv_act8<T, VEC, W, PACKED, ACT>), grid, dim3(64 * kWaves), 0, s, a)
    const bool packed = a.packed.seq || a.packed.count;
    if (a.act) {
        if (packed) GO(true, true);
        else GO(false, true);
    } else {
        if (packed) GO(true, false);
        else GO(false, false);
    }
#undef GO
    return hipGetLastError();
}
template <typename T, int VEC>
hipError_t launch_v(const ConvAct8Args &a, hipStream_t s) {
    switch (a.W) {
        case 2: return launch_w<T, VEC, 2>(a, s);
        case 3: return launch_w<T, VEC, 3>(a, s);
        case 4: return launch_w<T, VEC, 4>(a, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_conv_act8(ConvAct8Args a, bool bf16, hipStream_t s) {
    if (a.L == 0) return hipSuccess;
    const bool vec = conv_vectorized(bf16, a.hp, a.gn);   // else rows are not 4-byte aligned
    a.nvec = a.ch / (vec ? 4 : 1);
    a.slabs = (a.nvec + 63) / 64;
    // 32 positions a run, fewer where that leaves the chip short of waves
    // (2 x 333 tokens of 112 channels: 8 a run 5 us, 32 8; 1024 of 1024: 8 and 10;
    // where there are waves, shorter runs gain nothing)
    a.run = 32;
    while (a.run > 8 && (long long)((a.L + a.run - 1) / a.run) * a.slabs * a.batch * a.ndir < 2048) a.run /= 2;
    a.tiles = (a.L + a.run * kWaves - 1) / (a.run * kWaves);
    a.wgs = a.slabs * a.tiles * a.batch * a.ndir;
    if (bf16) return vec ? launch_v<uint16_t, 4>(a, s) : launch_v<uint16_t, 1>(a, s);
    return vec ? launch_v<float, 4>(a, s) : launch_v<float, 1>(a, s);
}

}  // namespace bm
