// Product of 8-bit rows (rms_norm.hip, rows8_pack) on the integer matrix cores:
//   out[r][n] = xs[r] ws[n] sum_c x[r][c] w[n][c] + bias[n]
// The sums are whole numbers in int32 (exact: |sum| <= 2^14 cin < 2^31), so no
// order of the products shows in the result; they are converted to fp32 once
// and scaled there.
//
// k_linear8: LDS tiles of 128 bytes of K, two buffers, v_mfma_i32_16x16x64_i8
// (lane l: row l % 16, bytes 16 (l / 16) .. of K for both operands). w is the
// first operand, so that a lane's four results lie in one row of out. Rows are
// copied to LDS without passing through registers (global_load_lds, a wave's 64
// lanes to consecutive 16-byte places: eight rows of 128 bytes); a row's chunk
// c is kept at place c ^ (row % 8), which spreads the 16 rows that a fragment
// read touches over the banks: the copy's lanes read their global chunks in
// that order. A K that ends inside a step reads zeros there. Rows whose length
// is no multiple of 16 go through registers (DIRECT = false).
//
// k_linear8_few: up to 64 rows, where the weights' bytes are the work. A
// workgroup takes 16 output channels; its eight waves split K and read both
// operands from memory straight into the fragments, and their sums meet in LDS.
#include "common.hpp"
#include "internal.hpp"
#include "mfma.hpp"

namespace bm {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t b16_a1 __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t h4_a2 __attribute__((ext_vector_type(2), aligned(2)));
typedef float f4_a4 __attribute__((ext_vector_type(4), aligned(4)));

__device__ const uint32_t kZeros[4] = {0u, 0u, 0u, 0u};

__device__ __forceinline__ i32x4 mfma_i8(u32x4 a, u32x4 b, i32x4 c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

// four results of one row, channels n .. n + 3
__device__ __forceinline__ void store4(uint16_t *p, const float *v) {
    *(h4_a2 *)p = h4_a2{pack2bf(v[0], v[1]), pack2bf(v[2], v[3])};
}
__device__ __forceinline__ void store4(float *p, const float *v) { *(f4_a4 *)p = f4_a4{v[0], v[1], v[2], v[3]}; }
__device__ __forceinline__ void store1(uint16_t *p, float v) { *p = f2bf(v); }
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }

template <typename T>
__device__ __forceinline__ void put(const Linear8Args &a, long long r, float xs, int n, i32x4 acc) {
    T *out = (T *)a.out + r * a.cout + n;
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int c = min(n + j, a.cout - 1);
        v[j] = fmaf((float)acc[j], xs * a.ws[c], a.bias ? a.bias[c] : 0.f);
    }
    if (n + 3 < a.cout) {
        store4(out, v);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (n + j < a.cout) store1(out + j, v[j]);
    }
}

constexpr int KB = 128;   // bytes of K a step

// WN x WM waves of 16 TN output channels by 16 TM rows each
template <int WN, int WM, int TN, int TM, bool DIRECT, typename T>
__global__ __launch_bounds__(64 * WN * WM) void k_linear8(Linear8Args a, int ntiles, int mtiles) {
    constexpr int NT = 16 * TN * WN, MT = 16 * TM * WM;
    constexpr int kCopies = (NT + MT) / 8 / (WN * WM);   // eight rows each, a wave
    static_assert((NT / 8) % (WN * WM) == 0 && (MT / 8) % (WN * WM) == 0, "a copy is of one operand");
    __shared__ __attribute__((aligned(16))) uint8_t lds[2][(NT + MT) * KB];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, l16 = lane & 15;
    // workgroup ids go round the 8 XCDs: each takes a run of tiles, eight row
    // panels under one another before the next channel panel, so that the
    // tiles at work on an XCD share both operands in its L2
    const long long total = (long long)ntiles * mtiles, per = (total + 7) / 8;
    const long long tile = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if ((long long)(blockIdx.x >> 3) >= per || tile >= total) return;
    const int band = (int)(tile / (8LL * ntiles)), tall = min(8, mtiles - 8 * band);
    const long long in = tile - 8LL * band * ntiles;
    const int n0 = (int)(in / tall) * NT;
    const long long m0 = (8LL * band + in % tall) * MT;
    // this lane's chunk of a copied row, and its rows
    const int row8 = lane >> 3, chunk = 16 * ((lane & 7) ^ row8);
    const int8_t *src[kCopies];
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
        const int rg = (i * WN * WM + wave) * 8 + row8;
        if (i * WN * WM * 8 < NT) src[i] = a.w + (long long)min(n0 + rg, a.cout - 1) * a.cin;
        else src[i] = a.x + min(m0 + rg - NT, a.rows - 1) * a.cin;
    }
    u32x4 held[DIRECT ? 1 : kCopies];
    auto fetch = [&](int k0, int buf) {
        if constexpr (DIRECT) {
            const bool ends = k0 + KB > a.cin;
#pragma unroll
            for (int i = 0; i < kCopies; ++i) {
                const int8_t *p = src[i] + k0 + chunk;
                if (ends && k0 + chunk >= a.cin) p = (const int8_t *)kZeros;
                __builtin_amdgcn_global_load_lds(
                    (const __attribute__((address_space(1))) void *)p,
                    (__attribute__((address_space(3))) void *)(lds[buf] + (i * WN * WM + wave) * 1024), 16, 0, 0);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kCopies; ++i) {
                const int at = k0 + chunk, left = a.cin - at;
                if (left >= 16) {
                    held[i] = *(const b16_a1 *)(src[i] + at);
                } else {
                    u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (j < left) v[j >> 2] |= (uint32_t)(uint8_t)src[i][at + j] << (8 * (j & 3));
                    held[i] = v;
                }
            }
        }
    };
    auto settle = [&](int buf) {
        if constexpr (DIRECT) {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        } else {
#pragma unroll
            for (int i = 0; i < kCopies; ++i)
                *(u32x4 *)(lds[buf] + (i * WN * WM + wave) * 1024 + 16 * lane) = held[i];
        }
        __syncthreads();
    };
    const int wn = (wave / WM) * 16 * TN, wm = (wave % WM) * 16 * TM;
    i32x4 acc[TN][TM];
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    fetch(0, 0);
    settle(0);
    const int steps = (a.cin + KB - 1) / KB;
    for (int s = 0; s < steps; ++s) {
        const int cur = s & 1;
        if (s + 1 < steps) fetch((s + 1) * KB, cur ^ 1);
        const uint8_t *wl = lds[cur], *xl = lds[cur] + NT * KB;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int place = 16 * ((4 * h + g) ^ (l16 & 7));
            u32x4 av[TN], bv[TM];
#pragma unroll
            for (int i = 0; i < TN; ++i) av[i] = *(const u32x4 *)(wl + (wn + 16 * i + l16) * KB + place);
#pragma unroll
            for (int j = 0; j < TM; ++j) bv[j] = *(const u32x4 *)(xl + (wm + 16 * j + l16) * KB + place);
#pragma unroll
            for (int i = 0; i < TN; ++i)
#pragma unroll
                for (int j = 0; j < TM; ++j) acc[i][j] = mfma_i8(av[i], bv[j], acc[i][j]);
        }
        // the other buffer is complete, and this one read, before either changes
        settle(cur ^ 1);
    }
#pragma unroll
    for (int j = 0; j < TM; ++j) {
        const long long r = m0 + wm + 16 * j + l16;
        if (r >= a.rows) continue;
        const float xs = a.xs[r];
#pragma unroll
        for (int i = 0; i < TN; ++i) {
            const int n = n0 + wn + 16 * i + 4 * g;
            if (n < a.cout) put<T>(a, r, xs, n, acc[i][j]);
        }
    }
}

constexpr int kFewWaves = 8;

// up to 16 TM rows, cin a multiple of 16
template <int TM, typename T>
__global__ __launch_bounds__(64 * kFewWaves) void k_linear8_few(Linear8Args a) {
    __shared__ i32x4 sums[kFewWaves][TM][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, l16 = lane & 15;
    const int n0 = 16 * blockIdx.x;
    const int8_t *wp = a.w + (long long)min(n0 + l16, a.cout - 1) * a.cin;
    const int8_t *xp[TM];
#pragma unroll
    for (int j = 0; j < TM; ++j) xp[j] = a.x + min((long long)(16 * j + l16), a.rows - 1) * a.cin;
    i32x4 acc[TM];
#pragma unroll
    for (int j = 0; j < TM; ++j) acc[j] = i32x4{0, 0, 0, 0};
    // four steps' loads at a time; one past the row's end multiplies zeros
    for (int kb = 64 * wave; kb < a.cin; kb += 4 * 64 * kFewWaves) {
        u32x4 wv[4], xv[4][TM];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int k = kb + 64 * kFewWaves * u + 16 * g;
            const bool in = k < a.cin;
            const int at = in ? k : 0;
            wv[u] = *(const u32x4 *)(wp + at);
            if (!in) wv[u] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
            for (int j = 0; j < TM; ++j) xv[u][j] = *(const u32x4 *)(xp[j] + at);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int j = 0; j < TM; ++j) acc[j] = mfma_i8(wv[u], xv[u][j], acc[j]);
    }
#pragma unroll
    for (int j = 0; j < TM; ++j) sums[wave][j][lane] = acc[j];
    __syncthreads();
    for (int e = tid; e < 64 * TM; e += 64 * kFewWaves) {
        const int j = e >> 6;
        i32x4 s = sums[0][j][lane];
#pragma unroll
        for (int i = 1; i < kFewWaves; ++i) s += sums[i][j][lane];
        const long long r = 16 * j + l16;
        const int n = n0 + 4 * g;
        if (r < a.rows && n < a.cout) put<T>(a, r, a.xs[r], n, s);
    }
}

template <int WN, int WM, int TN, int TM, bool DIRECT, typename T>
hipError_t launch_tiles(const Linear8Args &a, hipStream_t s) {
    constexpr int NT = 16 * TN * WN, MT = 16 * TM * WM;
    const int nt = (a.cout + NT - 1) / NT, mt = (int)((a.rows + MT - 1) / MT);
    const long long wgs = ((long long)nt * mt + 7) / 8 * 8;
    if (wgs > (1LL << 24) - 8) return hipErrorInvalidValue;
    BM_LAUNCH("linear8", (k_linear8<WN, WM, TN, TM, DIRECT, T>), dim3((unsigned)wgs), dim3(64 * WN * WM), 0, s, a, nt,
              mt);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_t(const Linear8Args &a, hipStream_t s) {
    const bool direct = a.cin % 16 == 0 && (((uintptr_t)a.x | (uintptr_t)a.w) & 15u) == 0;
    if (a.rows <= 64 && direct) {
        const dim3 grid((unsigned)((a.cout + 15) / 16)), block(64 * kFewWaves);
        if (a.rows <= 16) BM_LAUNCH("linear8_few", (k_linear8_few<1, T>), grid, block, 0, s, a);
        else if (a.rows <= 32) BM_LAUNCH("linear8_few", (k_linear8_few<2, T>), grid, block, 0, s, a);
        else BM_LAUNCH("linear8_few", (k_linear8_few<4, T>), grid, block, 0, s, a);
        return hipGetLastError();
    }
    auto tiles = [&](int nt, int mt) { return ((a.cout + nt - 1) / nt) * ((a.rows + mt - 1) / mt); };
    if (!direct) return tiles(128, 128) >= 256 ? launch_tiles<2, 2, 4, 4, false, T>(a, s)
                                               : launch_tiles<2, 2, 2, 2, false, T>(a, s);
    if (tiles(256, 256) >= 256) return launch_tiles<2, 4, 8, 4, true, T>(a, s);
    if (tiles(128, 128) >= 256) return launch_tiles<2, 2, 4, 4, true, T>(a, s);
    return launch_tiles<2, 2, 2, 2, true, T>(a, s);
}

}  // namespace

hipError_t launch_linear8(const Linear8Args &a, bool bf16, hipStream_t s) {
    if (a.rows == 0) return hipSuccess;
    return bf16 ? launch_t<uint16_t>(a, s) : launch_t<float>(a, s);
}

}  // namespace bm
