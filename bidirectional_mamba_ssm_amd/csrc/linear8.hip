// Product of 8-bit rows (rms_norm.hip, rows8_pack) on the integer matrix cores:
//   out[r][n] = xs[r] ws[n] sum_c x[r][c] w[n][c] + bias[n]
// The sums are whole numbers in int32 (exact: |sum| <= 2^14 cin < 2^31), so no
// order of the products shows in the result; they are converted to fp32 once
// and scaled there, or in fp64 where the two scales' product leaves fp32's normal
// numbers.
//
// k_linear8: v_mfma_i32_16x16x64_i8 (lane l: row l % 16, bytes 16 (l / 16) .. of K
// for both operands), w the first operand, so that a lane's four results lie in
// one row of out. Tiles of 64 bytes of K go to LDS without passing through
// registers (global_load_lds: a wave's lanes to consecutive 16-byte places, 16
// rows of 64 bytes, which is a fragment of each of the 16-row tiles as it is
// read, without bank conflicts). Four buffers: while a step's products run, the
// next step's fragments are read, the one after is landing and a third is asked
// for, so a load has two steps' time and each step waits for one barrier
// alone. A K that ends inside a step reads zeros there.
//
// k_linear8_rows: rows whose length is no multiple of 16, or that start
// elsewhere, go through registers byte by byte where they end, in steps of 128
// bytes and two buffers; chunk c of a row is kept at place c ^ (row % 8).
//
// k_linear8_few: up to 64 rows, where the weights' bytes are the work. A
// workgroup takes 16 or 32 output channels; its eight waves split K and read both
// operands from memory straight into the fragments, and their sums meet in LDS.
//
// Measured: 8192 rows, 2048 -> 8512 163 to 177 us as the clock is, 1.6 to
// 1.75 POP/s (138 us at the 2.08 POP/s that a large product reaches here); with the
// copies through registers and two buffers 224. Bound by the matrix cores and the
// clock that they are given: 202 us after a second of it. 64 rows, 4096 -> 2048
// 11 us in a row of calls and 12.7 alone, bound by the latency of its loads. Rows of
// 2047 and 4095 bytes take 380 and 27 us in those sizes.
#include "common.hpp"
#include "internal.hpp"
#include "mfma.hpp"
#include "rows.hpp"

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
    *(h4_a2 *)p = h4_a2{bf_pair(v[0], v[1]), bf_pair(v[2], v[3])};
}
__device__ __forceinline__ void store4(float *p, const float *v) { *(f4_a4 *)p = f4_a4{v[0], v[1], v[2], v[3]}; }
__device__ __forceinline__ void store1(uint16_t *p, float v) { *p = (uint16_t)bf_pair(v, 0.f); }
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }

// Workgroup ids go round the 8 XCDs: each takes a run of tiles, eight row panels
// under one another before the next channel panel, so that the tiles at work on
// an XCD share both operands in its L2.
template <int NT, int MT>
__device__ __forceinline__ bool place(int ntiles, int mtiles, int &n0, long long &m0) {
    const long long total = (long long)ntiles * mtiles, per = (total + 7) / 8;
    const long long tile = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if ((long long)(blockIdx.x >> 3) >= per || tile >= total) return false;
    const int band = (int)(tile / (8LL * ntiles)), tall = min(8, mtiles - 8 * band);
    const long long in = tile - 8LL * band * ntiles;
    n0 = (int)(in / tall) * NT;
    m0 = (8LL * band + in % tall) * MT;
    return true;
}

// A wave's results: row `row` and every 16th from it, channels n .. n + 3 and every
// 16th. whole: none of the wave's lies outside.
template <int TN, int TM, typename T>
__device__ __forceinline__ void finish(const Linear8Args &a, long long row, int n, bool whole, i32x4 (&acc)[TN][TM]) {
    float xs[TM];
#pragma unroll
    for (int j = 0; j < TM; ++j) xs[j] = a.xs[min(row + 16 * j, a.rows - 1)];
#pragma unroll
    for (int i = 0; i < TN; ++i) {
        const int c = n + 16 * i;
        float ws[4], b[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int at = min(c + e, a.cout - 1);
            ws[e] = a.ws[at];
            b[e] = a.bias ? a.bias[at] : 0.f;
        }
        // A product of two scales that is no normal number (subnormal, overflowed, or
        // of a row of zeros) has lost what the whole result may still hold
        bool far = false;
#pragma unroll
        for (int j = 0; j < TM; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) far |= !__builtin_isnormal(xs[j] * ws[e]);
        far = __any(far);
#pragma unroll
        for (int j = 0; j < TM; ++j) {
            T *out = (T *)a.out + (row + 16 * j) * a.cout + c;
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = fmaf((float)acc[i][j][e], xs[j] * ws[e], b[e]);
            if (far) {   // of these results alone: the others' bits are what they are beside any
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (!__builtin_isnormal(xs[j] * ws[e])) v[e] = (float)((double)acc[i][j][e] * xs[j] * ws[e] + b[e]);
            }
            if (whole) {
                store4(out, v);
            } else if (row + 16 * j < a.rows) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (c + e < a.cout) store1(out + e, v[e]);
            }
        }
    }
}

constexpr int KS = 64;   // bytes of K a step

// WN x WM waves of 16 TN output channels by 16 TM rows each
template <int WN, int WM, int TN, int TM, typename T>
__global__ __launch_bounds__(64 * WN * WM) void k_linear8(Linear8Args a, int ntiles, int mtiles) {
    constexpr int NT = 16 * TN * WN, MT = 16 * TM * WM, kWaves = WN * WM, kBufs = 4;
    constexpr int kGroups = (NT + MT) / 16, kCopies = (kGroups + kWaves - 1) / kWaves;   // 16 rows each
    __shared__ __attribute__((aligned(16))) uint8_t lds[kBufs][(NT + MT) * KS];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, l16 = lane & 15;
    int n0;
    long long m0;
    if (!place<NT, MT>(ntiles, mtiles, n0, m0)) return;
    // this lane's 16 bytes of a copied row, and its rows; waves without a last copy
    // repeat one, so that all have as many loads under way
    const int chunk = 16 * (lane & 3);
    const int8_t *src[kCopies];
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
        const int r = min(i * kWaves + wave, kGroups - 1) * 16 + (lane >> 2);
        src[i] = (r < NT ? a.w + (long long)min(n0 + r, a.cout - 1) * a.cin : a.x + min(m0 + r - NT, a.rows - 1) * a.cin) + chunk;
    }
    const int steps = (a.cin + KS - 1) / KS;
    // whole: the step does not reach past the rows' end
    auto fetch = [&](int s, bool whole) {
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
            const int8_t *p = src[i] + s * KS;
            if (!whole && s * KS + chunk >= a.cin) p = (const int8_t *)kZeros;
            __builtin_amdgcn_global_load_lds(
                (const __attribute__((address_space(1))) void *)p,
                (__attribute__((address_space(3))) void *)(lds[s % kBufs] + min(i * kWaves + wave, kGroups - 1) * 1024), 16,
                0, 0);
        }
    };
    const int wn = (wave / WM) * 16 * TN, wm = (wave % WM) * 16 * TM;
    u32x4 av[2][TN], bv[2][TM];
    auto read = [&](int s, u32x4 *av, u32x4 *bv) {
        const uint8_t *p = lds[s % kBufs] + l16 * KS + 16 * g;
#pragma unroll
        for (int i = 0; i < TN; ++i) av[i] = *(const u32x4 *)(p + (wn + 16 * i) * KS);
#pragma unroll
        for (int j = 0; j < TM; ++j) bv[j] = *(const u32x4 *)(p + (NT + wm + 16 * j) * KS);
    };
    i32x4 acc[TN][TM];
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    // a barrier that no access of memory moves across (and that waits for none)
    auto meet = [&]() {
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    auto products = [&](int cur) {
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int j = 0; j < TM; ++j) acc[i][j] = mfma_i8(av[cur][i], bv[cur][j], acc[i][j]);
    };
    // step s: its fragments are in registers, s + 1 landed or landing, s + 2 under
    // way; after the barrier everybody's part of s + 1 is there, and nobody reads
    // s - 1 any more
    auto inner = [&](int s, int cur) {
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kCopies) : "memory");
        meet();
        fetch(s + 3, true);
        read(s + 1, av[cur ^ 1], bv[cur ^ 1]);
        products(cur);
    };
    auto outer = [&](int s, int cur) {
        if (s + 1 < steps) {
            if (s + 2 < steps) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kCopies) : "memory");
            else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            meet();
            if (s + 3 < steps) fetch(s + 3, false);
            read(s + 1, av[cur ^ 1], bv[cur ^ 1]);
        }
        products(cur);
    };
    fetch(0, false);
    if (steps > 1) fetch(1, false);
    if (steps > 2) fetch(2, false);
    if (steps > 2) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * kCopies) : "memory");
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    meet();
    read(0, av[0], bv[0]);
    int s = 0;
    for (; s + 5 < steps; s += 2) {
        inner(s, 0);
        inner(s + 1, 1);
    }
    for (; s < steps; s += 2) {
        outer(s, 0);
        if (s + 1 < steps) outer(s + 1, 1);
    }
    if (n0 + NT <= a.cout && m0 + MT <= a.rows) finish<TN, TM, T>(a, m0 + wm + l16, n0 + wn + 4 * g, true, acc);
    else finish<TN, TM, T>(a, m0 + wm + l16, n0 + wn + 4 * g, false, acc);
}

constexpr int KB = 128;   // bytes of K a step

// WN x WM waves of 16 TN output channels by 16 TM rows each
template <int WN, int WM, int TN, int TM, typename T>
__global__ __launch_bounds__(64 * WN * WM) void k_linear8_rows(Linear8Args a, int ntiles, int mtiles) {
    constexpr int NT = 16 * TN * WN, MT = 16 * TM * WM;
    constexpr int kCopies = (NT + MT) / 8 / (WN * WM);   // eight rows each, a wave
    static_assert((NT / 8) % (WN * WM) == 0 && (MT / 8) % (WN * WM) == 0, "a copy is of one operand");
    __shared__ __attribute__((aligned(16))) uint8_t lds[2][(NT + MT) * KB];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, l16 = lane & 15;
    int n0;
    long long m0;
    if (!place<NT, MT>(ntiles, mtiles, n0, m0)) return;
    // this lane's chunk of a copied row, and its rows
    const int row8 = lane >> 3, chunk = 16 * ((lane & 7) ^ row8);
    const int8_t *src[kCopies];
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
        const int rg = (i * WN * WM + wave) * 8 + row8;
        if (i * WN * WM * 8 < NT) src[i] = a.w + (long long)min(n0 + rg, a.cout - 1) * a.cin;
        else src[i] = a.x + min(m0 + rg - NT, a.rows - 1) * a.cin;
    }
    u32x4 held[kCopies];
    auto fetch = [&](int k0) {
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
    };
    auto settle = [&](int buf) {
#pragma unroll
        for (int i = 0; i < kCopies; ++i)
            *(u32x4 *)(lds[buf] + (i * WN * WM + wave) * 1024 + 16 * lane) = held[i];
        __syncthreads();
    };
    const int wn = (wave / WM) * 16 * TN, wm = (wave % WM) * 16 * TM;
    i32x4 acc[TN][TM];
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    fetch(0);
    settle(0);
    const int steps = (a.cin + KB - 1) / KB;
    for (int s = 0; s < steps; ++s) {
        const int cur = s & 1;
        if (s + 1 < steps) fetch((s + 1) * KB);
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
    if (n0 + NT <= a.cout && m0 + MT <= a.rows) finish<TN, TM, T>(a, m0 + wm + l16, n0 + wn + 4 * g, true, acc);
    else finish<TN, TM, T>(a, m0 + wm + l16, n0 + wn + 4 * g, false, acc);
}

constexpr int kFewWaves = 8;

// up to 16 TM rows, 16 TN channels, cin a multiple of 16
template <int TN, int TM, typename T>
__global__ __launch_bounds__(64 * kFewWaves) void k_linear8_few(Linear8Args a) {
    __shared__ i32x4 sums[kFewWaves][TN * TM][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, l16 = lane & 15;
    const int n0 = 16 * TN * blockIdx.x;
    const int8_t *wp[TN], *xp[TM];
#pragma unroll
    for (int i = 0; i < TN; ++i) wp[i] = a.w + (long long)min(n0 + 16 * i + l16, a.cout - 1) * a.cin;
#pragma unroll
    for (int j = 0; j < TM; ++j) xp[j] = a.x + min((long long)(16 * j + l16), a.rows - 1) * a.cin;
    i32x4 acc[TN][TM];
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    // two steps' loads at a time; one past the row's end multiplies zeros
    constexpr int U = 2;
    for (int kb = 64 * wave; kb < a.cin; kb += U * 64 * kFewWaves) {
        u32x4 wv[U][TN], xv[U][TM];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = kb + 64 * kFewWaves * u + 16 * g;
            const bool in = k < a.cin;
            const int at = in ? k : 0;
#pragma unroll
            for (int i = 0; i < TN; ++i) {
                wv[u][i] = *(const u32x4 *)(wp[i] + at);
                if (!in) wv[u][i] = u32x4{0u, 0u, 0u, 0u};
            }
#pragma unroll
            for (int j = 0; j < TM; ++j) xv[u][j] = *(const u32x4 *)(xp[j] + at);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < TN; ++i)
#pragma unroll
                for (int j = 0; j < TM; ++j) acc[i][j] = mfma_i8(wv[u][i], xv[u][j], acc[i][j]);
    }
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) sums[wave][i * TM + j][lane] = acc[i][j];
    __syncthreads();
    for (int e = tid; e < 64 * TN * TM; e += 64 * kFewWaves) {
        const int i = (e >> 6) / TM, j = (e >> 6) % TM, n = n0 + 16 * i;
        i32x4 s = sums[0][e >> 6][lane];
#pragma unroll
        for (int w = 1; w < kFewWaves; ++w) s += sums[w][e >> 6][lane];
        i32x4 one[1][1] = {{s}};
        if (n < a.cout) finish<1, 1, T>(a, 16 * j + l16, n + 4 * g, n + 16 <= a.cout && 16 * j + 16 <= a.rows, one);
    }
}

template <int WN, int WM, int TN, int TM, bool DIRECT, typename T>
hipError_t launch_tiles(const Linear8Args &a, hipStream_t s) {
    constexpr int NT = 16 * TN * WN, MT = 16 * TM * WM;
    const int nt = (a.cout + NT - 1) / NT, mt = (int)((a.rows + MT - 1) / MT);
    const long long wgs = ((long long)nt * mt + 7) / 8 * 8;
    if (wgs > (1LL << 24) - 8) return hipErrorInvalidValue;
    const dim3 grid((unsigned)wgs), block(64 * WN * WM);
    if constexpr (DIRECT) BM_LAUNCH("linear8", (k_linear8<WN, WM, TN, TM, T>), grid, block, 0, s, a, nt, mt);
    else BM_LAUNCH("linear8_rows", (k_linear8_rows<WN, WM, TN, TM, T>), grid, block, 0, s, a, nt, mt);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_t(const Linear8Args &a, hipStream_t s) {
    const bool direct = a.cin % 16 == 0 && (((uintptr_t)a.x | (uintptr_t)a.w) & 15u) == 0;
    if (direct && (a.rows <= 16 || (a.rows <= 64 && a.cout <= 8192))) {
        // Up to 64 rows, while the tiles below are too few for the CUs (64 rows,
        // 2048 -> 2048: 9.2 us here, 10.2 in 64 x 64 tiles; 24 rows, 8192 -> 8192: 23.5
        // and 30.6; 8 rows, 2048 -> 32 000: 16.4 and 14.7; but 64 rows, 2048 -> 8512: 12.7
        // and 10.6, 24 rows, 2048 -> 32 000: 24.2 and 16.6).
        // Every workgroup reads all of x: with more than 32 rows 16 channels a
        // workgroup read more of it than of w. Twice as many where that still leaves
        // work for every CU (64 rows, 8192 -> 8192: 512 workgroups 40.3 us, 256 27.4;
        // 4096 -> 2048: 128 12.9, 64 14.8; one row, 8192 -> 8192: 512 15.0, 256 20.5).
        const int tn = a.rows <= 32 || a.cout <= 4096 ? 1 : 2;
        const dim3 grid((unsigned)((a.cout + 16 * tn - 1) / (16 * tn))), block(64 * kFewWaves);
        if (a.rows <= 16) BM_LAUNCH("linear8_few", (k_linear8_few<1, 1, T>), grid, block, 0, s, a);
        else if (a.rows <= 32) BM_LAUNCH("linear8_few", (k_linear8_few<1, 2, T>), grid, block, 0, s, a);
        else if (tn == 1) BM_LAUNCH("linear8_few", (k_linear8_few<1, 4, T>), grid, block, 0, s, a);
        else BM_LAUNCH("linear8_few", (k_linear8_few<2, 4, T>), grid, block, 0, s, a);
        return hipGetLastError();
    }
    auto tiles = [&](int nt, int mt) { return ((a.cout + nt - 1) / nt) * ((a.rows + mt - 1) / mt); };
    if (!direct) return tiles(128, 128) >= 256 ? launch_tiles<2, 2, 4, 4, false, T>(a, s)
                                               : launch_tiles<2, 2, 2, 2, false, T>(a, s);
    // The widest tiles that leave most CUs work (2048 -> 4096: 3200 rows, 208 tiles of
    // 256 45 us, of 128 52; 2048 rows 36 and 31; 2048 -> 2048: 2048 rows, 256 tiles of
    // 128 21 us, of 64 24; 1024 rows 20 and 14).
    if (tiles(256, 256) >= 200) {
        // one workgroup a CU: the width whose rounds of 256 tiles take the least time
        // (8192 rows, 2048 -> 8512, one after the other: 256 channels wide 208 us, 224
        // 202)
        int best = 256;
        long long least = 0;
        for (int w = 256; w >= 160; w -= 32) {
            const long long t = (tiles(w, 256) + 255) / 256 * (w + 16);
            if (!least || t < least) {
                least = t;
                best = w;
            }
        }
        switch (best) {
            case 160: return launch_tiles<2, 4, 5, 4, true, T>(a, s);
            case 192: return launch_tiles<2, 4, 6, 4, true, T>(a, s);
            case 224: return launch_tiles<2, 4, 7, 4, true, T>(a, s);
        }
        return launch_tiles<2, 4, 8, 4, true, T>(a, s);
    }
    if (tiles(128, 128) >= 256) return launch_tiles<2, 2, 4, 4, true, T>(a, s);
    return launch_tiles<2, 2, 2, 2, true, T>(a, s);
}

}  // namespace

hipError_t launch_linear8(const Linear8Args &a, bool bf16, hipStream_t s) {
    if (a.rows == 0) return hipSuccess;
    return bf16 ? launch_t<uint16_t>(a, s) : launch_t<float>(a, s);
}

}  // namespace bm
