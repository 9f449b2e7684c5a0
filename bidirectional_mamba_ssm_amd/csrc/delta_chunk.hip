// The gated delta rule by chunks of 64 tokens on the matrix cores. With G_i the
// sum of g up to token i of the chunk, Gam_ij = e^{G_i - G_j}, S the state that
// enters it and M_ij = Gam_ij beta_j k_i . k_j (j < i):
//   E = (I + M)^-1 (V - e^G K S)                 errors of all 64 tokens
//   Y = scale e^G Q S + A E,                     A_ij = scale Gam_ij beta_j q_i . k_j (j <= i)
//   S <- e^{G_C} S + K^T (e^{G_C - G} beta E)
// and the gradient's walk back, with D the gradient of the state that leaves
// the chunk, do = dy, L_ij = Gam_ij beta_i k_i . k_j (j < i), B_ij = scale Gam_ij q_i . k_j:
//   Z = (I + L)^-T (e^{G_C - G} K D + B^T do)    gradients of beta e
//   D <- e^{G_C} D + Q^T (scale e^G do) - K^T (e^G beta Z)
// (both inverses, since a beta may be 0 and (I + L)^-1 diag(beta) = diag(beta) (I + M)^-1).
//
// k_delta_prep, a chunk and head to a wave, makes what does not wait for the
// state: the triangles, inverted in fp32, as operand images. Everything but the
// diagonal 16 x 16 blocks stays in registers: a result's lanes (rows 4 g + r of a
// tile, column l % 16) are the transpose's first operand, or the second one's, as
// they come, for v_mfma_f32_16x16x4_f32 taken with k = 4 g + r in its r-th step. The
// diagonal blocks are inverted by substitution, a column a lane, all four at
// once. A tile's decays are products of a row's and a column's factor (and the
// tiles' between), both at most 1 where g <= 0; the diagonal tiles' are taken
// one by one.
//
// Bound by its loads' and products' latency: 39 us for the 4096 chunks and heads of
// the layer below, 50 with the gradient's third triangle.
//
// k_delta_walk takes a head's chunks in order. A wave owns 16 columns of the
// state for all N rows; columns never meet. The matrix cores' result order serves
// as the next product's second operand as it is, if the first one's k order
// follows it: so S, V, E and Y never leave the wave's registers, and no product
// waits for another wave. K and Q come to LDS row by row (read as rows for
// K S and Q S, transposed by ds_read_b64_tr_b16 for K^T E), the triangles as
// operand images; the next chunk's loads are under way meanwhile, in
// registers. A head's waves share both. A workgroup that has the CU (of eight
// waves, or in fp32) takes two buffers where they fit into LDS, filled in the
// middle of a chunk: one barrier a chunk. The others take one: bf16 walks of 64
// columns, two of whose workgroups share a CU and hide each other's waits, and
// fp32 ones forward and back with d_state 64 and 128.
//
// Measured, 8 rows of 1024 tokens, 32 heads of 128 x 128, bf16, in a row of calls:
// forward 117 us, keeping the states 109, back 177 (with one buffer 125, 116 and
// 183; two workgroups of 64 columns a CU 147, 125 and 201); in fp32 211, 161 and
// 258. A chunk takes a wave 3500 cycles of products and some 12 500 in all, since
// each of its products waits for the one before; with two waves a SIMD the sixteen
// chunks are 7 us each.
#include <algorithm>

#include "delta_split.hpp"
#include "internal.hpp"

namespace bm {
namespace {

constexpr int C = kDeltaChunk;
enum { FWD, KEEP, BACK };
// triangles of a chunk and head: FWD (I + M)^-1, A; for the gradient (I + M)^-1, (I + L)^-T, B^T
constexpr int triangles(bool grad) { return grad ? 3 : 2; }

// Workgroup ids go round the 8 XCDs: each takes a run of the work, so that what
// neighbours share (a group's K and Q, a head's triangles) meets in one L2.
__device__ __forceinline__ long long xcd_order(long long n) {
    const long long per = (n + 7) / 8, w = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    return (long long)(blockIdx.x >> 3) < per ? w : n;
}
inline long long xcd_grid(long long n) { return (n + 7) / 8 * 8; }

__device__ __forceinline__ f32x4 mfma4(float a, float b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

struct PrepDir {
    DeltaArgs a;
    uint8_t *tri;      // [slot][H]
    float *gates;      // [slot][H][kGateFloats]
};
struct PrepArgs {
    PrepDir dir[2];
};

constexpr int kPrepWaves = 4;
constexpr int kDiag = 16 * 20;   // a diagonal block in LDS: rows of 20 words

// one wave's exchange through LDS
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// the inverse of I + m for four strictly lower 16 x 16 blocks, a column a lane
__device__ __forceinline__ void invert_diagonal(const float *m, float *x, int g, int l16) {
    const float *from = m + g * kDiag;
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float s[2] = {i == l16 ? 1.f : 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < i; k += 4) {
            const f32x4 row = *(const f32x4 *)(from + i * 20 + k);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (k + e < i) s[e & 1] = fmaf(-row[e], v[k + e], s[e & 1]);
        }
        v[i] = s[0] + s[1];
    }
    float *to = x + g * kDiag + l16;
#pragma unroll
    for (int i = 0; i < 16; ++i) to[i * 20] = v[i];
}

template <typename T, int N, bool GRAD>
__global__ __launch_bounds__(64 * kPrepWaves, 2) void k_delta_prep(PrepArgs args, long long items) {
    constexpr int IN = Terms<T>::IN, KS = (N + 31) / 32, NM = GRAD ? 2 : 1;
    struct Wave {
        // diagonal blocks of M, (L,) and of M's inverse; L's takes M's place
        float d[NM + 1][4 * kDiag];
        double sums[C];
        float rows[C], cols[C], beta[C];
    };
    __shared__ __attribute__((aligned(16))) Wave waves[kPrepWaves];
    const PrepDir &pd = args.dir[blockIdx.y];
    const DeltaArgs &a = pd.a;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 4, l16 = lane & 15;
    Wave &w = waves[wave];
    const long long item = xcd_order((items + kPrepWaves - 1) / kPrepWaves) * kPrepWaves + wave;
    if (item >= items) return;
    const int h = (int)(item % a.H), grp = h / (a.H / a.G);
    const long long slot = item / a.H;
    int chunk;
    const DeltaUnit at = delta_slot(a, slot, chunk);
    const int first = chunk * C, live = min(C, at.len - first);
    if (live <= 0) return;
    const uint32_t row = (uint32_t)(a.G * N * sizeof(T)), off = (uint32_t)(grp * N * sizeof(T));
    const ChunkRows kr(a.k, at, a.reverse, first, live, row, off, N * sizeof(T));
    const ChunkRows qr(a.q, at, a.reverse, first, live, row, off, N * sizeof(T));
    auto operand = [&](const ChunkRows &r, int tile, int s) {
        constexpr int V = 16 / sizeof(T);
        const uint32_t from = r.offset(16 * tile + l16);
        const int n = 32 * s + 8 * g;
        const uint32_t col = n < N ? (uint32_t)(n * sizeof(T)) : kFar;
        if constexpr (IN == 1)
            return Operand<1>{buf16(r.rsrc, from + col)};
        else
            return split8<3>(__builtin_bit_cast(f32x4, buf16(r.rsrc, from + col)),
                             __builtin_bit_cast(f32x4, buf16(r.rsrc, from + col + 4 * V)));
    };
    const size_t gate = (size_t)delta_token(at, a.reverse, first + min(lane, live - 1)) * a.H + h;
    const float glog = lane < live ? a.g[gate] : 0.f, gbeta = lane < live ? a.beta[gate] : 0.f;
    // kk: rows i = 4 g + r, column j = l16 of tile (i, j); kt: its transpose; qk: FWD
    // rows j, column i, GRAD rows i, column j
    f32x4 kk[10], kt[GRAD ? 10 : 1], qk[10];
#pragma unroll
    for (int l = 0; l < 10; ++l) kk[l] = qk[l] = kt[GRAD ? l : 0] = zero4();
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        Operand<IN> k[4], q[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            k[t] = operand(kr, t, s);
            q[t] = operand(qr, t, s);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j <= i; ++j) {
                const int l = lower(i, j);
                kk[l] = mm(k[i], k[j], kk[l]);
                if (GRAD && i != j) kt[GRAD ? l : 0] = mm(k[j], k[i], kt[GRAD ? l : 0]);
                qk[l] = GRAD ? mm(q[i], k[j], qk[l]) : mm(k[j], q[i], qk[l]);
            }
    }
    {
        const double sum = decay_sums(glog, lane);
        const double before = __shfl(sum, max((lane & 48) - 1, 0)), end = __shfl(sum, lane | 15);
        w.sums[lane] = sum;
        w.rows[lane] = expf((float)(lane < 16 ? sum : sum - before));
        w.cols[lane] = expf((float)(end - sum));
        w.beta[lane] = gbeta;
        float *to = pd.gates + ((size_t)slot * a.H + h) * kGateFloats;
        ((double *)(to + kGates))[lane] = sum;
        to[lane] = expf((float)sum);
        to[C + lane] = expf((float)(__shfl(sum, 63) - sum));
        to[2 * C + lane] = gbeta;
    }
    wave_sync();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float ri = w.rows[16 * i + l16], bi = w.beta[16 * i + l16];
        const f32x4 r4 = *(const f32x4 *)&w.rows[16 * i + 4 * g], b4 = *(const f32x4 *)&w.beta[16 * i + 4 * g];
#pragma unroll
        for (int j = 0; j < i; ++j) {
            const int l = lower(i, j);
            // between the tiles: from column tile's end to row tile's start
            const float t = i - j > 1 ? expf((float)(w.sums[16 * i - 1] - w.sums[16 * j + 15])) : 1.f;
            const float cj = t * w.cols[16 * j + l16], bj = w.beta[16 * j + l16];
            const f32x4 c4 = t * *(const f32x4 *)&w.cols[16 * j + 4 * g], d4 = *(const f32x4 *)&w.beta[16 * j + 4 * g];
            kk[l] *= r4 * (cj * bj);                              // M
            if constexpr (GRAD) kt[l] *= c4 * (ri * bi);          // L^T
            qk[l] *= GRAD ? r4 * (cj * a.scale) : c4 * d4 * (ri * a.scale);
        }
        // diagonal tile: the rows' sums beside this lane's column's
        const int l = lower(i, i);
        const double own = w.sums[16 * i + l16];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int n = 4 * g + r;
            const double other = w.sums[16 * i + n];
            const float up = n >= l16 ? expf((float)(other - own)) : 0.f;   // rows i = n
            const float m = n > l16 ? up * kk[l][r] : 0.f;
            w.d[0][i * kDiag + n * 20 + l16] = m * bi;
            if constexpr (GRAD) {
                w.d[1][i * kDiag + n * 20 + l16] = m * b4[r];
                qk[l][r] *= a.scale * up;
            } else {
                const float dn = n <= l16 ? expf((float)(own - other)) : 0.f;   // rows j = n
                qk[l][r] *= a.scale * dn * b4[r];
            }
        }
    }
    uint8_t *tri = pd.tri + ((size_t)slot * a.H + h) * triangles(GRAD) * kTriangle + 16 * lane;
    auto put = [&](int which, const f32x4 *v) {
#pragma unroll
        for (int l = 0; l < kTiles; ++l) *(f32x4 *)(tri + which * kTriangle + l * 1024) = v[l];
    };
    put(GRAD ? 2 : 1, qk);
    wave_sync();
    invert_diagonal(w.d[0], w.d[NM], g, l16);
    wave_sync();
    if constexpr (GRAD) {
        invert_diagonal(w.d[1], w.d[0], g, l16);
        wave_sync();
    }
    // a diagonal block as a result of its own lanes (rows 4 g + r, column l16) and transposed
    auto plain = [&](int which, int i) {
        f32x4 v;
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = w.d[which][i * kDiag + (4 * g + r) * 20 + l16];
        return v;
    };
    auto turned = [&](int which, int i) { return *(const f32x4 *)&w.d[which][i * kDiag + l16 * 20 + 4 * g]; };
    {
        // X = (I + M)^-1 by its transpose: X^T_ji = -X^T_jj sum_{j < m <= i} M^T_jm X^T_mi
        f32x4 x[10];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[lower(i, i)] = turned(NM, i);
#pragma unroll
        for (int d = 1; d < 4; ++d) {
            f32x4 t[3], v[3];
#pragma unroll
            for (int j = 0; j < 4 - d; ++j) t[j] = v[j] = zero4();
#pragma unroll
            for (int m = 1; m <= d; ++m)
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int j = 0; j < 4 - d; ++j)
                        t[j] = mfma4(kk[lower(j + m, j)][r], x[lower(j + d, j + m)][r], t[j]);
            f32x4 own[3];
#pragma unroll
            for (int j = 0; j < 4 - d; ++j) own[j] = plain(NM, j);
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int j = 0; j < 4 - d; ++j) v[j] = mfma4(own[j][r], t[j][r], v[j]);
#pragma unroll
            for (int j = 0; j < 4 - d; ++j) x[lower(j + d, j)] = -v[j];
        }
        put(0, x);
    }
    if constexpr (GRAD) {
        // Y = (I + L)^-1: Y_ij = -Y_ii sum_{j <= m < i} L_im Y_mj
        f32x4 y[10];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[lower(i, i)] = plain(0, i);
#pragma unroll
        for (int d = 1; d < 4; ++d) {
            f32x4 t[3], v[3];
#pragma unroll
            for (int j = 0; j < 4 - d; ++j) t[j] = v[j] = zero4();
#pragma unroll
            for (int m = 0; m < d; ++m)
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int j = 0; j < 4 - d; ++j)
                        t[j] = mfma4(kt[lower(j + d, j + m)][r], y[lower(j + m, j)][r], t[j]);
            f32x4 own[3];
#pragma unroll
            for (int j = 0; j < 4 - d; ++j) own[j] = turned(0, j + d);
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int j = 0; j < 4 - d; ++j) v[j] = mfma4(own[j][r], t[j][r], v[j]);
#pragma unroll
            for (int j = 0; j < 4 - d; ++j) y[lower(j + d, j)] = -v[j];
        }
        put(1, y);
    }
}

typedef short v4i16_d __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4i16_d lds_v4i16_d;

struct WalkArgs {
    PrepDir dir[2];
    int ndir;          // FWD, one after the other: the forward output is added to the reverse one's
    int blocks;        // workgroups of a head
    bool apart;        // side by side, blockIdx.y the direction
};

// Where element (row, col) of K or Q is in LDS, col a multiple of 4: four
// columns and the four 16 beyond lie side by side, which is a lane's 16 bytes of a
// row operand; the 16-byte places of a row are permuted by its number, so that
// the 16 rows that a read touches lie in different banks. A row and the 16th
// after it are permuted alike. (64-bit reads of rows 72 words apart took 25
// cycles where these take 12.)
template <int NP>
__device__ __forceinline__ int row_place(int row, int col) {
    constexpr int kPlaces = NP / 8;
    const int place = col / 32 * 4 + col % 16 / 4;
    const int turn = row / (16 / kPlaces) % kPlaces;
    return row * NP * 2 + 16 * (place ^ turn) + col % 32 / 16 * 8;
}

// W waves: 64 columns, two workgroups a CU (bf16), or 128, one
template <typename T, int N, int MODE, int W>
__global__ __launch_bounds__(64 * W, sizeof(T) == 2 || W == 8 ? 2 : 1) void k_delta_walk(WalkArgs args) {
    using X = typename std::conditional<MODE == BACK, float, T>::type;   // the third input's type
    constexpr int IN = Terms<T>::IN, OWN = Terms<T>::OWN;
    constexpr bool GRAD = MODE != FWD;
    constexpr int NP = N < 32 ? 32 : N, KS = NP / 32, NT = N / 16;
    constexpr int kRows = C * NP * 2 * IN;              // bytes of K or Q in LDS
    constexpr bool kStaged = sizeof(X) == 2;            // the third input comes through LDS
    constexpr int kThreads = 64 * W;
    constexpr bool kQ = MODE != KEEP;                   // Q read, and a second image
    constexpr int kImages = kQ ? 2 : 1, kImg = kImage<OWN>;
    constexpr int kBuf = kRows * (kQ ? 2 : 1) + kImg * kImages + kGates * 4, kOwn = kStaged ? W * C * 32 : 0;
    // two buffers where one workgroup has the CU, and they fit
    constexpr bool kTwo = 2 * kBuf + kOwn <= 160 * 1024 && (sizeof(T) == 4 || W == 8);
    __shared__ __attribute__((aligned(16))) uint8_t lds[kBuf * (kTwo ? 2 : 1) + kOwn];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, l16 = lane & 15;
    const long long work = (long long)args.dir[0].a.units * args.dir[0].a.H * args.blocks, mine = xcd_order(work);
    if (mine >= work) return;
    const int block = (int)(mine % args.blocks), h = (int)(mine / args.blocks % args.dir[0].a.H);
    const int u = (int)(mine / args.blocks / args.dir[0].a.H);
    const int p0 = (block * W + wave) * 16;
    // Of the two waves of a SIMD one does its share of the copying before its first
    // products and the other after them (keeping the states 109 us at the layer's
    // shape, both after 113; forward it is 124 and 117 so, back 187 and 177)
    const bool early = kTwo && W == 8 && MODE == KEEP && wave >= W / 2;
    // the wave has columns, those of the walks' own arrays past the head's width among them
    const bool works = p0 < (GRAD ? padded(args.dir[0].a.P) : args.dir[0].a.P);
    // the halves of blocks that lie beyond the diagonal stay zeros
    for (int i = tid; i < kImages * 2 * OWN * 64; i += kThreads) {
        const int which = i / (2 * OWN * 64), e = i / 64 % (2 * OWN), term = e % OWN, second = e / OWN;
        const int half = MODE == BACK ? 2 * (second ? upper_block(3, 1) : upper_block(1, 0))
                                      : 2 * (second ? lower_block(2, 1) : lower_block(0, 0)) + 1;
#pragma unroll
        for (int b = 0; b < (kTwo ? 2 : 1); ++b)
            *(u32x2 *)(lds + b * kBuf + (kQ ? 2 : 1) * kRows + which * kImg + ((half >> 1) * OWN + term) * 1024 +
                       16 * lane + 8 * (half & 1)) = u32x2{0u, 0u};
    }
    const int d0 = args.apart ? blockIdx.y : 0, d1 = args.apart ? blockIdx.y : args.ndir - 1;
    for (int di = d1; di >= d0; --di) {
        const PrepDir &pd = args.dir[di];
        const DeltaArgs &a = pd.a;
        const int grp = h / (a.H / a.G), PP = padded(a.P);
        const DeltaUnit at = delta_unit(a, u);
        const int chunks = (at.len + C - 1) / C;
        // the lane's column, in the caller's arrays and in the walks' own
        const int p = p0 + l16;
        const bool own = p < a.P;
        const uint32_t pw = p < PP ? 4 * p : kFar;
        f32x4 S[NT];
        const size_t state = (((size_t)u * a.H + h) * a.P + p) * N + 4 * g;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            S[t] = zero4();
            if (a.init && own) S[t] = *(const f32x4 *)(a.init + state + 16 * t);
        }
        // chunks on their way: rows of K and Q, images, gates, the third input
        constexpr int V = 16 / sizeof(T), kAll = C * NP / V, kVecs = (kAll + kThreads - 1) / kThreads;
        constexpr int kVi = (kImages * kTiles + W - 1) / W;
        u32x4 nk[kVecs], nq[kQ ? kVecs : 1], ni[kVi], nv[2];
        float ngate = 0.f;
        X nx[4][4];
        const bool whole = a.P % 8 == 0;   // rows of V are 16-byte vectors
        auto order = [&](int i) { return MODE == BACK ? chunks - 1 - i : i; };
        // A lane's own numbers, as a stage of a chunk has them: the compiler would
        // keep what all stages make of them through the whole walk, which in these
        // forms is more than the registers hold (back 224 us, 177 made anew, in fp32 420
        // and 258, of 64 columns 277 and 136). What fits is kept: forward of 128 bf16
        // columns 117 us and 123 made anew, keeping the states 109 and 115. The other
        // forwards put 20 bytes a lane into scratch if kept, which costs them nothing:
        // of 64 bf16 columns 104 and 111, of 128 in fp32 207 and 211.
        constexpr bool kCrowded = N == 128 && (MODE == BACK || (MODE == FWD && (W == 4 || IN == 3)));
        auto fresh = [&](int v) {
            if constexpr (kCrowded) asm volatile("" : "+v"(v));
            return v;
        };
        auto fetch_rows = [&](int chunk) {
            const int tid = fresh(threadIdx.x);
            const int first = chunk * C, live = min(C, at.len - first);
            const uint32_t row = (uint32_t)(a.G * N * sizeof(T)), off = (uint32_t)(grp * N * sizeof(T));
            const ChunkRows kr(a.k, at, a.reverse, first, live, row, off, N * sizeof(T));
            const ChunkRows qr(a.q, at, a.reverse, first, live, row, off, N * sizeof(T));
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const int e = tid + kThreads * i, col = e % (NP / V) * V;
                const uint32_t o = kr.offset(e / (NP / V)) + (col < N && e < kAll ? (uint32_t)(col * sizeof(T)) : kFar);
                nk[i] = buf16(kr.rsrc, o);
                if (kQ) nq[i] = buf16(qr.rsrc, o);
            }
        };
        auto fetch = [&](int chunk) {
            const int tid = fresh(threadIdx.x);
            const int first = chunk * C, live = min(C, at.len - first);
            const size_t sh = (size_t)(at.slot + chunk) * a.H + h;
            const __amdgpu_buffer_rsrc_t ir = __builtin_amdgcn_make_buffer_rsrc(
                pd.tri + (sh * triangles(GRAD) + (MODE == BACK ? 1 : 0)) * kTriangle, 0, kImages * kTriangle, 0x00027000);
#pragma unroll
            for (int i = 0; i < kVi; ++i) ni[i] = buf16(ir, 16 * (tid + kThreads * i));
            if (tid < kGates) ngate = pd.gates[sh * kGateFloats + tid];
            if constexpr (kStaged) {
                const ChunkRows xr(a.v, at, a.reverse, first, live, (uint32_t)(a.H * a.P * sizeof(X)),
                                   (uint32_t)(h * a.P * sizeof(X)), a.P * sizeof(X));
                // eight of the wave's columns
                const int c = p0 + 8 * (tid & 1);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t from = xr.offset(((tid & 63) >> 1) + 32 * i);
                    if (whole) {
                        nv[i] = buf16(xr.rsrc, from + (c < a.P ? 2 * c : kFar));
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            nv[i][j] = (uint32_t)buf_value(xr.rsrc, from + (c + 2 * j < a.P ? 2 * (c + 2 * j) : kFar), X()) |
                                       (uint32_t)buf_value(xr.rsrc, from + (c + 2 * j + 1 < a.P ? 2 * (c + 2 * j + 1) : kFar), X())
                                           << 16;
                    }
                }
            }
        };
        auto fetch_values = [&](int chunk) {
            if constexpr (!kStaged) {
                const int first = chunk * C, live = min(C, at.len - first), g = (fresh(threadIdx.x) & 63) >> 4;
                const ChunkRows xr(a.v, at, a.reverse, first, live, (uint32_t)(a.H * a.P * sizeof(X)),
                                   (uint32_t)(h * a.P * sizeof(X)), a.P * sizeof(X));
                const uint32_t to = xr.offset(4 * g) + (own ? (uint32_t)(p * sizeof(X)) : kFar);
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) nx[t][r] = buf_value(xr.rsrc, to + (16 * t + r) * xr.step, X());
            }
        };
        auto stash = [&](uint8_t *buf) {
            const int tid = fresh(threadIdx.x), lane = tid & 63;
#pragma unroll
            for (int w = 0; w < (kQ ? 2 : 1); ++w)
#pragma unroll
                for (int i = 0; i < kVecs; ++i) {
                    const int e = tid + kThreads * i, row = e / (NP / V), col = e % (NP / V) * V;
                    if (kAll % kThreads && e >= kAll) break;
                    uint8_t *to = buf + w * kRows;
                    const u32x4 r = w ? nq[i] : nk[i];
                    if constexpr (IN == 1) {
                        *(u32x2 *)(to + row_place<NP>(row, col)) = u32x2{r[0], r[1]};
                        *(u32x2 *)(to + row_place<NP>(row, col + 4)) = u32x2{r[2], r[3]};
                    } else {
                        uint32_t lo[IN], hi[IN];
                        split2<IN>(__uint_as_float(r[0]), __uint_as_float(r[1]), lo);
                        split2<IN>(__uint_as_float(r[2]), __uint_as_float(r[3]), hi);
#pragma unroll
                        for (int t = 0; t < IN; ++t)
                            *(u32x2 *)(to + t * C * NP * 2 + row_place<NP>(row, col)) = u32x2{lo[t], hi[t]};
                    }
                }
#pragma unroll
            for (int i = 0; i < kVi; ++i) {
                const int tile = wave + W * i, which = tile / kTiles, l = tile % kTiles;
                if (kImages * kTiles % W && tile >= kImages * kTiles) break;
                const int half = MODE == BACK ? upper_half(l) : lower_half(l);
                uint8_t *to = buf + (kQ ? 2 : 1) * kRows + which * kImg + (half >> 1) * OWN * 1024 + 16 * lane + 8 * (half & 1);
                const f32x4 v = __builtin_bit_cast(f32x4, ni[i]);
                uint32_t lo[OWN], hi[OWN];
                split2<OWN>(v[0], v[1], lo);
                split2<OWN>(v[2], v[3], hi);
#pragma unroll
                for (int t = 0; t < OWN; ++t) *(u32x2 *)(to + t * 1024) = u32x2{lo[t], hi[t]};
            }
            if (tid < kGates) *(float *)(buf + (kQ ? 2 : 1) * kRows + kImages * kImg + 4 * tid) = ngate;
            if constexpr (kStaged) {
#pragma unroll
                for (int i = 0; i < 2; ++i) *(u32x4 *)(lds + sizeof(lds) - kOwn + wave * C * 32 + 1024 * i + 16 * lane) = nv[i];
            }
        };
        if (di != d1) __syncthreads();   // the direction before has read its last chunk
        if (chunks > 0) {
            fetch(order(0));
            fetch_rows(order(0));
            fetch_values(order(0));
            stash(lds);
            if (kTwo && chunks > 1) {
                fetch(order(1));
                fetch_rows(order(1));
            }
        }
        for (int step = 0; step < chunks; ++step) {
            const int chunk = order(step), first = chunk * C, live = min(C, at.len - first);
            __syncthreads();
            const int lane = fresh(threadIdx.x & 63), g = lane >> 4, l16 = lane & 15;
            const int cur = kTwo ? step & 1 : 0;
            uint8_t *buf = lds + cur * kBuf;
            f32x4 x[4];
            if constexpr (kStaged) {
                // a tile's columns as lanes, four rows a lane: a result's order
                const uint16_t *v = (const uint16_t *)(lds + sizeof(lds) - kOwn + wave * C * 32) + 4 * lane;
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const u32x2 r = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16_d *)(v + 256 * t)));
                    x[t] = f32x4{__uint_as_float(r[0] << 16), __uint_as_float(r[0] & 0xffff0000u),
                                 __uint_as_float(r[1] << 16), __uint_as_float(r[1] & 0xffff0000u)};
                }
            } else {
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) x[t][r] = nx[t][r];
            }
            const bool more = step + 1 < chunks;
            if (more) fetch_values(order(step + 1));
            if (!kTwo && more) fetch(order(step + 1));
            // between the chunk's two halves
            auto middle = [&]() {
                if constexpr (kTwo) {
                    if (more) stash(lds + (cur ^ 1) * kBuf);
                    if (step + 2 < chunks) {
                        fetch(order(step + 2));
                        fetch_rows(order(step + 2));
                    }
                } else if (more) {
                    fetch_rows(order(step + 1));
                }
            };
            const uint8_t *kl = buf, *ql = buf + kRows;
            const uint8_t *one = buf + (kQ ? 2 : 1) * kRows, *two = one + kImg;
            const float *gate = (const float *)(one + kImages * kImg);
            // rows 16 rt .. of K or Q, k = n in the order of S's tiles
            auto rows = [&](const uint8_t *m, int rt, int s) {
                Operand<IN> o;
#pragma unroll
                for (int t = 0; t < IN; ++t)
                    o.t[t] = *(const u32x4 *)(m + t * C * NP * 2 + row_place<NP>(16 * rt + l16, 32 * s + 4 * g));
                return o;
            };
            // columns 16 nt .. as rows, k = tokens 32 s .. in the order of a result's tiles
            auto cols = [&](const uint8_t *m, int nt, int s) {
                Operand<IN> o;
#pragma unroll
                for (int t = 0; t < IN; ++t) {
                    const int row = 32 * s + 4 * g + (l16 >> 2), col = 16 * nt + 4 * (l16 & 3);
                    const uint8_t *q = m + t * C * NP * 2 + row_place<NP>(row, col);
                    const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16_d *)q));
                    const u32x2 hi = __builtin_bit_cast(
                        u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16_d *)(q + 16 * NP * 2)));
                    o.t[t] = u32x4{lo[0], lo[1], hi[0], hi[1]};
                }
                return o;
            };
            auto image = [&](const uint8_t *m, int b) {
                Operand<OWN> o;
#pragma unroll
                for (int t = 0; t < OWN; ++t) o.t[t] = *(const u32x4 *)(m + (b * OWN + t) * 1024 + 16 * lane);
                return o;
            };
            // c += the triangle times what b holds, two tiles at a time
            auto times_lower = [&](const uint8_t *m, const Operand<OWN> *b, f32x4 *c) {
                {
                    const Operand<OWN> i[2] = {image(m, lower_block(0, 0)), image(m, lower_block(1, 0))};
                    mm_tiles(i, b[0], c);
                }
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const Operand<OWN> i[2] = {image(m, lower_block(2, s)), image(m, lower_block(3, s))};
                    mm_tiles(i, b[s], c + 2);
                }
            };
            auto times_upper = [&](const uint8_t *m, const Operand<OWN> *b, f32x4 *c) {
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const Operand<OWN> i[2] = {image(m, upper_block(0, s)), image(m, upper_block(1, s))};
                    mm_tiles(i, b[s], c);
                }
                const Operand<OWN> i[2] = {image(m, upper_block(2, 1)), image(m, upper_block(3, 1))};
                mm_tiles(i, b[1], c + 2);
            };
            auto gates = [&](int which, int rt) { return *(const f32x4 *)(gate + which * C + 16 * rt + 4 * g); };
            f32x4 out[4];
            if (works) {
                if constexpr (GRAD) {
                    const __amdgpu_buffer_rsrc_t sr = __builtin_amdgcn_make_buffer_rsrc(
                        a.states + ((size_t)(at.slot + chunk) * a.H + h) * N * PP, 0, N * PP * 4, 0x00027000);
                    const uint32_t to = pw + 4 * g * PP * 4;
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int r = 0; r < 4; ++r) buf_store(sr, to + (16 * t + r) * PP * 4, S[t][r]);
                }
                if (early) middle();
                // K S and Q S
                f32x4 ks[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) ks[t] = out[t] = zero4();
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    const Operand<OWN> sb = split8<OWN>(S[2 * s], 2 * s + 1 < NT ? S[min(2 * s + 1, NT - 1)] : zero4());
                    Operand<IN> r[4];
#pragma unroll
                    for (int t = 0; t < 4; ++t) r[t] = rows(kl, t, s);
                    mm_tiles(r, sb, ks);
                    if constexpr (MODE == FWD) {
#pragma unroll
                        for (int t = 0; t < 4; ++t) r[t] = rows(ql, t, s);
                        mm_tiles(r, sb, out);
                    }
                }
                if (!early) middle();
                Operand<OWN> b[2], kb[2];   // kb: what K^T multiplies
                if constexpr (MODE != BACK) {
#pragma unroll
                    for (int t = 0; t < 4; ++t) x[t] -= gates(0, t) * ks[t];
#pragma unroll
                    for (int s = 0; s < 2; ++s) b[s] = split8<OWN>(x[2 * s], x[2 * s + 1]);
#pragma unroll
                    for (int t = 0; t < 4; ++t) ks[t] = zero4();
                    times_lower(one, b, ks);
#pragma unroll
                    for (int t = 0; t < 4; ++t) x[t] = gates(1, t) * gates(2, t) * ks[t];
#pragma unroll
                    for (int s = 0; s < 2; ++s) kb[s] = split8<OWN>(x[2 * s], x[2 * s + 1]);
                } else {
#pragma unroll
                    for (int s = 0; s < 2; ++s) b[s] = split8<OWN>(x[2 * s], x[2 * s + 1]);
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        ks[t] *= gates(1, t);
                        x[t] *= a.scale * gates(0, t);
                    }
                    times_upper(two, b, ks);
#pragma unroll
                    for (int s = 0; s < 2; ++s) b[s] = split8<OWN>(ks[2 * s], ks[2 * s + 1]);
                    times_upper(one, b, out);
#pragma unroll
                    for (int t = 0; t < 4; ++t) ks[t] = -gates(0, t) * gates(2, t) * out[t];
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        kb[s] = split8<OWN>(ks[2 * s], ks[2 * s + 1]);
                        b[s] = split8<OWN>(x[2 * s], x[2 * s + 1]);   // Q^T's
                    }
                }
                const float last = gate[C - 1];
#pragma unroll
                for (int t = 0; t < NT; ++t) S[t] *= last;
                constexpr int kGroup = NT < 4 ? NT : 4;
#pragma unroll
                for (int t = 0; t < NT; t += kGroup)
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        Operand<IN> m[kGroup];
#pragma unroll
                        for (int e = 0; e < kGroup; ++e) m[e] = cols(kl, t + e, s);
                        mm_tiles(m, kb[s], S + t);
                        if constexpr (MODE == BACK) {
#pragma unroll
                            for (int e = 0; e < kGroup; ++e) m[e] = cols(ql, t + e, s);
                            mm_tiles(m, b[s], S + t);
                        }
                    }
                if constexpr (MODE == FWD) {
#pragma unroll
                    for (int s = 0; s < 2; ++s) b[s] = split8<OWN>(ks[2 * s], ks[2 * s + 1]);
#pragma unroll
                    for (int t = 0; t < 4; ++t) out[t] *= a.scale * gates(0, t);
                    times_lower(two, b, out);
                } else if constexpr (MODE == KEEP) {
#pragma unroll
                    for (int t = 0; t < 4; ++t) out[t] = ks[t];
                }
            }
            else {
                middle();
            }
            if constexpr (!kTwo) {
                __syncthreads();
                // the next chunk goes to LDS before this one's results go out, so that
                // nothing waits for stores
                if (more) stash(buf);
            }
            if (works) {
                const int P = GRAD ? PP : a.P;
                const ChunkRows yr(a.y, at, a.reverse, first, live, (uint32_t)(a.H * P * 4), (uint32_t)(h * P * 4), P * 4);
                const uint32_t to = yr.offset(4 * g) + (GRAD ? pw : own ? (uint32_t)(4 * p) : kFar);
                if (MODE == FWD && a.add) {
#pragma unroll
                    for (int t = 0; t < 4; ++t)
#pragma unroll
                        for (int r = 0; r < 4; ++r) out[t][r] += buf_value(yr.rsrc, to + (16 * t + r) * yr.step, 0.f);
                }
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) buf_store(yr.rsrc, to + (16 * t + r) * yr.step, out[t][r]);
            }
        }
        if (a.last && own) {
#pragma unroll
            for (int t = 0; t < NT; ++t) *(f32x4 *)(a.last + state + 16 * t) = S[t];
        }
    }
}

// y += other, with both directions' outputs
__global__ __launch_bounds__(256) void k_delta_join(float *y, const float *other, long long n) {
    for (long long i = 4 * (blockIdx.x * 256LL + threadIdx.x); i < n; i += 1024LL * gridDim.x) {
        if (i + 4 <= n) {
            *(f32x4 *)(y + i) += *(const f32x4 *)(other + i);
        } else {
            for (long long j = i; j < n; ++j) y[j] += other[j];
        }
    }
}

template <typename T, int N>
struct Chunked {
    static hipError_t prep(const PrepDir *d, int ndir, bool grad, hipStream_t s) {
        PrepArgs p;
        p.dir[0] = d[0];
        p.dir[1] = d[ndir - 1];
        const DeltaArgs &a = d[0].a;
        const long long items = delta_slots(a.units, a.L, a.cu != nullptr) * a.H;
        const dim3 grid((unsigned)xcd_grid((items + kPrepWaves - 1) / kPrepWaves), ndir), block(64 * kPrepWaves);
        if (grad) BM_LAUNCH("delta_prep", (k_delta_prep<T, N, true>), grid, block, 0, s, p, items);
        else BM_LAUNCH("delta_prep", (k_delta_prep<T, N, false>), grid, block, 0, s, p, items);
        return hipGetLastError();
    }
    template <int MODE>
    static hipError_t walk(const PrepDir *d, int ndir, hipStream_t s) {
        static const char *const names[] = {"delta_walk", "delta_walk_keep", "delta_walk_back"};
        WalkArgs w;
        w.dir[0] = d[0];
        w.dir[1] = d[ndir - 1];
        w.ndir = ndir;
        const DeltaArgs &a = d[0].a;
        w.apart = ndir == 2 && d[0].a.y != d[1].a.y;
        const int ny = w.apart ? 2 : 1;
        // a wide head's 128 columns in one workgroup share its loads, on two CUs they
        // do not wait for each other (32 heads of 1024 tokens: forward 96 -> 89 us in bf16
        // and 168 -> 135 in fp32, back 121 -> 98 and 200 -> 149)
        w.blocks = a.P > 64 && 2LL * a.units * a.H * ny <= 256 ? 2 : 1;
        const dim3 grid((unsigned)xcd_grid((long long)a.units * a.H * w.blocks), ny);
        if (a.P > 64 && w.blocks == 1) BM_LAUNCH(names[MODE], (k_delta_walk<T, N, MODE, 8>), grid, dim3(512), 0, s, w);
        else BM_LAUNCH(names[MODE], (k_delta_walk<T, N, MODE, 4>), grid, dim3(256), 0, s, w);
        return hipGetLastError();
    }
};

// the workspace of a direction: triangles, then gates
size_t prep_triangles(const DeltaArgs &a, bool grad) {
    return (size_t)delta_slots(a.units, a.L, a.cu != nullptr) * a.H * triangles(grad) * kTriangle;
}
PrepDir prep_dir(const DeltaArgs &a, void *ws, bool grad) {
    PrepDir d;
    d.a = a;
    d.tri = (uint8_t *)ws;
    d.gates = (float *)((uint8_t *)ws + prep_triangles(a, grad));
    return d;
}

template <typename F>
hipError_t with_shape(const DeltaArgs &a, bool bf16, F f) {
#define GO(n)                                                              \
    if (a.N == n) return bf16 ? f(Chunked<uint16_t, n>()) : f(Chunked<float, n>());
    GO(16) GO(32) GO(64) GO(128)
#undef GO
    return hipErrorInvalidValue;
}

}  // namespace

// bytes, a multiple of 256; L and units of a, and whether it is packed (cu)
size_t delta_chunk_workspace(const DeltaArgs &a, bool grad) {
    const size_t slots = (size_t)delta_slots(a.units, a.L, a.cu != nullptr) * a.H;
    return prep_triangles(a, grad) + ((slots * kGateFloats * 4 + 255) & ~(size_t)255);
}

hipError_t launch_delta_chunked(const DeltaArgs *a, int ndir, bool bf16, void *const *ws, hipStream_t s) {
    PrepDir d[2];
    for (int i = 0; i < ndir; ++i) d[i] = prep_dir(a[i], ws[i], false);
    return with_shape(a[0], bf16, [&](auto k) {
        hipError_t e = hipSuccess;
        if (a[0].L > 0) e = k.prep(d, ndir, false, s);
        if (e == hipSuccess) e = k.template walk<FWD>(d, ndir, s);
        if (e != hipSuccess || ndir == 1 || a[0].y == a[1].y) return e;
        const long long n = (a[0].cu ? 1LL : a[0].units) * a[0].L * a[0].H * a[0].P;
        BM_LAUNCH("delta_join", k_delta_join, dim3((unsigned)std::min((n + 1023) / 1024, 1LL << 20)), dim3(256), 0, s, a[0].y, a[1].y, n);
        return hipGetLastError();
    });
}

hipError_t launch_delta_keep(const DeltaArgs *a, int ndir, bool bf16, void *const *ws, hipStream_t s) {
    PrepDir d[2];
    for (int i = 0; i < ndir; ++i) d[i] = prep_dir(a[i], ws[i], true);
    return with_shape(a[0], bf16, [&](auto k) {
        hipError_t e = k.prep(d, ndir, true, s);
        return e != hipSuccess ? e : k.template walk<KEEP>(d, ndir, s);
    });
}

const float *delta_gates(const DeltaArgs &a, void *ws) { return prep_dir(a, ws, true).gates; }

hipError_t launch_delta_back(const DeltaArgs *a, int ndir, bool bf16, void *const *ws, hipStream_t s) {
    PrepDir d[2];
    for (int i = 0; i < ndir; ++i) d[i] = prep_dir(a[i], ws[i], true);
    return with_shape(a[0], bf16, [&](auto k) { return k.template walk<BACK>(d, ndir, s); });
}

}  // namespace bm
