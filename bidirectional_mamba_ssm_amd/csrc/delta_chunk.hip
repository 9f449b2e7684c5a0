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
// k_delta_prep, a chunk and head to a workgroup, makes what does not wait for
// the state: the triangles, inverted in fp32 (16 x 16 blocks by substitution, a
// column a lane; the blocks below by products on v_mfma_f32_16x16x4_f32), as
// operand images.
//
// k_delta_walk takes a head's chunks in order. A wave owns 16 NC columns of the
// state for all N rows; columns never meet. The matrix cores' result order (rows
// 4 g + r of a tile, column l % 16) serves as the next product's second operand as
// it is, if the first one's k order follows it: so S, V, E and Y never leave the
// wave's registers, and no product waits for another wave. K and Q come
// to LDS row by row (read as rows for K S and Q S, transposed by
// ds_read_b64_tr_b16 for K^T E), the images as they are; the next chunk's
// loads are under way meanwhile, one barrier a chunk (two where one buffer
// is all that fits).
#include "delta_split.hpp"
#include "internal.hpp"

namespace bm {
namespace {

constexpr int C = kDeltaChunk;
constexpr int kLd = C + 4;   // rows of the fp32 triangles in LDS
enum { FWD, KEEP, BACK };
// images of a chunk and head: FWD (I + M)^-1, A; for the gradient (I + M)^-1, (I + L)^-T, B^T
constexpr int images(bool grad) { return grad ? 3 : 2; }

__device__ __forceinline__ f32x4 mfma4(float a, float b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

struct PrepDir {
    DeltaArgs a;
    uint8_t *images;   // [slot][H]
    float *gates;      // [slot][H][kGates]
};
struct PrepArgs {
    PrepDir dir[2];
};

template <typename T, int N, bool GRAD>
__global__ __launch_bounds__(256) void k_delta_prep(PrepArgs args) {
    constexpr int IN = Terms<T>::IN, OWN = Terms<T>::OWN, KS = (N + 31) / 32, NM = GRAD ? 2 : 1;
    __shared__ __attribute__((aligned(16))) float ms[NM][C * kLd], xs[NM][C * kLd];
    __shared__ double sums[C];
    __shared__ float beta[C];
    const PrepDir &pd = args.dir[blockIdx.y];
    const DeltaArgs &a = pd.a;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, l16 = lane & 15;
    const int h = blockIdx.x % a.H, grp = h / (a.H / a.G);
    const long long slot = blockIdx.x / a.H;
    int chunk;
    const DeltaUnit at = delta_slot(a, slot, chunk);
    const int first = chunk * C, live = min(C, at.len - first);
    if (live <= 0) return;
    const uint32_t row = (uint32_t)(a.G * N * sizeof(T)), off = (uint32_t)(grp * N * sizeof(T));
    const ChunkRows kr(a.k, at, a.reverse, first, live, row, off, N * sizeof(T));
    const ChunkRows qr(a.q, at, a.reverse, first, live, row, off, N * sizeof(T));
    // all of K and this wave's 16 rows of Q, k in the rows' order
    constexpr int V = 16 / sizeof(T), kRegs = 8 / V;
    u32x4 kv[4][KS][kRegs], qv[KS][kRegs];
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int e = 0; e < kRegs; ++e) {
            const int n = 32 * s + 8 * g + V * e;
            const uint32_t col = n < N ? n * sizeof(T) : kFar;
            qv[s][e] = buf16(qr.rsrc, qr.offset(16 * wave + l16) + col);
#pragma unroll
            for (int c = 0; c < 4; ++c) kv[c][s][e] = buf16(kr.rsrc, kr.offset(16 * c + l16) + col);
        }
    if (wave == 0) {
        const size_t i = (size_t)delta_token(at, a.reverse, first + min(lane, live - 1)) * a.H + h;
        const double sum = decay_sums(lane < live ? a.g[i] : 0.f, lane);
        const float b = lane < live ? a.beta[i] : 0.f;
        sums[lane] = sum;
        beta[lane] = b;
        float *to = pd.gates + ((size_t)slot * a.H + h) * kGates;
        to[lane] = expf((float)sum);
        to[C + lane] = expf((float)(__shfl(sum, 63) - sum));
        to[2 * C + lane] = b;
    }
    auto operand = [&](const u32x4 *r) {
        if constexpr (IN == 1) return Operand<1>{r[0]};
        else return split8<3>(__builtin_bit_cast(f32x4, r[0]), __builtin_bit_cast(f32x4, r[1]));
    };
    // column c of the wave's rows of K K^T; of the other triangle the tile that is
    // an image's lane as it comes (rows j for q_i k_j, rows i for its transpose)
    f32x4 kk[4], qk[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) kk[c] = qk[c] = zero4();
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        const Operand<IN> q = operand(qv[s]);
        Operand<IN> k[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) k[c] = operand(kv[c][s]);
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int w = 0; w < 4; ++w)
                if (c <= w && w == wave) {
                    kk[c] = mm(k[w], k[c], kk[c]);
                    qk[c] = GRAD ? mm(q, k[c], qk[c]) : mm(k[c], q, qk[c]);
                }
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        if (c > wave) break;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            {
                const int i = 16 * wave + 4 * g + r, j = 16 * c + l16;
                const float w = j < i ? expf((float)(sums[i] - sums[j])) * kk[c][r] : 0.f;
                ms[0][i * kLd + j] = w * beta[j];
                if constexpr (GRAD) ms[1][i * kLd + j] = w * beta[i];
            }
            // FWD: lane's row i = l16, columns j; GRAD: rows i, lane's column j
            const int i = 16 * wave + (GRAD ? 4 * g + r : l16), j = 16 * c + (GRAD ? l16 : 4 * g + r);
            const float w = j <= i && i < live ? a.scale * expf((float)(sums[i] - sums[j])) : 0.f;
            qk[c][r] *= GRAD ? w : w * beta[j];
        }
    }
    uint8_t *img = pd.images + ((size_t)slot * a.H + h) * images(GRAD) * kImage<OWN>;
    auto put = [&](uint8_t *image, int b, f32x4 lo, f32x4 hi) {
        const Operand<OWN> o = split8<OWN>(lo, hi);
#pragma unroll
        for (int t = 0; t < OWN; ++t) *(u32x4 *)(image + (b * OWN + t) * 1024 + 16 * lane) = o.t[t];
    };
    if constexpr (!GRAD) {
        // tiles above the diagonal are zeros as they were
        put(img + kImage<OWN>, wave < 2 ? wave : 2 * wave - 2, qk[0], qk[1]);
        if (wave >= 2) put(img + kImage<OWN>, 2 * wave - 1, qk[2], qk[3]);
    } else {
        // the transposed triangle's rows 16 c .. take k from 16 wave ..: half a
        // block is one wave's, four slots of eight
        uint8_t *to = img + 2 * kImage<OWN>;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            uint32_t lo[OWN], hi[OWN];
            split2<OWN>(qk[c][0], qk[c][1], lo);
            split2<OWN>(qk[c][2], qk[c][3], hi);
            if (c < 2 || wave >= 2) {
#pragma unroll
                for (int t = 0; t < OWN; ++t)
                    *(u32x2 *)(to + (upper_block(c, wave >> 1) * OWN + t) * 1024 + 16 * lane + 8 * (wave & 1)) =
                        u32x2{lo[t], hi[t]};
            }
        }
    }
    __syncthreads();
    {   // this wave's diagonal block: lane's column l16 of the inverse
        const int which = GRAD ? g >> 1 : 0, o = 16 * wave;
        const float *m = ms[which] + o * kLd + o;
        f32x4 rows[16][4];
#pragma unroll
        for (int i = 1; i < 16; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (4 * k < i) rows[i][k] = *(const f32x4 *)(m + i * kLd + 4 * k);
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float v[4] = {i == l16 ? 1.f : 0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < i; ++k) v[k & 3] = fmaf(-rows[i][k >> 2][k & 3], x[k], v[k & 3]);
            x[i] = (v[0] + v[1]) + (v[2] + v[3]);
        }
        if (GRAD ? (g & 1) == 0 : g == 0) {
#pragma unroll
            for (int i = 0; i < 16; ++i) xs[which][(o + i) * kLd + o + l16] = x[i];
        }
    }
    __syncthreads();
    // X_ij = -X_ii sum_m M_im X_mj, a subdiagonal of blocks at a time
#pragma unroll
    for (int d = 1; d < 4; ++d) {
        for (int job = wave; job < NM * (4 - d); job += 4) {
            const int which = job / (4 - d), j = job % (4 - d), i = j + d;
            const float *m = ms[which];
            float *x = xs[which];
            const f32x4 own = *(const f32x4 *)(x + (16 * i + l16) * kLd + 16 * i + 4 * g);
            f32x4 t[2] = {zero4(), zero4()};
#pragma unroll
            for (int k = 0; k < 16 * d; k += 4) {
                const int n = 16 * j + k + g;
                t[(k >> 2) & 1] = mfma4(m[(16 * i + l16) * kLd + n], x[n * kLd + 16 * j + l16], t[(k >> 2) & 1]);
            }
            t[0] += t[1];
            f32x4 v = zero4();
#pragma unroll
            for (int r = 0; r < 4; ++r) v = mfma4(own[r], t[0][r], v);
#pragma unroll
            for (int r = 0; r < 4; ++r) x[(16 * i + 4 * g + r) * kLd + 16 * j + l16] = -v[r];
        }
        __syncthreads();
    }
    for (int job = wave; job < NM * kBlocks; job += 4) {
        const int which = job / kBlocks, b = job % kBlocks;
        const bool upper = which > 0;   // transposed
        const int rt = upper ? (b < 4 ? b >> 1 : b - 2) : (b < 2 ? b : (b + 2) >> 1);
        const int s = upper ? (b < 4 ? b & 1 : 1) : (b < 2 ? 0 : b & 1);
        const float *src = xs[which];
        f32x4 v[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int ct = 2 * s + e, col = 16 * ct + 4 * g, at16 = 16 * rt + l16;
            v[e] = zero4();
            if (!upper) {
                if (ct <= rt) v[e] = *(const f32x4 *)(src + at16 * kLd + col);
            } else if (ct >= rt) {
#pragma unroll
                for (int r = 0; r < 4; ++r) v[e][r] = src[(col + r) * kLd + at16];
            }
        }
        put(img + which * kImage<OWN>, b, v[0], v[1]);
    }
}

typedef short v4i16_d __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4i16_d lds_v4i16_d;

struct WalkArgs {
    PrepDir dir[2];
    int ndir;          // FWD: both directions' outputs are added, the reverse one's first
    int blocks;        // workgroups of a head
};

template <typename T, int N, int NC, int MODE>
__global__ __launch_bounds__(256, 1) void k_delta_walk(WalkArgs args) {
    using X = typename std::conditional<MODE == BACK, float, T>::type;   // the third input's type
    constexpr int IN = Terms<T>::IN, OWN = Terms<T>::OWN;
    constexpr bool GRAD = MODE != FWD;
    constexpr int NP = N < 32 ? 32 : N, KS = NP / 32, NT = N / 16;
    constexpr int RS = NP + 16;                         // row stride of K and Q in LDS, in elements
    constexpr int kRows = C * RS * 2 * IN;              // bytes of K or Q
    constexpr bool kQ = MODE != KEEP;                   // Q read, and a second image
    constexpr int kImages = kQ ? 2 : 1, kImg = kImage<OWN>;
    constexpr int kBuf = kRows * (kQ ? 2 : 1) + kImg * kImages + kGates * 4;
    constexpr int kBufs = 2 * kBuf <= 160 * 1024 ? 2 : 1;
    __shared__ __attribute__((aligned(16))) uint8_t lds[kBufs][kBuf];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, l16 = lane & 15;
    const int block = blockIdx.x % args.blocks, h = blockIdx.x / args.blocks % args.dir[0].a.H;
    const int u = blockIdx.x / args.blocks / args.dir[0].a.H;
    const int p0 = (block * 4 + wave) * 16 * NC;
    // the wave has columns, those of the walks' own arrays past the head's width among them
    const bool works = p0 < (GRAD ? padded(args.dir[0].a.P) : args.dir[0].a.P);
    for (int di = args.ndir - 1; di >= 0; --di) {
        const PrepDir &pd = args.dir[di];
        const DeltaArgs &a = pd.a;
        const int grp = h / (a.H / a.G), PP = padded(a.P);
        const DeltaUnit at = delta_unit(a, u);
        const int chunks = (at.len + C - 1) / C;
        // a lane's columns, in the caller's arrays and in the walks' own
        uint32_t pc[NC], pw[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int p = p0 + 16 * c + l16;
            pc[c] = p < a.P ? p : kFar;
            pw[c] = p < PP ? 4 * p : kFar;
        }
        f32x4 S[NT][NC];
        const size_t state = ((size_t)u * a.H + h) * a.P * N + 4 * g;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                S[t][c] = zero4();
                if (a.init && pc[c] != kFar) S[t][c] = *(const f32x4 *)(a.init + state + (size_t)pc[c] * N + 16 * t);
            }
        // the next chunk on its way: rows of K and Q, gates, the third input (the
        // images go straight to LDS)
        constexpr int V = 16 / sizeof(T), kVecs = C * NP / V / 256;
        u32x4 nk[kVecs], nq[kQ ? kVecs : 1];
        float ngate = 0.f;
        X nx[4][NC][4];
        auto order = [&](int i) { return MODE == BACK ? chunks - 1 - i : i; };
        auto fetch = [&](int chunk, uint8_t *to) {
            const int first = chunk * C, live = min(C, at.len - first);
            const size_t sh = (size_t)(at.slot + chunk) * a.H + h;
            const uint32_t row = (uint32_t)(a.G * N * sizeof(T)), off = (uint32_t)(grp * N * sizeof(T));
            const ChunkRows kr(a.k, at, a.reverse, first, live, row, off, N * sizeof(T));
            const ChunkRows qr(a.q, at, a.reverse, first, live, row, off, N * sizeof(T));
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const int e = tid + 256 * i, col = e % (NP / V) * V;
                const uint32_t o = kr.offset(e / (NP / V)) + (col < N ? (uint32_t)(col * sizeof(T)) : kFar);
                nk[i] = buf16(kr.rsrc, o);
                if (kQ) nq[i] = buf16(qr.rsrc, o);
            }
            const uint8_t *img = pd.images + sh * images(GRAD) * kImg + (MODE == BACK ? kImg : 0) + 16 * lane;
            for (int i = wave; i < kImages * kImg / 1024; i += 4)
                __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)(img + i * 1024),
                                                 (__attribute__((address_space(3))) void *)(to + (kQ ? 2 : 1) * kRows + i * 1024),
                                                 16, 0, 0);
            if (tid < kGates) ngate = pd.gates[sh * kGates + tid];
            if (!works) return;
            const uint32_t xrow = (uint32_t)(a.H * a.P * sizeof(X));
            const ChunkRows xr(a.v, at, a.reverse, first, live, xrow, (uint32_t)(h * a.P * sizeof(X)), a.P * sizeof(X));
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const uint32_t col = xr.offset(4 * g) + (pc[c] == kFar ? kFar : pc[c] * (uint32_t)sizeof(X));
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) nx[t][c][r] = buf_value(xr.rsrc, col + (16 * t + r) * xr.step, X());
            }
        };
        auto stash = [&](uint8_t *to) {
#pragma unroll
            for (int w = 0; w < (kQ ? 2 : 1); ++w)
#pragma unroll
                for (int i = 0; i < kVecs; ++i) {
                    const int e = tid + 256 * i, row = e / (NP / V), col = e % (NP / V) * V;
                    uint16_t *at16 = (uint16_t *)(to + w * kRows) + row * RS + col;
                    const u32x4 r = w ? nq[i] : nk[i];
                    if constexpr (IN == 1) {
                        *(u32x4 *)at16 = r;
                    } else {
                        uint32_t lo[IN], hi[IN];
                        split2<IN>(__uint_as_float(r[0]), __uint_as_float(r[1]), lo);
                        split2<IN>(__uint_as_float(r[2]), __uint_as_float(r[3]), hi);
#pragma unroll
                        for (int t = 0; t < IN; ++t) *(u32x2 *)(at16 + t * C * RS) = u32x2{lo[t], hi[t]};
                    }
                }
            if (tid < kGates) *(float *)(to + (kQ ? 2 : 1) * kRows + kImages * kImg + 4 * tid) = ngate;
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // the images are in LDS
        };
        if (di != args.ndir - 1) __syncthreads();   // the direction before has read its last chunk
        if (chunks > 0) {
            fetch(order(0), lds[0]);
            stash(lds[0]);
        }
        for (int step = 0; step < chunks; ++step) {
            const int chunk = order(step), first = chunk * C, live = min(C, at.len - first);
            const uint8_t *buf = lds[kBufs == 2 ? step & 1 : 0];
            uint8_t *nextbuf = lds[kBufs == 2 ? (step + 1) & 1 : 0];
            const bool more = step + 1 < chunks;
            __syncthreads();
            f32x4 x[4][NC];
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int c = 0; c < NC; ++c)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        if constexpr (sizeof(X) == 2) x[t][c][r] = bf2f(nx[t][c][r]);
                        else x[t][c][r] = nx[t][c][r];
                    }
            if (kBufs == 2 && more) fetch(order(step + 1), nextbuf);
            const uint16_t *kl = (const uint16_t *)buf, *ql = (const uint16_t *)(buf + kRows);
            const uint8_t *one = buf + (kQ ? 2 : 1) * kRows, *two = one + kImg;
            const float *gate = (const float *)(one + kImages * kImg);
            // rows 16 rt .. of K or Q, k = n in the order of S's tiles
            auto rows = [&](const uint16_t *m, int rt, int s) {
                Operand<IN> o;
#pragma unroll
                for (int t = 0; t < IN; ++t) {
                    const uint16_t *q = m + t * C * RS + (16 * rt + l16) * RS + 32 * s + 4 * g;
                    const u32x2 lo = *(const u32x2 *)q, hi = *(const u32x2 *)(q + 16);
                    o.t[t] = u32x4{lo[0], lo[1], hi[0], hi[1]};
                }
                return o;
            };
            // columns 16 nt .. as rows, k = tokens 32 s .. in the order of a result's tiles
            auto cols = [&](const uint16_t *m, int nt, int s) {
                Operand<IN> o;
#pragma unroll
                for (int t = 0; t < IN; ++t) {
                    const uint16_t *q =
                        m + t * C * RS + (32 * s + 4 * g + (l16 >> 2)) * RS + 16 * nt + 4 * (l16 & 3);
                    const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16_d *)q));
                    const u32x2 hi =
                        __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16_d *)(q + 16 * RS)));
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
            auto gates = [&](int which, int rt) { return *(const f32x4 *)(gate + which * C + 16 * rt + 4 * g); };
            f32x4 out[4][NC];
            if (works) {
                if constexpr (GRAD) {
                    const __amdgpu_buffer_rsrc_t sr = __builtin_amdgcn_make_buffer_rsrc(
                        a.states + ((size_t)(at.slot + chunk) * a.H + h) * N * PP, 0, N * PP * 4, 0x00027000);
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        const uint32_t o = pw[c] + 4 * g * PP * 4;
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int r = 0; r < 4; ++r) buf_store(sr, o + (16 * t + r) * PP * 4, S[t][c][r]);
                    }
                }
                // K S and Q S
                f32x4 ks[4][NC];
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int c = 0; c < NC; ++c) ks[t][c] = out[t][c] = zero4();
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    Operand<OWN> sb[NC];
#pragma unroll
                    for (int c = 0; c < NC; ++c)
                        sb[c] = split8<OWN>(S[2 * s][c], 2 * s + 1 < NT ? S[min(2 * s + 1, NT - 1)][c] : zero4());
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const Operand<IN> k = rows(kl, t, s);
#pragma unroll
                        for (int c = 0; c < NC; ++c) ks[t][c] = mm(k, sb[c], ks[t][c]);
                        if constexpr (MODE == FWD) {
                            const Operand<IN> q = rows(ql, t, s);
#pragma unroll
                            for (int c = 0; c < NC; ++c) out[t][c] = mm(q, sb[c], out[t][c]);
                        }
                    }
                }
                Operand<OWN> b[2][NC], kb[2][NC];   // kb: what K^T multiplies
                if constexpr (MODE != BACK) {
#pragma unroll
                    for (int s = 0; s < 2; ++s)
#pragma unroll
                        for (int c = 0; c < NC; ++c)
                            b[s][c] = split8<OWN>(x[2 * s][c] - gates(0, 2 * s) * ks[2 * s][c],
                                                  x[2 * s + 1][c] - gates(0, 2 * s + 1) * ks[2 * s + 1][c]);
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
#pragma unroll
                        for (int c = 0; c < NC; ++c) ks[t][c] = zero4();
#pragma unroll
                        for (int s = 0; s < (t < 2 ? 1 : 2); ++s) {
                            const Operand<OWN> m = image(one, lower_block(t, s));
#pragma unroll
                            for (int c = 0; c < NC; ++c) ks[t][c] = mm(m, b[s][c], ks[t][c]);
                        }
                    }
#pragma unroll
                    for (int s = 0; s < 2; ++s)
#pragma unroll
                        for (int c = 0; c < NC; ++c)
                            kb[s][c] = split8<OWN>(gates(1, 2 * s) * gates(2, 2 * s) * ks[2 * s][c],
                                                   gates(1, 2 * s + 1) * gates(2, 2 * s + 1) * ks[2 * s + 1][c]);
                } else {
#pragma unroll
                    for (int s = 0; s < 2; ++s)
#pragma unroll
                        for (int c = 0; c < NC; ++c) b[s][c] = split8<OWN>(x[2 * s][c], x[2 * s + 1][c]);
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
#pragma unroll
                        for (int c = 0; c < NC; ++c) ks[t][c] *= gates(1, t);
#pragma unroll
                        for (int s = t < 2 ? 0 : 1; s < 2; ++s) {
                            const Operand<OWN> m = image(two, upper_block(t, s));
#pragma unroll
                            for (int c = 0; c < NC; ++c) ks[t][c] = mm(m, b[s][c], ks[t][c]);
                        }
                    }
#pragma unroll
                    for (int s = 0; s < 2; ++s)
#pragma unroll
                        for (int c = 0; c < NC; ++c) b[s][c] = split8<OWN>(ks[2 * s][c], ks[2 * s + 1][c]);
#pragma unroll
                    for (int t = 0; t < 4; ++t)
#pragma unroll
                        for (int s = t < 2 ? 0 : 1; s < 2; ++s) {
                            const Operand<OWN> m = image(one, upper_block(t, s));
#pragma unroll
                            for (int c = 0; c < NC; ++c) out[t][c] = mm(m, b[s][c], out[t][c]);
                        }
#pragma unroll
                    for (int s = 0; s < 2; ++s)
#pragma unroll
                        for (int c = 0; c < NC; ++c) {
                            kb[s][c] = split8<OWN>(-gates(0, 2 * s) * gates(2, 2 * s) * out[2 * s][c],
                                                   -gates(0, 2 * s + 1) * gates(2, 2 * s + 1) * out[2 * s + 1][c]);
                            b[s][c] = split8<OWN>(a.scale * gates(0, 2 * s) * x[2 * s][c],
                                                  a.scale * gates(0, 2 * s + 1) * x[2 * s + 1][c]);   // Q^T's
                        }
                }
                const float last = gate[C - 1];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
#pragma unroll
                    for (int c = 0; c < NC; ++c) S[t][c] *= last;
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const Operand<IN> k = cols(kl, t, s);
#pragma unroll
                        for (int c = 0; c < NC; ++c) S[t][c] = mm(k, kb[s][c], S[t][c]);
                        if constexpr (MODE == BACK) {
                            const Operand<IN> q = cols(ql, t, s);
#pragma unroll
                            for (int c = 0; c < NC; ++c) S[t][c] = mm(q, b[s][c], S[t][c]);
                        }
                    }
                }
                if constexpr (MODE == FWD) {
#pragma unroll
                    for (int s = 0; s < 2; ++s)
#pragma unroll
                        for (int c = 0; c < NC; ++c) b[s][c] = split8<OWN>(ks[2 * s][c], ks[2 * s + 1][c]);
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
#pragma unroll
                        for (int c = 0; c < NC; ++c) out[t][c] *= a.scale * gates(0, t);
#pragma unroll
                        for (int s = 0; s < (t < 2 ? 1 : 2); ++s) {
                            const Operand<OWN> m = image(two, lower_block(t, s));
#pragma unroll
                            for (int c = 0; c < NC; ++c) out[t][c] = mm(m, b[s][c], out[t][c]);
                        }
                    }
                } else if constexpr (MODE == KEEP) {
#pragma unroll
                    for (int t = 0; t < 4; ++t)
#pragma unroll
                        for (int c = 0; c < NC; ++c) out[t][c] = ks[t][c];
                }
            }
            // what the next chunk brought goes to LDS before this one's results go
            // out, so that nothing waits for stores
            if (kBufs == 1) {
                __syncthreads();
                if (more) fetch(order(step + 1), nextbuf);
            }
            if (more) stash(nextbuf);
            if (works) {
                const int P = GRAD ? PP : a.P;
                const ChunkRows yr(a.y, at, a.reverse, first, live, (uint32_t)(a.H * P * 4), (uint32_t)(h * P * 4), P * 4);
                uint32_t o[NC];
#pragma unroll
                for (int c = 0; c < NC; ++c) o[c] = yr.offset(4 * g) + (GRAD ? pw[c] : pc[c] == kFar ? kFar : 4 * pc[c]);
                if (MODE == FWD && a.add) {
#pragma unroll
                    for (int c = 0; c < NC; ++c)
#pragma unroll
                        for (int t = 0; t < 4; ++t)
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                out[t][c][r] += buf_value(yr.rsrc, o[c] + (16 * t + r) * yr.step, 0.f);
                }
#pragma unroll
                for (int c = 0; c < NC; ++c)
#pragma unroll
                    for (int t = 0; t < 4; ++t)
#pragma unroll
                        for (int r = 0; r < 4; ++r) buf_store(yr.rsrc, o[c] + (16 * t + r) * yr.step, out[t][c][r]);
            }
        }
        if (a.last) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int c = 0; c < NC; ++c)
                    if (pc[c] != kFar) *(f32x4 *)(a.last + state + (size_t)pc[c] * N + 16 * t) = S[t][c];
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
        const dim3 grid((unsigned)(delta_slots(a.units, a.L, a.cu != nullptr) * a.H), ndir);
        if (grad) BM_LAUNCH("delta_prep", (k_delta_prep<T, N, true>), grid, dim3(256), 0, s, p);
        else BM_LAUNCH("delta_prep", (k_delta_prep<T, N, false>), grid, dim3(256), 0, s, p);
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
        const long long heads = (long long)a.units * a.H;
        const int wide = (a.P + 127) / 128, narrow = (a.P + 63) / 64;
        if constexpr (sizeof(T) == 2) {
            if (a.P > 64 && heads * wide >= 256) {
                w.blocks = wide;
                BM_LAUNCH(names[MODE], (k_delta_walk<T, N, 2, MODE>), dim3((unsigned)(heads * wide)), dim3(256), 0, s, w);
                return hipGetLastError();
            }
        }
        w.blocks = narrow;
        BM_LAUNCH(names[MODE], (k_delta_walk<T, N, 1, MODE>), dim3((unsigned)(heads * narrow)), dim3(256), 0, s, w);
        return hipGetLastError();
    }
};

// the workspace of a direction: images, then gates
size_t prep_images(const DeltaArgs &a, bool grad) {
    return (size_t)delta_slots(a.units, a.L, a.cu != nullptr) * a.H * images(grad) * kImage<3>;
}
PrepDir prep_dir(const DeltaArgs &a, void *ws, bool grad) {
    PrepDir d;
    d.a = a;
    d.images = (uint8_t *)ws;
    d.gates = (float *)((uint8_t *)ws + prep_images(a, grad));
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
    return prep_images(a, grad) + ((slots * kGates * 4 + 255) & ~(size_t)255);
}

hipError_t launch_delta_chunked(const DeltaArgs *a, int ndir, bool bf16, void *const *ws, hipStream_t s) {
    PrepDir d[2];
    for (int i = 0; i < ndir; ++i) d[i] = prep_dir(a[i], ws[i], false);
    return with_shape(a[0], bf16, [&](auto k) {
        hipError_t e = hipSuccess;
        if (a[0].L > 0) e = k.prep(d, ndir, false, s);
        return e != hipSuccess ? e : k.template walk<FWD>(d, ndir, s);
    });
}

hipError_t launch_delta_keep(const DeltaArgs &a, bool bf16, void *ws, hipStream_t s) {
    const PrepDir d = prep_dir(a, ws, true);
    return with_shape(a, bf16, [&](auto k) {
        hipError_t e = k.prep(&d, 1, true, s);
        return e != hipSuccess ? e : k.template walk<KEEP>(&d, 1, s);
    });
}

hipError_t launch_delta_back(const DeltaArgs &a, bool bf16, void *ws, hipStream_t s) {
    const PrepDir d = prep_dir(a, ws, true);
    return with_shape(a, bf16, [&](auto k) { return k.template walk<BACK>(&d, 1, s); });
}

}  // namespace bm
