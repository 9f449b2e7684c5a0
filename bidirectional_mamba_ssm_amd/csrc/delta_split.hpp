// Operands of the delta rule's chunk kernels: numbers as sums of bf16 terms.
//
// bf16 inputs are one term, exactly; fp32 inputs and everything the kernels
// compute (states, errors, the chunk's inverse) are three terms, bf16(v), bf16 of
// what is left and bf16 of what is left then: all 24 bits of a magnitude from 2^-110
// up to bf16's largest number. Below, what is left ends at bf16's last step, 2^-133;
// the numbers above (from 3.396e38 on, the last 1 in 256 of the top binade) round to
// an infinity (a first term held at the largest number would keep them, and cost
// the layer's forward 154 -> 159 us and its gradient 806 -> 819). A
// product of operands keeps the pairs of terms that reach its last one: 3 for one
// by three, 6 for three by three, each a v_mfma_f32_16x16x32_bf16 summed in
// fp32, the smallest first. (Two terms, 2 and 3 products, are off by 5e-6 of a
// result's norm, three by 1e-7; six bf16 products take 96 cycles where the fp32
// matrix instructions take 256.)
//
// Rows of tokens are read and written through buffer descriptors that end
// with the chunk's last token: reads past it give zeros, writes past it are
// dropped, and so are those of lanes whose column is put far outside.
#pragma once
#include "delta.hpp"
#include "mfma.hpp"
#include "rows.hpp"

namespace bm {
namespace {

template <typename T> struct Terms;
template <> struct Terms<uint16_t> {
    static constexpr int IN = 1, OWN = 3;
};
template <> struct Terms<float> {
    static constexpr int IN = 3, OWN = 3;
};

template <int N> struct Operand {
    u32x4 t[N];
};

// two numbers as N terms each
template <int N>
__device__ __forceinline__ void split2(float a, float b, uint32_t *t) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        t[i] = bf_pair(a, b);
        if (i + 1 < N) {
            a -= __uint_as_float(t[i] << 16);
            b -= __uint_as_float(t[i] & 0xffff0000u);
        }
    }
}
// k slots 0..3 from v, 4..7 from w
template <int N>
__device__ __forceinline__ Operand<N> split8(f32x4 v, f32x4 w) {
    Operand<N> o;
    uint32_t t[4][N];
    split2<N>(v[0], v[1], t[0]);
    split2<N>(v[2], v[3], t[1]);
    split2<N>(w[0], w[1], t[2]);
    split2<N>(w[2], w[3], t[3]);
#pragma unroll
    for (int i = 0; i < N; ++i) o.t[i] = u32x4{t[0][i], t[1][i], t[2][i], t[3][i]};
    return o;
}
template <int A, int B>
__device__ __forceinline__ f32x4 mm(const Operand<A> &a, const Operand<B> &b, f32x4 c) {
    constexpr int most = A > B ? A : B;
#pragma unroll
    for (int s = most - 1; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < A; ++i) {
            const int j = s - i;
            if (j >= 0 && j < B) c = mfma16x16x32(a.t[i], b.t[j], c);
        }
    return c;
}

constexpr uint32_t kFar = 0x80000000u;   // an offset past every descriptor's end (chunks are under 2^30 bytes)

// The rows of one chunk of an array [tok][row bytes], `len` bytes of each from
// `off` on. Row i of the walk is at offset(i).
struct ChunkRows {
    __amdgpu_buffer_rsrc_t rsrc;
    uint32_t base;    // of row 0
    int32_t step;     // to the next row
    __device__ __forceinline__ ChunkRows(const void *p, const DeltaUnit &d, bool reverse, int first, int live,
                                         uint32_t row, uint32_t off, uint32_t len) {
        const long long low = d.start + (reverse ? d.len - first - live : first);
        rsrc = __builtin_amdgcn_make_buffer_rsrc((uint8_t *)const_cast<void *>(p) + low * row + off, 0,
                                                 (int)((live - 1) * row + len), 0x00027000);
        base = reverse ? (uint32_t)(live - 1) * row : 0u;
        step = reverse ? -(int32_t)row : (int32_t)row;
    }
    __device__ __forceinline__ uint32_t offset(int i) const { return base + (uint32_t)(i * step); }
};
__device__ __forceinline__ u32x4 buf16(__amdgpu_buffer_rsrc_t r, uint32_t at) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
}
__device__ __forceinline__ float buf_value(__amdgpu_buffer_rsrc_t r, uint32_t at, float) {
    return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0));
}
__device__ __forceinline__ uint16_t buf_value(__amdgpu_buffer_rsrc_t r, uint32_t at, uint16_t) {
    return __builtin_amdgcn_raw_buffer_load_b16(r, at, 0, 0);
}
__device__ __forceinline__ void buf_store(__amdgpu_buffer_rsrc_t r, uint32_t at, float v) {
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), r, at, 0, 0);
}

// the sum of a chunk's logarithms of decays up to each token, a token a lane, in
// 64 bits: nothing is told from a reset below e^-1000, infinities would cancel,
// and a reset in the middle takes nothing from the decays behind it
__device__ __forceinline__ double decay_sums(float g, int lane) {
    double s = g < -1000.f ? -1000.0 : (double)g;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const double o = __shfl_up(s, d);
        if (lane >= d) s += o;
    }
    return s;
}

// all pairs of terms for M tiles at a time, so that products on one result
// are apart
template <int A, int B, int M>
__device__ __forceinline__ void mm_tiles(const Operand<A> (&a)[M], const Operand<B> &b, f32x4 *c) {
    constexpr int most = A > B ? A : B;
#pragma unroll
    for (int s = most - 1; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < A; ++i) {
            const int j = s - i;
            if (j >= 0 && j < B) {
#pragma unroll
                for (int m = 0; m < M; ++m) c[m] = mfma16x16x32(a[m].t[i], b.t[j], c[m]);
            }
        }
}

// Workspace of a chunk and head: 64 x 64 triangles and the gates. A triangle is
// kept as its 10 tiles of 16 x 16, fp32, a kilobyte each, a lane's four
// entries as an operand wants them: row l % 16, k = 4 (l / 16) ... In LDS it is
// an image: 6 blocks of 16 rows by 32 that are not zero, each as the operand's
// registers, a kilobyte a term: k slots 0..3 from one tile, 4..7 from the next.
constexpr int kBlocks = 6, kTiles = 10;
__device__ __forceinline__ constexpr int lower(int i, int j) { return i * (i + 1) / 2 + j; }
__device__ __forceinline__ constexpr int lower_block(int rt, int s) { return rt < 2 ? rt : 2 * rt - 2 + s; }
__device__ __forceinline__ constexpr int upper_block(int rt, int s) { return rt < 2 ? 2 * rt + s : rt + 2; }
// row and column tile of the l-th lower tile
__device__ __forceinline__ constexpr int lower_row(int l) { return l < 1 ? 0 : l < 3 ? 1 : l < 6 ? 2 : 3; }
__device__ __forceinline__ constexpr int lower_col(int l) { return l - lower_row(l) * (lower_row(l) + 1) / 2; }
template <int OWN> constexpr int kImage = kBlocks * OWN * 1024;   // bytes, in LDS
constexpr int kTriangle = kTiles * 1024;                          // bytes, in memory
// where a tile's half of a block is, in kilobytes of one term and its half of the
// 16 bytes of a lane: as rows i with k = j, or as rows j with k = i
__device__ __forceinline__ int lower_half(int l) {
    const int i = lower_row(l), j = lower_col(l);
    return 2 * lower_block(i, j >> 1) + (j & 1);
}
__device__ __forceinline__ int upper_half(int l) {
    const int i = lower_row(l), j = lower_col(l);
    return 2 * upper_block(j, i >> 1) + (i & 1);
}
// the gates: e^{G_i}, e^{G_C - G_i}, beta, and G_i in 64 bits
constexpr int kGates = 3 * kDeltaChunk, kGateFloats = 5 * kDeltaChunk;
// columns of the walks' own arrays: e and z [tok][H][padded], states [slot][H][N][padded]
__host__ __device__ constexpr int padded(int P) { return (P + 31) & ~31; }

}  // namespace
}  // namespace bm
