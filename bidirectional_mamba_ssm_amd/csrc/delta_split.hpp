// Operands of the delta rule's chunk kernels: numbers as sums of bf16 terms.
//
// bf16 inputs are one term, exactly. What the kernels compute (states, errors,
// the chunk's inverse) is kept as two terms, hi = bf16(v) and bf16(v - hi): 16
// significant bits over fp32's range. fp32 inputs and what is computed
// from them are three terms, all 24 bits. A product of operands keeps the pairs
// of terms that reach its last one: 2 for one by two, 3 for two by two, 6
// for three by three, each a v_mfma_f32_16x16x32_bf16 summed in fp32, the
// smallest first.
#pragma once
#include "delta.hpp"
#include "mfma.hpp"
#include "rows.hpp"

namespace bm {
namespace {

template <typename T> struct Terms;
template <> struct Terms<uint16_t> {
    static constexpr int IN = 1, OWN = 2;
};
template <> struct Terms<float> {
    static constexpr int IN = 3, OWN = 3;
};

template <int N> struct Operand {
    u32x4 t[N];
};

__device__ __forceinline__ uint32_t bf_pair(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(rf2{a, b}, rbf2));
}
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

// Workspace of a chunk and head: images of 64 x 64 triangles and the gates. An
// image holds the 6 blocks of 16 rows by 32 that are not zero, each as the
// operand's registers, a kilobyte a term: lane l's row l % 16, k slots 0..3 at
// 4 (l / 16) and 4..7 at 16 more.
constexpr int kBlocks = 6;
__device__ __forceinline__ constexpr int lower_block(int rt, int s) { return rt < 2 ? rt : 2 * rt - 2 + s; }
__device__ __forceinline__ constexpr int upper_block(int rt, int s) { return rt < 2 ? 2 * rt + s : rt + 2; }
template <int OWN> constexpr int kImage = kBlocks * OWN * 1024;   // bytes
constexpr int kGates = 3 * kDeltaChunk;                           // e^{G_i}, e^{G_C - G_i}, beta

}  // namespace
}  // namespace bm
