// Device helpers of the row-wise training kernels (norms, 8-bit checkpoints):
// 16-byte lane vectors of a row, sums over a wave by DPP lane moves, and the
// 8-bit checkpoint code.
//
// 8-bit checkpoints (bimamba_act8): 32 consecutive channels of a row share
// one power of two. With E the largest fp32 exponent field among them, an
// element v is kept as the integer q = clamp(round(v 2^(133-E)), -127, 127)
// (nearest, ties to even) and stands for q 2^(E-133). Scaling by a power of
// two is exact, so the one rounding is the integer's: half a unit, 2^(E-134).
// For E >= 1 that is at most 2^-7 of the block's largest magnitude (one unit,
// as much, where the clamp takes effect); for E = 0, a largest magnitude of
// zero or an fp32 subnormal, the unit is 2^-133 whatever that magnitude is. q
// has 7 bits, so a decoded value is exact in bf16.
// A block that holds an infinity or a NaN has E = 255 and decodes as NaN.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"

namespace bm {

// Rows of any length start at any multiple of the element size; gfx950 takes
// vector loads and stores at such addresses (unaligned access is the
// target's default), so these types promise only the element's alignment.
typedef uint32_t u4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u4_a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u2_a1 __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t u1_a1 __attribute__((aligned(1)));
typedef uint32_t rvec __attribute__((ext_vector_type(4)));
typedef __bf16 rbf2 __attribute__((ext_vector_type(2)));
typedef float rf2 __attribute__((ext_vector_type(2)));

// two floats -> bf16, the first in the low half: round to nearest even, a NaN of
// any bits stays a NaN (hardware conversion)
__device__ __forceinline__ uint32_t bf_pair(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(rf2{a, b}, rbf2));
}

// one lane's vector of a row: 16 bytes, V elements
template <typename T> struct Lane;
template <> struct Lane<uint16_t> {
    static constexpr int V = 8;
    __device__ __forceinline__ static rvec load(const uint16_t *p) { return *(const u4_a2 *)p; }
    __device__ __forceinline__ static float get(rvec r, int j) {
        const uint32_t w = r[j >> 1];
        return __uint_as_float((j & 1) ? (w & 0xffff0000u) : (w << 16));
    }
    // round to nearest even (hardware conversion)
    __device__ __forceinline__ static rvec pack(const float *v) {
        rvec r;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const rf2 p = {v[2 * j], v[2 * j + 1]};
            r[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(p, rbf2));
        }
        return r;
    }
    __device__ __forceinline__ static void store(uint16_t *p, rvec r) { *(u4_a2 *)p = r; }
};
template <> struct Lane<float> {
    static constexpr int V = 4;
    __device__ __forceinline__ static rvec load(const float *p) { return *(const u4_a4 *)p; }
    __device__ __forceinline__ static float get(rvec r, int j) { return __uint_as_float(r[j]); }
    __device__ __forceinline__ static rvec pack(const float *v) {
        rvec r;
#pragma unroll
        for (int j = 0; j < 4; ++j) r[j] = __float_as_uint(v[j]);
        return r;
    }
    __device__ __forceinline__ static void store(float *p, rvec r) { *(u4_a4 *)p = r; }
};

// the low bytes of four words
__device__ __forceinline__ uint32_t bytes4(const uint32_t *q) {
    const uint32_t lo = __builtin_amdgcn_perm(q[1], q[0], 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(q[3], q[2], 0x04000c0cu);
    return lo | hi;
}
// q unit of four signed bytes (a sign-extending byte select and conversion,
// one instruction, and a product)
__device__ __forceinline__ void values4(uint32_t r, float unit, float *v) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = (float)(int8_t)(r >> (8 * j)) * unit;
}

// V bytes of an 8-bit checkpoint
template <int V> struct Bytes;
template <> struct Bytes<8> {
    typedef uint32_t type __attribute__((ext_vector_type(2)));
    __device__ __forceinline__ static type load(const int8_t *p) { return *(const u2_a1 *)p; }
    __device__ __forceinline__ static void store(int8_t *p, type r) { *(u2_a1 *)p = r; }
    __device__ __forceinline__ static type pack(const uint32_t *q) { return type{bytes4(q), bytes4(q + 4)}; }
    __device__ __forceinline__ static void values(type r, float unit, float *v) {
        values4(r[0], unit, v);
        values4(r[1], unit, v + 4);
    }
};
template <> struct Bytes<4> {
    typedef uint32_t type;
    __device__ __forceinline__ static type load(const int8_t *p) { return *(const u1_a1 *)p; }
    __device__ __forceinline__ static void store(int8_t *p, type r) { *(u1_a1 *)p = r; }
    __device__ __forceinline__ static type pack(const uint32_t *q) { return bytes4(q); }
    __device__ __forceinline__ static void values(type r, float unit, float *v) { values4(r, unit, v); }
};

// 2^(e-133) for a block's exponent field e, down to the subnormal 2^-133; NaN
// for 255
__device__ __forceinline__ float act8_unit(uint32_t e) {
    const float u = __builtin_ldexpf(1.0f, (int)e - 133);
    return e == 255 ? __uint_as_float(0x7fc00000u) : u;
}
// The integers kept for V values of a block whose largest magnitude has the
// bits `top`, in the low bytes of code[]. 1.5 2^23 + m holds round(m), ties to
// even, in its low bits, so one fma scales and rounds. Its factor 2^(133-E)
// overflows for E < 6, below 2^-121: there (but for zeros, whose factor does
// not matter) the scaling is a separate, also exact, step.
template <int V>
__device__ __forceinline__ void act8_codes(const float *v, uint32_t top, uint32_t *code) {
    constexpr float kInt = 12582912.f;
    const int e = (int)(top >> 23);
    const bool far = e < 6 && top != 0;
    const float s = __uint_as_float((uint32_t)(133 - max(e, 6) + 127) << 23);
    if (__any(far)) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float m = far ? __builtin_ldexpf(v[j], 133 - e) + kInt : fmaf(v[j], s, kInt);
            code[j] = __float_as_uint(fminf(fmaxf(m, kInt - 127.f), kInt + 127.f));
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
            code[j] = __float_as_uint(__builtin_amdgcn_fmed3f(fmaf(v[j], s, kInt), kInt - 127.f, kInt + 127.f));
    }
    if (__any(e == 255)) {   // a NaN block holds zeros
#pragma unroll
        for (int j = 0; j < V; ++j) code[j] = e == 255 ? 0u : code[j];
    }
}
// bits of a magnitude: they order as magnitudes do, infinities and NaN above all
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

template <int CTRL, int ROW = 0xf, int BANK = 0xf, bool BOUND = true>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROW, BANK, BOUND);
}
template <int CTRL, int ROW = 0xf>
__device__ __forceinline__ float dpp_add(float v) {
    return v + __uint_as_float(dpp<CTRL, ROW>(__float_as_uint(v)));
}
// largest over the LANES (2, 4 or 8) adjacent lanes that hold one block
template <int LANES>
__device__ __forceinline__ uint32_t block_max(uint32_t v) {
    v = max(v, dpp<0xB1>(v));                     // quad_perm [1,0,3,2]
    if constexpr (LANES > 2) v = max(v, dpp<0x4E>(v));   // quad_perm [2,3,0,1]
    if constexpr (LANES > 4) v = max(v, dpp<0x141>(v));  // row_half_mirror
    return v;
}
// sum over each G adjacent lanes (8, 16 or 32), the same in each of them
template <int G>
__device__ __forceinline__ float group_total(float v) {
    v = dpp_add<0xB1>(v);
    v = dpp_add<0x4E>(v);
    v = dpp_add<0x141>(v);
    if constexpr (G > 8) v = dpp_add<0x140>(v);
    if constexpr (G > 16) v += __shfl_xor(v, 16);
    return v;
}
// sum over the wave's 64 lanes, the same in every lane; a fixed order
__device__ __forceinline__ float wave_total(float v) {
    v = dpp_add<0xB1>(v);                         // lanes 1 apart
    v = dpp_add<0x4E>(v);                         // 2 apart
    v = dpp_add<0x141>(v);                        // the other quad of 8
    v = dpp_add<0x140>(v);                        // the other half of 16
    v = dpp_add<0x142, 0xa>(v);                   // row 0 into 1, 2 into 3
    v = dpp_add<0x143, 0xc>(v);                   // rows 0..1 into 2..3
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}

}  // namespace bm
