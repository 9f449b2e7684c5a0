// 8-bit activation checkpoints (rows.hpp): packing an array of rows and
// reading it back. Both are streams bounded by HBM: an element of 2 or 4
// bytes is read or written once, its 1 + 1/32 bytes of checkpoint once. A lane
// holds 16 bytes of a row (8 bf16 or 4 fp32 channels), a block of 32 channels
// 4 or 8 adjacent lanes, whose largest magnitude comes by DPP lane moves.
// Measured at 8192 x 4352 bf16: packing 20 us, 108 MB at 5.5 TB/s, reading back
// 17 us. Rows of whole blocks are one run of lanes with no gaps; rows that end
// inside a block start a new one, and their last vector is moved element by
// element.
#include "internal.hpp"
#include "rows.hpp"

namespace bm {
namespace {

constexpr int kThreads = 256;

// FLAT: rows of whole blocks, taken as one long row
template <typename T, bool PACK, bool FLAT>
__global__ __launch_bounds__(kThreads) void k_act8(Act8Args a) {
    using L = Lane<T>;
    constexpr int V = L::V, LB = 32 / V;                 // lanes of a block
    const long long lanes = (a.C + 31) / 32 * LB;        // lanes of a row
    const long long total = a.rows * lanes;
    // whole waves stay in the loop together (block_max reads its neighbours)
    const long long base = (long long)blockIdx.x * kThreads + threadIdx.x;
    const long long wave0 = base & ~63LL;
    for (long long off = 0; wave0 + off < total; off += (long long)gridDim.x * kThreads) {
        const long long i = base + off;
        const long long row = FLAT ? 0 : i / lanes;
        const long long l = i - row * lanes;
        const long long c = l * V;
        const bool in = i < total;
        const int n = !in ? 0 : FLAT ? V : (int)min((long long)V, max(0LL, a.C - c));   // elements of this lane
        const size_t at = (size_t)row * a.C + c;
        const size_t sat = (size_t)row * (lanes / LB) + l / LB;
        if constexpr (PACK) {
            const T *x = (const T *)a.x + at;
            float v[V];
            if (n == V) {
                const rvec r = L::load(x);
#pragma unroll
                for (int j = 0; j < V; ++j) v[j] = L::get(r, j);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) v[j] = j < n ? Elem<T>::load(x, j) : 0.f;
            }
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < V; ++j) top = max(top, abs_bits(v[j]));
            top = block_max<LB>(top);
            uint32_t code[V];
            act8_codes<V>(v, top, code);
            if (n == V) {
                Bytes<V>::store(a.q + at, Bytes<V>::pack(code));
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (j < n) a.q[at + j] = (int8_t)code[j];
            }
            if (in && l % LB == 0) a.scale[sat] = (uint8_t)(top >> 23);
        } else {
            if (n == 0) continue;
            const float unit = act8_unit(a.scale[sat]);
            T *x = (T *)a.x + at;
            if (n == V) {
                float v[V];
                Bytes<V>::values(Bytes<V>::load(a.q + at), unit, v);
                L::store(x, L::pack(v));
            } else {
                for (int j = 0; j < n; ++j) {
                    const float v = (float)a.q[at + j] * unit;
                    if constexpr (sizeof(T) == 2) x[j] = f2bf(v);
                    else x[j] = v;
                }
            }
        }
    }
}

template <typename T, bool PACK, bool FLAT>
hipError_t launch_f(const Act8Args &a, hipStream_t s) {
    const long long lanes = (a.C + 31) / 32 * (32 / Lane<T>::V) * a.rows;
    const long long wgs = (lanes + kThreads - 1) / kThreads;
    const dim3 grid((unsigned)(wgs < 8192 ? wgs : 8192));
    BM_LAUNCH(PACK ? "act8_pack" : "act8_unpack", (k_act8<T, PACK, FLAT>), grid, dim3(kThreads), 0, s, a);
    return hipGetLastError();
}
template <typename T, bool PACK>
hipError_t launch_t(Act8Args a, hipStream_t s) {
    if (a.C % 32) return launch_f<T, PACK, false>(a, s);
    a.C *= a.rows;
    a.rows = 1;
    return launch_f<T, PACK, true>(a, s);
}

}  // namespace

hipError_t launch_act8(Act8Args a, bool bf16, bool pack, hipStream_t s) {
    if (a.rows == 0) return hipSuccess;
    if (pack) return bf16 ? launch_t<uint16_t, true>(a, s) : launch_t<float, true>(a, s);
    return bf16 ? launch_t<uint16_t, false>(a, s) : launch_t<float, false>(a, s);
}

}  // namespace bm
