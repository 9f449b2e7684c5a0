// Where packed sequences start, as bits: what the training-step convolutions
// (conv1d_act8.hip, conv1d_bwd.hip) know of them. Both walk scan positions p
// (token p, or L-1-p in the reverse direction), where a sequence's first
// position is its offset, or L minus the offset of the sequence after it.
#pragma once
#include "common.hpp"
#include "internal.hpp"

namespace bm {

// Bit m of the pair tells that position base + m (m < 128) is the first of a
// sequence and not of the row. The same in every lane.
struct StartBits {
    uint64_t lo = 0, hi = 0;
    __device__ __forceinline__ StartBits() {}
    __device__ __forceinline__ StartBits(const ConvSeqs &s, int base, int L, bool rev) {
        const int lane = threadIdx.x & 63;
        if (s.seq) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int p = base + 64 * h + lane;
                const bool in = p > 0 && p < L;
                const int t = in ? (rev ? L - 1 - p : p) : 0, u = in ? (rev ? t + 1 : t - 1) : 0;
                (h ? hi : lo) = __ballot(in && s.seq[t] != s.seq[u]);
            }
        } else {
            for (int i = 0; i < s.count; i += 64) {
                const int off = i + lane < s.count ? s.off[i + lane] : 0;
                const int m = (rev ? L - off : off) - base;
                uint64_t hit = __ballot(off > 0 && off < L && m >= 0 && m < 128);
                while (hit) {
                    const int at = __builtin_amdgcn_readlane(m, __builtin_ctzll(hit));
                    if (at < 64) lo |= 1ull << at;
                    else hi |= 1ull << (at - 64);
                    hit &= hit - 1;
                }
            }
        }
    }
    // n bits from m on (m + n <= 128)
    __device__ __forceinline__ uint32_t from(int m, int n) const {
        const uint64_t w = m >= 64 ? hi >> (m - 64) : lo >> m | (m ? hi << (64 - m) : 0);
        return (uint32_t)w & ((1u << n) - 1);
    }
};

}  // namespace bm
