// Second half of the weight gradients' reductions: the workgroups of a
// gradient kernel each leave a row of partial sums, and these are added here
// down the columns, in a fixed order and in fp64 (the partial sums are fp32;
// adding them is a small part of the work, and this way the number of
// workgroups does not show in the result's accuracy).
//
// Columns are [taps][channels], and [channels] more where there is a bias:
// column (k, c) goes to w[c * taps + k], column (taps, c) to b[c]. A workgroup takes 64 columns, its 16 waves 16
// interleaved slices of the rows, joined through LDS.
#include "internal.hpp"

namespace bm {
namespace {

constexpr int kSlices = 16;

struct ColSums {
    ColSum set[2];
};

__global__ __launch_bounds__(64 * kSlices) void k_col_sum(ColSums all) {
    const ColSum a = all.set[blockIdx.y];
    __shared__ double part[kSlices][64];
    const int lane = threadIdx.x & 63, slice = threadIdx.x >> 6;
    const long long cols = (long long)(a.taps + a.bias) * a.ch;
    const long long col = (long long)blockIdx.x * 64 + lane;
    double s = 0.0;
    if (col < cols) {
        const float *p = a.part + col;
        int r = slice;
        for (; r + 3 * kSlices < a.n; r += 4 * kSlices) {
            const float v0 = p[(size_t)r * cols], v1 = p[(size_t)(r + kSlices) * cols];
            const float v2 = p[(size_t)(r + 2 * kSlices) * cols], v3 = p[(size_t)(r + 3 * kSlices) * cols];
            s += ((double)v0 + (double)v1) + ((double)v2 + (double)v3);
        }
        for (; r < a.n; r += kSlices) s += (double)p[(size_t)r * cols];
    }
    part[slice][lane] = s;
    __syncthreads();
    if (slice != 0 || col >= cols) return;
    s = 0.0;
#pragma unroll
    for (int i = 0; i < kSlices; ++i) s += part[i][lane];
    const int k = (int)(col / a.ch), c = (int)(col % a.ch);
    if (k < a.taps) {
        if (a.w) a.w[(size_t)c * a.taps + k] = (float)s;
    } else if (a.b) {
        a.b[c] = (float)s;
    }
}

}  // namespace

hipError_t launch_col_sum(const ColSum *sets, int nsets, hipStream_t s) {
    ColSums all;
    all.set[0] = sets[0];
    all.set[1] = sets[nsets - 1];
    const long long cols = (long long)(sets[0].taps + sets[0].bias) * sets[0].ch;
    BM_LAUNCH("col_sum", k_col_sum, dim3((unsigned)((cols + 63) / 64), nsets), dim3(64 * kSlices), 0, s, all);
    return hipGetLastError();
}

}  // namespace bm
