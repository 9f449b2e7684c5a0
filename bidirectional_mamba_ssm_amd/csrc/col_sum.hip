// Second half of the weight gradients' reductions: the workgroups of a
// gradient kernel each leave a row of partial sums, and these are added here
// down the columns, in a fixed order and in fp64 (the partial sums are fp32;
// adding them is a small part of the work, and this way the number of
// workgroups does not show in the result's accuracy).
//
// Columns are [taps][channels], and [channels] more where there is a bias:
// column (k, c) goes to w[c * taps + k], column (taps, c) to b[c]. A workgroup
// takes 32 columns (128-byte runs of a row) and 32 interleaved slices of the
// rows, joined through LDS, or, where there are columns enough for every CU, 128
// and 8: more work a thread and fewer joins (2 x 21 760 columns of 64 rows 9.5
// -> 5 us; 4096 columns of 512 rows, 32 workgroups then, 4 -> 6).
#include "internal.hpp"

namespace bm {
namespace {

constexpr int kThreads = 1024;

struct ColSums {
    ColSum set[2];
};

template <int kCols>
__global__ __launch_bounds__(kThreads) void k_col_sum(ColSums all) {
    constexpr int kSlices = kThreads / kCols;
    const ColSum a = all.set[blockIdx.y];
    __shared__ double part[kSlices][kCols];
    const int lane = threadIdx.x % kCols, slice = threadIdx.x / kCols;
    const long long cols = (long long)(a.taps + a.bias) * a.ch;
    const long long col = (long long)blockIdx.x * kCols + lane;
    double s = 0.0;
    if (col < cols) {
        const float *p = a.part + col;
        int r = slice;
        for (; r + 7 * kSlices < a.n; r += 8 * kSlices) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = p[(size_t)(r + i * kSlices) * cols];
#pragma unroll
            for (int i = 0; i < 8; ++i) s += (double)v[i];
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
    if ((cols + 127) / 128 * nsets < 256)
        BM_LAUNCH("col_sum", k_col_sum<32>, dim3((unsigned)((cols + 31) / 32), nsets), dim3(kThreads), 0, s, all);
    else
        BM_LAUNCH("col_sum", k_col_sum<128>, dim3((unsigned)((cols + 127) / 128), nsets), dim3(kThreads), 0, s, all);
    return hipGetLastError();
}

}  // namespace bm
