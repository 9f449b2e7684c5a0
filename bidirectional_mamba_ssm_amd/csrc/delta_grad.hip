// The gated delta rule's gradient from its two walks (delta_seq.hip), a
// 64-token chunk and a query and key group to a workgroup. With G_i the sum of
// g up to token i of the chunk, Gam_ij = e^{G_i - G_j}, S the state that enters
// the chunk, D the gradient of the one that leaves it, e and z the walks' errors
// and gradients, u = beta e, f = beta z, do = scale dy:
//   dP_ij = Gam_ij beta_j do_i . e_j (j <= i)    dM_ij = -Gam_ij beta_j f_i . e_j (j < i)
//   dq = e^{G_i} S do_i + sum_j dP_ij k_j
//   dk = -e^{G_i} S f_i + sum_j dM_ij k_j                                 (as row)
//      + e^{G_C - G_j} D u_j + sum_i dP_ij q_i + sum_i dM_ij k_i          (as column)
//   dv = f,  dbeta = e . z
//   dG_i = q_i . dq_i + k_i . dk_i (row) - k_i . dk_i (column), and at the chunk's
//   end <S, D> e^{G_C} + sum_j k_j . e^{G_C - G_j} D u_j;  dg = sum of dG from i on
// G is summed in 64 bits: differences of far larger sums enter the exponents.
// All products run on v_mfma_f32_16x16x4_f32 (lane l: row or column l % 16, k =
// l / 16), so that they are as exact as the walks. Rows of LDS are kept
// 20 words more than a multiple of 64 apart: four rows by sixteen columns and
// sixteen rows by four columns then both read without bank conflicts but for a
// few lanes. A wave owns 16 of the N columns; S and D have one reader each and
// go from memory to the operand's lanes. Heads that share the group are walked
// in order, their dq and dk summed in registers.
#include "delta.hpp"
#include "internal.hpp"
#include "mfma.hpp"
#include "rows.hpp"

namespace bm {
namespace {

constexpr int C = kDeltaChunk, kWaves = 8, kSlice = 32;
constexpr int kLd = kSlice + 4;   // rows of a slice: 36 words
constexpr int kLdM = C + 20;      // rows of dP and dM

__device__ __forceinline__ f32x4 mfma4(float a, float b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ float val(const uint16_t *p, size_t i) { return bf2f(p[i]); }
__device__ __forceinline__ float val(const float *p, size_t i) { return p[i]; }

template <typename T, int N>
__global__ __launch_bounds__(64 * kWaves) void k_delta_grad(DeltaArgs a, DeltaGradArgs o) {
    constexpr int LD = N + 20;
    // slices of do, e and z; dP and dM once those are done with
    constexpr int kShared = 3 * C * kLd > 2 * C * kLdM ? 3 * C * kLd : 2 * C * kLdM;
    __shared__ float qs[C * LD], ks[C * LD], shared[kShared];
    __shared__ float beta[C], up[C], down[C], logs[2][kWaves][C], ends[kWaves];
    __shared__ double sums[C], dlog[C], dend[C];
    float *dos = shared, *es = shared + C * kLd, *zs = shared + 2 * C * kLd;
    float *dp = shared, *dm = shared + C * kLdM;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g4 = lane >> 4, l16 = lane & 15;
    const int grp = blockIdx.x % a.G;
    const long long slot = blockIdx.x / a.G;
    int chunk;
    const DeltaUnit at = delta_slot(a, slot, chunk);
    const int first = chunk * C, live = min(C, at.len - first);
    if (live <= 0) return;
    auto token = [&](int i) { return (size_t)delta_token(at, a.reverse, first + i); };
    for (int e = tid; e < C * N; e += 64 * kWaves) {
        const int r = e / N, c = e % N;
        const size_t i = r < live ? (token(r) * a.G + grp) * N + c : 0;
        qs[r * LD + c] = r < live ? val((const T *)a.q, i) : 0.f;
        ks[r * LD + c] = r < live ? val((const T *)a.k, i) : 0.f;
    }
    const int n0 = 16 * wave;              // this wave's columns of dq and dk
    const bool mine = n0 < N;
    f32x4 dq[4], dk[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) dq[i] = dk[i] = zero4();
    const int rep = a.H / a.G;
    for (int h = grp * rep; h < (grp + 1) * rep; ++h) {
        __syncthreads();   // what the head before left in LDS is read
        if (tid < C) {
            beta[tid] = tid < live ? a.beta[token(tid) * a.H + h] : 0.f;
            // no decay below e^-1000 is told from a reset, and infinities cancel
            const float g = tid < live ? a.g[token(tid) * a.H + h] : 0.f;
            sums[tid] = g < -1000.f ? -1000.0 : (double)g;
        }
        __syncthreads();
        double sum = 0.0;
        if (tid < C)
            for (int i = 0; i <= tid; ++i) sum += sums[i];
        __syncthreads();
        if (tid < C) sums[tid] = sum;
        __syncthreads();
        if (tid < C) {
            up[tid] = expf((float)sum);
            down[tid] = expf((float)(sums[C - 1] - sum));
        }
        f32x4 aq[4], af[4], ae[4], x1[2], x2[2];
#pragma unroll
        for (int i = 0; i < 4; ++i) aq[i] = af[i] = ae[i] = zero4();
        x1[0] = x1[1] = x2[0] = x2[1] = zero4();
        float along = 0.f, db = 0.f;   // <S, D> and e . z of this lane
        const float *S = o.enter + ((size_t)slot * a.H + h) * a.P * N, *D = o.leave + ((size_t)slot * a.H + h) * a.P * N;
        const int row = tid >> 3, col = (tid & 7) * 4;
        for (int p0 = 0; p0 < a.P; p0 += kSlice) {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int p = p0 + col + j;
                const bool in = row < live && p < a.P;
                const size_t i = in ? (token(row) * a.H + h) * a.P + p : 0;
                const float e = in ? o.e[i] : 0.f, z = in ? o.z[i] : 0.f;
                dos[row * kLd + col + j] = in ? a.scale * o.dy[i] : 0.f;
                es[row * kLd + col + j] = e;
                zs[row * kLd + col + j] = z;
                db = fmaf(e, z, db);
                if (in) o.dv[i] = beta[row] * z;
            }
            __syncthreads();
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int tile = wave + kWaves * t, it = tile >> 2, jt = tile & 3;
                if (jt > it) continue;
#pragma unroll
                for (int k = 0; k < kSlice; k += 4) {
                    const float b = es[(16 * jt + l16) * kLd + k + g4];
                    x1[t] = mfma4(dos[(16 * it + l16) * kLd + k + g4], b, x1[t]);
                    x2[t] = mfma4(zs[(16 * it + l16) * kLd + k + g4], b, x2[t]);
                }
            }
            if (mine) {
#pragma unroll
                for (int k = 0; k < kSlice; k += 4) {
                    const int p = p0 + k + g4;
                    const float s = p < a.P ? S[(size_t)p * N + n0 + l16] : 0.f;
                    const float d = p < a.P ? D[(size_t)p * N + n0 + l16] : 0.f;
                    along = fmaf(s, d, along);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int m = (16 * i + l16) * kLd + k + g4;
                        aq[i] = mfma4(dos[m], s, aq[i]);
                        af[i] = mfma4(zs[m], s, af[i]);
                        ae[i] = mfma4(es[m], d, ae[i]);
                    }
                }
            }
        }
        __syncthreads();   // slices read: dP and dM take their place
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int tile = wave + kWaves * t, it = tile >> 2, jt = tile & 3;
            if (jt > it) continue;
            const int j = 16 * jt + l16;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 16 * it + 4 * g4 + r;
                const float w = j <= i ? beta[j] * expf((float)(sums[i] - sums[j])) : 0.f;
                dp[i * kLdM + j] = j <= i ? w * x1[t][r] : 0.f;
                dm[i * kLdM + j] = j < i ? -w * beta[i] * x2[t][r] : 0.f;
            }
        }
        __syncthreads();
        if (mine) {
            f32x4 rowk[4], colk[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int t = 16 * i + 4 * g4 + r;
                    aq[i][r] *= up[t];
                    rowk[i][r] = -up[t] * beta[t] * af[i][r];
                    ae[i][r] *= down[t] * beta[t];
                }
                colk[i] = ae[i];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // rows of tile i take columns up to it
                for (int k = 0; k < 16 * (i + 1); k += 4) {
                    const float b = ks[(k + g4) * LD + n0 + l16];
                    aq[i] = mfma4(dp[(16 * i + l16) * kLdM + k + g4], b, aq[i]);
                    rowk[i] = mfma4(dm[(16 * i + l16) * kLdM + k + g4], b, rowk[i]);
                }
                // columns of tile i take rows from it
                for (int k = 16 * i; k < C; k += 4) {
                    const int m = (k + g4) * kLdM + 16 * i + l16, b = (k + g4) * LD + n0 + l16;
                    colk[i] = mfma4(dp[m], qs[b], colk[i]);
                    colk[i] = mfma4(dm[m], ks[b], colk[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int t = 16 * i + 4 * g4 + r, m = t * LD + n0 + l16;
                    const float q = qs[m], k = ks[m];
                    const float l = group_total<16>(fmaf(q, aq[i][r], k * (rowk[i][r] - colk[i][r])));
                    const float f = group_total<16>(k * ae[i][r]);
                    if (l16 == 0) {
                        logs[0][wave][t] = l;
                        logs[1][wave][t] = f;
                    }
                }
                dq[i] += aq[i];
                dk[i] += rowk[i] + colk[i];
            }
        }
        along = wave_total(along);
        if (lane == 0) ends[wave] = along;
        db = group_total<8>(db);
        if ((tid & 7) == 0 && row < live) o.dbeta[token(row) * a.H + h] = db;
        __syncthreads();
        if (tid < C) {
            double d = 0.0, f = 0.0;
#pragma unroll
            for (int w = 0; w < N / 16; ++w) {
                d += (double)logs[0][w][tid];
                f += (double)logs[1][w][tid];
            }
            // dG of this token, and its part of the chunk's end, which is the
            // last token's (places past it hold zeros)
            dlog[tid] = d;
            dend[tid] = f;
        }
        __syncthreads();
        if (tid < C) {
            double d = 0.0;
            for (int w = 0; w < N / 16; ++w) d += (double)ends[w];
            d *= (double)up[C - 1];
#pragma unroll 4
            for (int i = 0; i < C; ++i) d += i >= tid ? dlog[i] + dend[i] : dend[i];
            if (tid < live) o.dg[token(tid) * a.H + h] = (float)d;
        }
    }
    if (!mine) return;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int t = 16 * i + 4 * g4 + r;
            if (t >= live) continue;
            const size_t m = (token(t) * a.G + grp) * N + n0 + l16;
            o.dq[m] = dq[i][r];
            o.dk[m] = dk[i][r];
        }
}

template <typename T>
hipError_t launch_t(const DeltaArgs &a, const DeltaGradArgs &o, hipStream_t s) {
    const dim3 grid((unsigned)(delta_slots(a.units, a.L, a.cu != nullptr) * a.G)), block(64 * kWaves);
#define GO(n)                                                                        \
    if (a.N == n) {                                                                  \
        BM_LAUNCH("delta_grad", (k_delta_grad<T, n>), grid, block, 0, s, a, o);        \
        return hipGetLastError();                                                    \
    }
    GO(16) GO(32) GO(64) GO(128)
#undef GO
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_delta_grad(const DeltaArgs &a, const DeltaGradArgs &o, bool bf16, hipStream_t s) {
    return bf16 ? launch_t<uint16_t>(a, o, s) : launch_t<float>(a, o, s);
}

}  // namespace bm
