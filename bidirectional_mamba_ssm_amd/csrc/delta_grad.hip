// The gated delta rule's gradient from its two walks (delta_chunk.hip), a
// 64-token chunk and a query and key group to a workgroup. With G_i the sum of
// g up to token i of the chunk, Gam_ij = e^{G_i - G_j}, S the state that enters
// the chunk, D the gradient of the one that leaves it, e and z the walks' errors
// and gradients, u = beta e, f = beta z, do = dy:
//   dP_ij = scale Gam_ij beta_j do_i . e_j (j <= i)    dM_ij = -Gam_ij beta_j f_i . e_j (j < i)
//   dq = scale e^{G_i} S do_i + sum_j dP_ij k_j
//   dk = -e^{G_i} S f_i + sum_j dM_ij k_j                                 (as row)
//      + e^{G_C - G_j} D u_j + sum_i dP_ij q_i + sum_i dM_ij k_i          (as column)
//   dv = f,  dbeta = e . z
//   dG_i = q_i . dq_i + k_i . dk_i (row) - k_i . dk_i (column), and at the chunk's
//   end <S, D> e^{G_C} + sum_j k_j . e^{G_C - G_j} D u_j;  dg = sum of dG from i on
//
// Products are of three-term operands (delta_split.hpp). A wave owns 16 of the N
// columns of dq and dk: its rows of S and D and its columns of K and Q have no other
// reader and go from memory to the operand's registers. do, e and z are
// everyone's: 32 columns a k step come to LDS as operand images, rows of tokens
// with the head's columns as k, which serve as either operand. The triangles
// dP and dM take their place then, each twice: a result's lanes are the
// transpose's operand as they come, and the other way goes by halves of a word.
// Heads that share the group are walked in order, each lane adding to its own
// elements of dq and dk: no atomics, the same bits every time.
#include "delta_split.hpp"
#include "internal.hpp"

namespace bm {
namespace {

constexpr int C = kDeltaChunk;

template <typename T, int N>
__global__ __launch_bounds__(N == 128 ? 512 : 256) void k_delta_grad(DeltaArgs a, DeltaGradArgs o) {
    constexpr int IN = Terms<T>::IN, OWN = 3, W = N == 128 ? 8 : 4, SL = W / 4;   // waves; k steps of a slice
    constexpr int kRow = 4 * OWN * 1024;                   // images of 64 rows, a k step
    constexpr int kSlice = 3 * SL * kRow, kTri = 4 * kImage<OWN>;
    constexpr int kJobs = (20 + W - 1) / W;                // lower tiles of dP and dM, a wave
    __shared__ __attribute__((aligned(16))) uint8_t lds[kSlice > kTri ? kSlice : kTri];
    __shared__ double sums[C];
    __shared__ float gate[3][C], logs[2][W][C], ends[W], dbs[SL][C];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, l16 = lane & 15;
    const int grp = blockIdx.x % a.G, PP = padded(a.P);
    const long long slot = blockIdx.x / a.G;
    int chunk;
    const DeltaUnit at = delta_slot(a, slot, chunk);
    const int first = chunk * C, live = min(C, at.len - first);
    if (live <= 0) return;
    auto image = [&](int off, int b) {
        Operand<OWN> v;
#pragma unroll
        for (int t = 0; t < OWN; ++t) v.t[t] = *(const u32x4 *)(lds + off + (b * OWN + t) * 1024 + 16 * lane);
        return v;
    };
    const int n0 = 16 * wave;              // this wave's columns of dq and dk
    const bool mine = n0 < N;
    // its columns of K and Q: a lane's column, tokens in the order of a result's tiles
    Operand<IN> kb[2], qb[2];
    if (mine) {
        const uint32_t row = (uint32_t)(a.G * N * sizeof(T)), off = (uint32_t)(grp * N * sizeof(T));
        const ChunkRows kr(a.k, at, a.reverse, first, live, row, off, N * sizeof(T));
        const ChunkRows qr(a.q, at, a.reverse, first, live, row, off, N * sizeof(T));
        const uint32_t base = kr.offset(4 * g) + (n0 + l16) * (uint32_t)sizeof(T);
        auto columns = [&](const ChunkRows &rows, int s) {
            f32x4 v[2];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const T x = buf_value(rows.rsrc, base + (32 * s + 16 * (e >> 2) + (e & 3)) * rows.step, T());
                if constexpr (sizeof(T) == 2) v[e >> 2][e & 3] = bf2f(x);
                else v[e >> 2][e & 3] = x;
            }
            return split8<IN>(v[0], v[1]);
        };
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            kb[s] = columns(kr, s);
            qb[s] = columns(qr, s);
        }
    }
    // the value of token 16 t + 4 g + r back from its terms
    auto value = [&](const Operand<IN> *m, int t, int r) {
        float v = 0.f;
#pragma unroll
        for (int e = IN - 1; e >= 0; --e) {
            const uint32_t w = m[t >> 1].t[e][2 * (t & 1) + (r >> 1)];
            v += __uint_as_float(r & 1 ? w & 0xffff0000u : w << 16);
        }
        return v;
    };
    const uint32_t row4 = (uint32_t)(a.G * N * 4), off4 = (uint32_t)(grp * N * 4);
    const ChunkRows dqr(o.dq, at, a.reverse, first, live, row4, off4, N * 4);
    const ChunkRows dkr(o.dk, at, a.reverse, first, live, row4, off4, N * 4);
    const int rep = a.H / a.G;
    for (int h = grp * rep; h < (grp + 1) * rep; ++h) {
        if (wave == 0) {
            const size_t i = (size_t)delta_token(at, a.reverse, first + min(lane, live - 1)) * a.H + h;
            const double sum = decay_sums(lane < live ? a.g[i] : 0.f, lane);
            sums[lane] = sum;
            gate[0][lane] = expf((float)sum);
            gate[1][lane] = expf((float)(__shfl(sum, 63) - sum));
            gate[2][lane] = lane < live ? a.beta[i] : 0.f;
        }
        // a thread brings eight columns of a token of do, e and z
        const uint32_t off = (uint32_t)h * a.P * 4, row = (uint32_t)a.H * a.P * 4;
        const uint32_t offp = (uint32_t)h * PP * 4, rowp = (uint32_t)a.H * PP * 4;
        const ChunkRows dr(o.dy, at, a.reverse, first, live, row, off, a.P * 4);
        const ChunkRows vr(o.dv, at, a.reverse, first, live, row, off, a.P * 4);
        const ChunkRows er(o.e, at, a.reverse, first, live, rowp, offp, PP * 4);
        const ChunkRows zr(o.z, at, a.reverse, first, live, rowp, offp, PP * 4);
        const int mytok = 16 * (wave & 3) + l16, mycol = 32 * (wave >> 2) + 8 * g;
        const bool whole = a.P % 8 == 0;
        u32x4 nd[2], ne[2], nz[2];
        u32x4 ns[SL][2], nl[SL][2];
        const float *S = o.enter + (((size_t)slot * a.H + h) * N + n0 + l16) * PP;
        const float *D = o.leave + (((size_t)slot * a.H + h) * N + n0 + l16) * PP;
        auto fetch = [&](int p0) {
            const int p = p0 + mycol;
            const uint32_t in = p < PP ? 4 * p : kFar;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                ne[e] = buf16(er.rsrc, er.offset(mytok) + in + 16 * e);
                nz[e] = buf16(zr.rsrc, zr.offset(mytok) + in + 16 * e);
                if (whole) {
                    nd[e] = buf16(dr.rsrc, dr.offset(mytok) + (p < a.P ? 4 * p : kFar) + 16 * e);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int q = p + 4 * e + j;
                        nd[e][j] = __float_as_uint(buf_value(dr.rsrc, dr.offset(mytok) + (q < a.P ? 4 * q : kFar), 0.f));
                    }
                }
            }
        };
        auto fetch_states = [&](int s, int p0) {
            if (!mine || p0 + 32 * s >= PP) return;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                ns[s][e] = *(const u32x4 *)(S + p0 + 32 * s + 8 * g + 4 * e);
                nl[s][e] = *(const u32x4 *)(D + p0 + 32 * s + 8 * g + 4 * e);
            }
        };
        f32x4 aq[4], af[4], ae[4], x[kJobs];
#pragma unroll
        for (int i = 0; i < 4; ++i) aq[i] = af[i] = ae[i] = zero4();
#pragma unroll
        for (int i = 0; i < kJobs; ++i) x[i] = zero4();
        float along = 0.f, db = 0.f;   // <S, D> and e . z of this lane
        fetch(0);
#pragma unroll
        for (int s = 0; s < SL; ++s) fetch_states(s, 0);
        for (int p0 = 0; p0 < a.P; p0 += 32 * SL) {
            __syncthreads();
            const f32x4 e0 = __builtin_bit_cast(f32x4, ne[0]), e1 = __builtin_bit_cast(f32x4, ne[1]);
            const f32x4 z0 = __builtin_bit_cast(f32x4, nz[0]), z1 = __builtin_bit_cast(f32x4, nz[1]);
            {
                const Operand<OWN> d = split8<OWN>(__builtin_bit_cast(f32x4, nd[0]), __builtin_bit_cast(f32x4, nd[1]));
                const Operand<OWN> e = split8<OWN>(e0, e1), z = split8<OWN>(z0, z1);
                uint8_t *to = lds + (wave >> 2) * 3 * kRow + (wave & 3) * OWN * 1024 + 16 * lane;
#pragma unroll
                for (int t = 0; t < OWN; ++t) {
                    *(u32x4 *)(to + t * 1024) = d.t[t];
                    *(u32x4 *)(to + kRow + t * 1024) = e.t[t];
                    *(u32x4 *)(to + 2 * kRow + t * 1024) = z.t[t];
                }
            }
            const float beta = gate[2][mytok];
#pragma unroll
            for (int j = 0; j < 4; ++j) db = fmaf(e0[j], z0[j], fmaf(e1[j], z1[j], db));
            {
                const int p = p0 + mycol;
                const f32x4 f[2] = {beta * z0, beta * z1};
                if (whole) {
                    const uint32_t to = vr.offset(mytok) + (p < a.P ? 4 * p : kFar);
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, f[0]), vr.rsrc, to, 0, 0);
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, f[1]), vr.rsrc, to + 16, 0, 0);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        buf_store(vr.rsrc, vr.offset(mytok) + (p + j < a.P ? 4 * (p + j) : kFar), f[j >> 2][j & 3]);
                }
            }
            __syncthreads();
            if (p0 + 32 * SL < a.P) fetch(p0 + 32 * SL);
#pragma unroll
            for (int s = 0; s < SL; ++s) {
                const int im = s * 3 * kRow;
#pragma unroll
                for (int t = 0; t < kJobs; ++t) {
                    const int job = wave + W * t;
                    if (job >= 20) break;
                    const int l = job < 10 ? job : job - 10;
                    x[t] = mm(image(im + (job < 10 ? 0 : 2) * kRow, lower_row(l)), image(im + kRow, lower_col(l)), x[t]);
                }
                if (mine && p0 + 32 * s < PP) {
                    const f32x4 s0 = __builtin_bit_cast(f32x4, ns[s][0]), s1 = __builtin_bit_cast(f32x4, ns[s][1]);
                    const f32x4 l0 = __builtin_bit_cast(f32x4, nl[s][0]), l1 = __builtin_bit_cast(f32x4, nl[s][1]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) along = fmaf(s0[j], l0[j], fmaf(s1[j], l1[j], along));
                    const Operand<OWN> sb = split8<OWN>(s0, s1), lb = split8<OWN>(l0, l1);
                    fetch_states(s, p0 + 32 * SL);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        aq[i] = mm(image(im, i), sb, aq[i]);
                        ae[i] = mm(image(im + kRow, i), lb, ae[i]);
                        af[i] = mm(image(im + 2 * kRow, i), sb, af[i]);
                    }
                }
            }
        }
        __syncthreads();   // slices read: dP, dM and their transposes take their place
        if (wave < 4) {
            // tiles beyond the diagonal that share a block with one that is not
            const int b = wave == 0 ? lower_block(0, 0) : wave == 1 ? lower_block(2, 1) : wave == 2 ? upper_block(1, 0) : upper_block(3, 1);
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
                for (int t = 0; t < OWN; ++t)
                    *(u32x2 *)(lds + (wave < 2 ? w : 2 + w) * kImage<OWN> + (b * OWN + t) * 1024 + 16 * lane +
                               (wave < 2 ? 8 : 0)) = u32x2{0u, 0u};
        }
#pragma unroll
        for (int t = 0; t < kJobs; ++t) {
            const int job = wave + W * t;
            if (job >= 20) break;
            const bool second = job >= 10;
            const int l = second ? job - 10 : job, it = lower_row(l), jt = lower_col(l), j = 16 * jt + l16;
            float v[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 16 * it + 4 * g + r;
                const float w = j <= i ? gate[2][j] * expf((float)(sums[i] - sums[j])) : 0.f;
                v[r] = !second ? a.scale * w * x[t][r] : j < i ? -w * gate[2][i] * x[t][r] : 0.f;
            }
            uint32_t lo[OWN], hi[OWN];
            split2<OWN>(v[0], v[1], lo);
            split2<OWN>(v[2], v[3], hi);
            // as rows j (a lane's), k = i
            uint8_t *up = lds + (2 + second) * kImage<OWN> + upper_block(jt, it >> 1) * OWN * 1024 + 16 * lane + 8 * (it & 1);
            // as rows i, k = j: one slot in each of four lanes' registers
            uint8_t *low = lds + second * kImage<OWN> + lower_block(it, jt >> 1) * OWN * 1024 +
                           16 * (4 * g + 16 * (l16 >> 2)) + 2 * ((l16 & 3) + 4 * (jt & 1));
#pragma unroll
            for (int e = 0; e < OWN; ++e) {
                *(u32x2 *)(up + e * 1024) = u32x2{lo[e], hi[e]};
                *(uint16_t *)(low + e * 1024) = (uint16_t)lo[e];
                *(uint16_t *)(low + e * 1024 + 16) = (uint16_t)(lo[e] >> 16);
                *(uint16_t *)(low + e * 1024 + 32) = (uint16_t)hi[e];
                *(uint16_t *)(low + e * 1024 + 48) = (uint16_t)(hi[e] >> 16);
            }
        }
        __syncthreads();
        if (mine) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f32x4 up = *(const f32x4 *)&gate[0][16 * i + 4 * g], down = *(const f32x4 *)&gate[1][16 * i + 4 * g];
                const f32x4 beta = *(const f32x4 *)&gate[2][16 * i + 4 * g];
                f32x4 rowk = -up * beta * af[i], colk = down * beta * ae[i];
                const f32x4 fall = colk;
                aq[i] *= a.scale * up;
#pragma unroll
                for (int s = 0; s < (i < 2 ? 1 : 2); ++s) {
                    aq[i] = mm(image(0, lower_block(i, s)), kb[s], aq[i]);
                    rowk = mm(image(kImage<OWN>, lower_block(i, s)), kb[s], rowk);
                }
#pragma unroll
                for (int s = i < 2 ? 0 : 1; s < 2; ++s) {
                    colk = mm(image(2 * kImage<OWN>, upper_block(i, s)), qb[s], colk);
                    colk = mm(image(3 * kImage<OWN>, upper_block(i, s)), kb[s], colk);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float q = value(qb, i, r), k = value(kb, i, r);
                    const float l = group_total<16>(fmaf(q, aq[i][r], k * (rowk[r] - colk[r])));
                    const float f = group_total<16>(k * fall[r]);
                    if (l16 == 0) {
                        logs[0][wave][16 * i + 4 * g + r] = l;
                        logs[1][wave][16 * i + 4 * g + r] = f;
                    }
                }
                // this lane's sums over the heads so far
                rowk += colk;
                const uint32_t to = dqr.offset(4 * g) + 4 * (n0 + l16);
                if (h > grp * rep) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        aq[i][r] += buf_value(dqr.rsrc, to + (16 * i + r) * dqr.step, 0.f);
                        rowk[r] += buf_value(dkr.rsrc, to + (16 * i + r) * dqr.step, 0.f);
                    }
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    buf_store(dqr.rsrc, to + (16 * i + r) * dqr.step, aq[i][r]);
                    buf_store(dkr.rsrc, to + (16 * i + r) * dqr.step, rowk[r]);
                }
            }
        }
        along = wave_total(along);
        if (lane == 0) ends[wave] = along;
        db += __shfl_xor(db, 16);
        db += __shfl_xor(db, 32);
        if (g == 0) dbs[wave >> 2][mytok] = db;
        __syncthreads();
        if (wave == 0) {
            // dG of this lane's token; the chunk's end is its last token's, which
            // every token reaches back from (places past it hold zeros)
            double d = 0.0, f = 0.0, dot = 0.0;
            float b = 0.f;
#pragma unroll
            for (int w = 0; w < N / 16; ++w) {
                d += (double)logs[0][w][lane];
                f += (double)logs[1][w][lane];
                dot += (double)ends[w];
            }
#pragma unroll
            for (int w = 0; w < SL; ++w) b += dbs[w][lane];
#pragma unroll
            for (int m = 1; m < 64; m *= 2) {
                const double from = __shfl_down(d, m);
                if (lane + m < 64) d += from;
                f += __shfl_xor(f, m);
            }
            d += f + dot * (double)gate[0][C - 1];
            if (lane < live) {
                const size_t i = (size_t)delta_token(at, a.reverse, first + lane) * a.H + h;
                o.dg[i] = (float)d;
                o.dbeta[i] = b;
            }
        }
        __syncthreads();   // the next head's gates and slices
    }
}

template <typename T>
hipError_t launch_t(const DeltaArgs &a, const DeltaGradArgs &o, hipStream_t s) {
    const dim3 grid((unsigned)(delta_slots(a.units, a.L, a.cu != nullptr) * a.G));
#define GO(n)                                                                                    \
    if (a.N == n) {                                                                              \
        BM_LAUNCH("delta_grad", (k_delta_grad<T, n>), grid, dim3(n == 128 ? 512 : 256), 0, s, a, o); \
        return hipGetLastError();                                                                \
    }
    GO(16) GO(32) GO(64) GO(128)
#undef GO
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_delta_grad(const DeltaArgs &a, const DeltaGradArgs &o, bool bf16, hipStream_t s) {
    return bf16 ? launch_t<uint16_t>(a, o, s) : launch_t<float>(a, o, s);
}

// bytes of e or z, and of the kept states or their gradients
size_t delta_rows_bytes(const DeltaArgs &a) {
    const size_t tok = a.cu ? (size_t)a.L : (size_t)a.units * a.L;
    return tok * a.H * padded(a.P) * 4;
}
size_t delta_states_bytes(const DeltaArgs &a) {
    return (size_t)delta_slots(a.units, a.L, a.cu != nullptr) * a.H * a.N * padded(a.P) * 4;
}

}  // namespace bm
