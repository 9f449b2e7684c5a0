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
// elements of dq and dk: no atomics, the same bits every time. Where chunks and
// groups are few, a group's heads go to several workgroups, whose sums are added
// in order at the end.
//
// Measured, 8 rows of 1024 tokens, 32 heads of 128 x 128 in 16 groups, bf16: 470 us
// for 1.2 GB (236 us at a copy's rate) and 225 GFLOP of three-term products; heads
// 96 wide 440; fp32 590. A head
// takes a workgroup 55 000 cycles: two slices 10 000 each, of which 5800 are
// products and 6900 the LDS's reads of the images, dP and dM 4000, their products
// 9000, and waits for the slices' arrays. Tried without gain (466 at
// the time): chunks in a loop with the next one's first slice under way (474), two
// workgroups of 64 columns a CU (505), tile pairs that share their reads (487).
#include <algorithm>

#include "delta_split.hpp"
#include "internal.hpp"

namespace bm {
namespace {

constexpr int C = kDeltaChunk;

struct GradArgs {
    DeltaArgs a[2];
    DeltaGradArgs o[2];
    int parts;      // workgroups that share a chunk and group
    long long n;    // elements of dq or dk
};

// The parts of a group's heads: enough that 256 workgroups, one a CU, have work
// (32 heads of one group, 1024 tokens: 467 us in one part, 55 in 16 with the sums)
int grad_parts(const DeltaArgs &a) {
    const long long work = delta_slots(a.units, a.L, a.cu != nullptr) * a.G * (delta_apart(a.units, a.H) ? 2 : 1);
    const int heads = a.H / a.G, most = (int)std::min<long long>(heads, (255 + work) / work);
    const int each = (heads + most - 1) / most;
    return (heads + each - 1) / each;
}

template <typename T, int N>
__global__ __launch_bounds__(N == 128 ? 512 : 256) void k_delta_grad(GradArgs args) {
    const DeltaArgs &a = args.a[blockIdx.y];
    const DeltaGradArgs &o = args.o[blockIdx.y];
    constexpr int IN = Terms<T>::IN, OWN = 3, W = N == 128 ? 8 : 4, SL = W / 4;   // waves; k steps of a slice
    constexpr int kRow = 4 * OWN * 1024;                   // images of 64 rows, a k step
    constexpr int kSlice = 3 * SL * kRow, kTri = 4 * kImage<OWN>;
    constexpr int kJobs = (20 + W - 1) / W;                // lower tiles of dP and dM, a wave
    __shared__ __attribute__((aligned(16))) uint8_t lds[kSlice > kTri ? kSlice : kTri];
    __shared__ double sums[C];
    __shared__ float gate[3][C], logs[2][W][C], ends[W], dbs[SL][C];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, l16 = lane & 15;
    const int part = (int)(blockIdx.x % args.parts), grp = (int)(blockIdx.x / args.parts % a.G), PP = padded(a.P);
    const long long slot = blockIdx.x / args.parts / a.G;
    int chunk;
    const DeltaUnit at = delta_slot(a, slot, chunk);
    const int first = chunk * C, live = min(C, at.len - first);
    if (live <= 0) return;
    // A lane's own number, as a stage of a head's work has it: the compiler would
    // keep what all stages make of it through the whole walk, far more than the
    // registers hold (58 of them went to memory, 590 us at the layer's shape). With
    // d_state 128 10 still do, and 57 in fp32, whose K and Q are three terms each.
    auto fresh = [&]() {
        int l = lane;
        asm volatile("" : "+v"(l));
        return l;
    };
    auto image = [&](int off, int b, int l) {
        Operand<OWN> v;
#pragma unroll
        for (int t = 0; t < OWN; ++t) v.t[t] = *(const u32x4 *)(lds + off + (b * OWN + t) * 1024 + 16 * l);
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
    float *own = o.parts + 2 * (part - 1) * args.n;
    const ChunkRows dqr(part ? own : o.dq, at, a.reverse, first, live, row4, off4, N * 4);
    const ChunkRows dkr(part ? own + args.n : o.dk, at, a.reverse, first, live, row4, off4, N * 4);
    const int heads = a.H / a.G, each = (heads + args.parts - 1) / args.parts;
    const int h0 = grp * heads + part * each, h1 = min(h0 + each, (grp + 1) * heads);
    // a thread brings eight columns of a token of do, e and z, a wave's lanes their
    // row of S and of D, the first wave's the gates
    const bool whole = a.P % 8 == 0;
    u32x4 nd[2], ne[2], nz[2], ns[SL][2], nl[SL][2];
    float ng[3];
    double nsum;
    auto fetch = [&](int h, int p0) {
        const int lane = fresh(), mytok = 16 * (wave & 3) + (lane & 15), mycol = 32 * (wave >> 2) + 8 * (lane >> 4);
        const ChunkRows dr(o.dy, at, a.reverse, first, live, (uint32_t)a.H * a.P * 4, (uint32_t)h * a.P * 4, a.P * 4);
        const ChunkRows er(o.e, at, a.reverse, first, live, (uint32_t)a.H * PP * 4, (uint32_t)h * PP * 4, PP * 4);
        const ChunkRows zr(o.z, at, a.reverse, first, live, (uint32_t)a.H * PP * 4, (uint32_t)h * PP * 4, PP * 4);
        const int p = p0 + mycol;
        const uint32_t in = er.offset(mytok) + (p < PP ? 4 * p : kFar);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            ne[e] = buf16(er.rsrc, in + 16 * e);
            nz[e] = buf16(zr.rsrc, in + 16 * e);
        }
        if (whole) {
            const uint32_t from = dr.offset(mytok) + (p < a.P ? 4 * p : kFar);
#pragma unroll
            for (int e = 0; e < 2; ++e) nd[e] = buf16(dr.rsrc, from + 16 * e);
        } else {
            const uint32_t from = dr.offset(mytok) + 4 * p;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                nd[j >> 2][j & 3] = __float_as_uint(buf_value(dr.rsrc, p + j < a.P ? from + 4 * j : kFar, 0.f));
        }
        if (p0 == 0 && wave == 0) {
            const float *from = o.gates + ((size_t)slot * a.H + h) * kGateFloats;
#pragma unroll
            for (int e = 0; e < 3; ++e) ng[e] = from[e * C + lane];
            nsum = ((const double *)(from + kGates))[lane];
        }
    };
    auto fetch_states = [&](int h, int p0, int s) {
        const int lane = fresh();
        const size_t from = (((size_t)slot * a.H + h) * N + n0 + (lane & 15)) * PP + p0 + 32 * s + 8 * (lane >> 4);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            ns[s][e] = *(const u32x4 *)(o.enter + from + 4 * e);
            nl[s][e] = *(const u32x4 *)(o.leave + from + 4 * e);
        }
    };
    fetch(h0, 0);
#pragma unroll
    for (int s = 0; s < SL; ++s)
        if (mine && 32 * s < PP) fetch_states(h0, 0, s);
    for (int h = h0; h < h1; ++h) {
        if (wave == 0) {
#pragma unroll
            for (int e = 0; e < 3; ++e) gate[e][lane] = ng[e];
            sums[lane] = nsum;
        }
        const ChunkRows vr(o.dv, at, a.reverse, first, live, (uint32_t)a.H * a.P * 4, (uint32_t)h * a.P * 4, a.P * 4);
        f32x4 acc[4][3], x[kJobs];   // acc: do S, e D, z S
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i][0] = acc[i][1] = acc[i][2] = zero4();
#pragma unroll
        for (int i = 0; i < kJobs; ++i) x[i] = zero4();
        float along = 0.f, db = 0.f;   // <S, D> and e . z of this lane
        for (int p0 = 0; p0 < a.P; p0 += 32 * SL) {
            __syncthreads();
            const int lane = fresh(), mytok = 16 * (wave & 3) + (lane & 15), mycol = 32 * (wave >> 2) + 8 * (lane >> 4);
            {
                const f32x4 e0 = __builtin_bit_cast(f32x4, ne[0]), e1 = __builtin_bit_cast(f32x4, ne[1]);
                const f32x4 z0 = __builtin_bit_cast(f32x4, nz[0]), z1 = __builtin_bit_cast(f32x4, nz[1]);
                uint8_t *to = lds + (wave >> 2) * 3 * kRow + (wave & 3) * OWN * 1024 + 16 * lane;
                auto put = [&](int which, f32x4 lo, f32x4 hi) {
                    const Operand<OWN> v = split8<OWN>(lo, hi);
#pragma unroll
                    for (int t = 0; t < OWN; ++t) *(u32x4 *)(to + which * kRow + t * 1024) = v.t[t];
                };
                put(0, __builtin_bit_cast(f32x4, nd[0]), __builtin_bit_cast(f32x4, nd[1]));
                put(1, e0, e1);
                put(2, z0, z1);
                const float beta = gate[2][mytok];
#pragma unroll
                for (int j = 0; j < 4; ++j) db = fmaf(e0[j], z0[j], fmaf(e1[j], z1[j], db));
                const int p = p0 + mycol;
                const f32x4 f[2] = {beta * z0, beta * z1};
                if (whole) {
                    const uint32_t out = vr.offset(mytok) + (p < a.P ? 4 * p : kFar);
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, f[0]), vr.rsrc, out, 0, 0);
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, f[1]), vr.rsrc, out + 16, 0, 0);
                } else {
                    const uint32_t out = vr.offset(mytok) + 4 * p;
#pragma unroll
                    for (int j = 0; j < 8; ++j) buf_store(vr.rsrc, p + j < a.P ? out + 4 * j : kFar, f[j >> 2][j & 3]);
                }
            }
            __syncthreads();
            // the next slice, this head's or the next one's
            const bool ends_head = p0 + 32 * SL >= a.P;
            const int hn = ends_head ? h + 1 : h, pn = ends_head ? 0 : p0 + 32 * SL;
            if (hn < h1) fetch(hn, pn);
#pragma unroll
            for (int s = 0; s < SL; ++s) {
                const int im = s * 3 * kRow;
                if (mine && p0 + 32 * s < PP) {
                    const f32x4 s0 = __builtin_bit_cast(f32x4, ns[s][0]), s1 = __builtin_bit_cast(f32x4, ns[s][1]);
                    const f32x4 l0 = __builtin_bit_cast(f32x4, nl[s][0]), l1 = __builtin_bit_cast(f32x4, nl[s][1]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) along = fmaf(s0[j], l0[j], fmaf(s1[j], l1[j], along));
                    const Operand<OWN> sb = split8<OWN>(s0, s1), lb = split8<OWN>(l0, l1);
                    if (hn < h1 && pn + 32 * s < PP) fetch_states(hn, pn, s);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        Operand<OWN> m[3];
#pragma unroll
                        for (int e = 0; e < 3; ++e) m[e] = image(im + e * kRow, i, lane);
#pragma unroll
                        for (int q = OWN - 1; q >= 0; --q)
#pragma unroll
                            for (int t = 0; t <= q; ++t) {
                                acc[i][0] = mfma16x16x32(m[0].t[t], sb.t[q - t], acc[i][0]);
                                acc[i][1] = mfma16x16x32(m[1].t[t], lb.t[q - t], acc[i][1]);
                                acc[i][2] = mfma16x16x32(m[2].t[t], sb.t[q - t], acc[i][2]);
                            }
                    }
                } else if (mine && hn < h1 && pn + 32 * s < PP) {
                    // a head's last slice ends before these columns, the next head's first one has them
                    fetch_states(hn, pn, s);
                }
#pragma unroll
                for (int t = 0; t < kJobs; ++t) {
                    const int job = wave + W * t;
                    if (job >= 20) break;
                    const int l = job < 10 ? job : job - 10;
                    x[t] = mm(image(im + (job < 10 ? 0 : 2) * kRow, lower_row(l), lane), image(im + kRow, lower_col(l), lane), x[t]);
                }
            }
        }
        __syncthreads();   // slices read: dP, dM and their transposes take their place
        {
        const int lane = fresh(), g = lane >> 4, l16 = lane & 15;
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
            const double from = sums[j];
            const float bj = gate[2][j];
            const f32x4 bi = *(const f32x4 *)&gate[2][16 * it + 4 * g];
            float v[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 16 * it + 4 * g + r;
                const float decay = expf((float)(sums[i] - from));
                const float w = x[t][r] * bj * (second ? -bi[r] : a.scale);
                v[r] = j < i || (j == i && !second) ? w * decay : 0.f;
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
        }
        __syncthreads();
        if (mine) {
            const int lane = fresh(), g = lane >> 4, l16 = lane & 15;
            const uint32_t to = dqr.offset(4 * g) + 4 * (n0 + l16);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f32x4 up = *(const f32x4 *)&gate[0][16 * i + 4 * g], down = *(const f32x4 *)&gate[1][16 * i + 4 * g];
                const f32x4 beta = *(const f32x4 *)&gate[2][16 * i + 4 * g];
                f32x4 q4 = acc[i][0] * (a.scale * up), rowk = -up * beta * acc[i][2], colk = down * beta * acc[i][1];
                const f32x4 fall = colk;
                // row i's blocks of dP and dM, and column i's, four results at a time
                f32x4 more = zero4();
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const bool low = s < (i < 2 ? 1 : 2), up4 = s >= (i < 2 ? 0 : 1);
                    Operand<OWN> m[4];
                    if (low) {
                        m[0] = image(0, lower_block(i, s), lane);
                        m[1] = image(kImage<OWN>, lower_block(i, s), lane);
                    }
                    if (up4) {
                        m[2] = image(2 * kImage<OWN>, upper_block(i, s), lane);
                        m[3] = image(3 * kImage<OWN>, upper_block(i, s), lane);
                    }
#pragma unroll
                    for (int q = OWN - 1; q >= 0; --q)
#pragma unroll
                        for (int t = 0; t <= q; ++t) {
                            const int u = q - t;
                            if (u >= IN) continue;
                            if (low) {
                                q4 = mfma16x16x32(m[0].t[t], kb[s].t[u], q4);
                                rowk = mfma16x16x32(m[1].t[t], kb[s].t[u], rowk);
                            }
                            if (up4) {
                                colk = mfma16x16x32(m[2].t[t], qb[s].t[u], colk);
                                more = mfma16x16x32(m[3].t[t], kb[s].t[u], more);
                            }
                        }
                }
                colk += more;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float q = value(qb, i, r), k = value(kb, i, r);
                    const float l = group_total<16>(fmaf(q, q4[r], k * (rowk[r] - colk[r])));
                    const float f = group_total<16>(k * fall[r]);
                    if (l16 == 0) {
                        logs[0][wave][16 * i + 4 * g + r] = l;
                        logs[1][wave][16 * i + 4 * g + r] = f;
                    }
                }
                // this lane's sums over the heads so far
                rowk += colk;
                if (h > h0) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        q4[r] += buf_value(dqr.rsrc, to + (16 * i + r) * dqr.step, 0.f);
                        rowk[r] += buf_value(dkr.rsrc, to + (16 * i + r) * dqr.step, 0.f);
                    }
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    buf_store(dqr.rsrc, to + (16 * i + r) * dqr.step, q4[r]);
                    buf_store(dkr.rsrc, to + (16 * i + r) * dqr.step, rowk[r]);
                }
            }
        }
        along = wave_total(along);
        if (lane == 0) ends[wave] = along;
        db += __shfl_xor(db, 16);
        db += __shfl_xor(db, 32);
        if (g == 0) dbs[wave >> 2][16 * (wave & 3) + l16] = db;
        __syncthreads();
        if (wave == 0) {
            // dG of this lane's token; the chunk's end is its last token's, which
            // every token reaches back from (places past it hold zeros)
            float d = 0.f, f = 0.f, dot = 0.f, b = 0.f;
#pragma unroll
            for (int w = 0; w < N / 16; ++w) {
                d += logs[0][w][lane];
                f += logs[1][w][lane];
                dot += ends[w];
            }
#pragma unroll
            for (int w = 0; w < SL; ++w) b += dbs[w][lane];
            // sums from this lane on: within 16 lanes, then the groups behind
            d += __uint_as_float(dpp<0x101>(__float_as_uint(d)));
            d += __uint_as_float(dpp<0x102>(__float_as_uint(d)));
            d += __uint_as_float(dpp<0x104>(__float_as_uint(d)));
            d += __uint_as_float(dpp<0x108>(__float_as_uint(d)));
            auto total = [&](int l) { return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(d), l)); };
            const float t3 = total(48), t2 = total(32) + t3, t1 = total(16) + t2;
            d += g == 0 ? t1 : g == 1 ? t2 : g == 2 ? t3 : 0.f;
            d += wave_total(f) + dot * gate[0][C - 1];
            if (lane < live) {
                const size_t i = (size_t)delta_token(at, a.reverse, first + lane) * a.H + h;
                o.dg[i] = d;
                o.dbeta[i] = b;
            }
        }
    }
}

// dq and dk (blockIdx.y) of a direction (blockIdx.z): the parts' sums. The caller's
// arrays are aligned to their elements.
typedef float f4_a4 __attribute__((ext_vector_type(4), aligned(4)));
__global__ __launch_bounds__(256) void k_delta_parts(GradArgs args) {
    const DeltaGradArgs &o = args.o[blockIdx.z];
    const long long i = 4 * (blockIdx.x * 256LL + threadIdx.x);
    if (i >= args.n) return;
    f4_a4 *to = (f4_a4 *)((blockIdx.y ? o.dk : o.dq) + i);
    f32x4 v = *to;
    for (int p = 1; p < args.parts; ++p) v += *(const f32x4 *)(o.parts + (2 * (p - 1) + blockIdx.y) * args.n + i);
    *to = v;
}

template <typename T>
hipError_t launch_t(const GradArgs &args, int ndir, hipStream_t s) {
    const DeltaArgs &a = args.a[0];
    const dim3 grid((unsigned)(delta_slots(a.units, a.L, a.cu != nullptr) * a.G * args.parts), ndir);
#define GO(n)                                                                                    \
    if (a.N == n) {                                                                              \
        BM_LAUNCH("delta_grad", (k_delta_grad<T, n>), grid, dim3(n == 128 ? 512 : 256), 0, s, args); \
        return hipGetLastError();                                                                \
    }
    GO(16) GO(32) GO(64) GO(128)
#undef GO
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_delta_grad(const DeltaArgs *a, const DeltaGradArgs *o, int ndir, bool bf16, hipStream_t s) {
    const long long n = (a[0].cu ? 1LL : a[0].units) * a[0].L * a[0].G * a[0].N;
    const GradArgs args = {{a[0], a[ndir - 1]}, {o[0], o[ndir - 1]}, grad_parts(a[0]), n};
    const hipError_t e = bf16 ? launch_t<uint16_t>(args, ndir, s) : launch_t<float>(args, ndir, s);
    if (e != hipSuccess || args.parts == 1) return e;
    BM_LAUNCH("delta_parts", k_delta_parts, dim3((unsigned)((n / 4 + 255) / 256), 2, ndir), dim3(256), 0, s, args);
    return hipGetLastError();
}
size_t delta_parts_bytes(const DeltaArgs &a) {
    const size_t tok = a.cu ? (size_t)a.L : (size_t)a.units * a.L;
    return tok ? (size_t)(grad_parts(a) - 1) * 2 * tok * a.G * a.N * 4 : 0;
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
