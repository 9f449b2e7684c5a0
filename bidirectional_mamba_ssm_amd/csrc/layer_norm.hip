// Layer norm of the residual stream in front of a mixer block, and its
// gradient. Per row (token) of C channels:
//   h = x + residual (rounded to the dtype), mu = mean h,
//   var = mean (h - mu)^2, rstd = (var + eps)^-1/2,
//   out = (h - mu) rstd w + b
// and, with xh = (h - mu) rstd, g = dout w, dsum the gradient that reaches h
// along the residual path:
//   dh = rstd (g - mean g - xh mean(g xh)) + dsum
//   dw = sum_rows dout xh,  db = sum_rows dout
// h may be read back from its 8-bit checkpoint (rows.hpp), which the forward
// pass can write as it goes.
//
// Both are streams bounded by HBM. A row lives in the registers of 8, 16, 32
// or 64 lanes of a wave (narrow rows share one) or of several waves of a
// workgroup, NV 16-byte vectors a lane, so every array is read or written once; the next row's loads are under way while a row is
// worked on. Sums over a row are DPP lane moves, and one exchange through LDS
// where it has several waves: the forward pass sends each wave's mean and sum
// of squares about it, which join exactly, so the variance is never a
// difference of large numbers. dw and db are summed in registers over the rows
// a workgroup walks, then over workgroups in a fixed order by a second launch
// (col_sum.hip): no atomics, the same bits every time.
//
// Measured (bf16, residual): 131 072 x 2048 with the checkpoint 464 us, 2.43 GB
// at 5.2 TB/s (a copy of that size moves 4.7); 64 x 2560 3.5 us. The gradient
// from the checkpoint, 8192 x 2048, 24 us (118 MB at 4.9 TB/s) and 4 us for
// the sums; 16 384 x 4096 105 us, 5.1 TB/s. What it took: no element masks in
// the loops (1249 us with them, their flags spilled), 16 elements a lane and
// two waves for 2048 channels (8 and four: 483), two rows a workgroup (16:
// 521); in the gradient 8 waves a workgroup and two workgroups a CU (four
// waves: 35 us; 1024 workgroups: 28 us and 10 us of sums; more workgroups than
// are resident cost a second round).
//
// The last vector of a row whose length is no multiple of it starts at C - V
// instead: it overlaps its neighbour, its first `skip` elements count in no
// sum, and its stores repeat the neighbour's values. No load leaves the row.
#include "internal.hpp"
#include "rows.hpp"

namespace bm {
namespace {

constexpr int kMaxWaves = 8;   // of a row

// Where a lane's vectors lie in a row of C channels shared by `waves` waves:
// vector k starts at channel c[k]. has[k] is false for a lane past the end (it
// reads the row's last vector again). In vector kt (-1: none) some lane's
// first `skip` elements belong to the vector before.
template <int V, int NV>
struct Place {
    int c[NV];
    bool has[NV];
    int kt, skip;
    float count;   // elements of this wave
    __device__ __forceinline__ Place(int C, int t, int lanes) {
        kt = C % V ? C / (V * lanes) : -1;
        skip = 0;
        int n = 0;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int at = (k * lanes + t) * V;
            c[k] = min(at, C - V);
            has[k] = at < C;
            if (at < C && at != c[k]) skip = at - c[k];
            const int first = (k * lanes + (t & ~63)) * V;
            n += max(0, min(64 * V, C - first));
        }
        count = (float)n;
    }
    // v's element j of vector k counts: all do but the overlapped ones
    __device__ __forceinline__ float own(int k, int j, float v) const { return k == kt && j < skip ? 0.f : v; }
};

template <int V>
__device__ __forceinline__ void load_w(const float *p, int c, float none, float *v) {
    if (p) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            const rvec r = *(const u4_a4 *)(p + c + 4 * i);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[4 * i + j] = __uint_as_float(r[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = none;
    }
}

// Lanes of a row: G of a wave, or (G = 0) several waves.
// The forward pass has workgroups of kRows waves, or (G = 0) one row each.
constexpr int kRows = 4;

template <int G>
__device__ __forceinline__ float lanes_total(float v) {
    if constexpr (G == 0 || G == 64) return wave_total(v);
    else return group_total<G>(v);
}

template <typename T, int NV, int G, bool RES, bool CK>
__global__ __launch_bounds__(G == 0 ? 64 * kMaxWaves : 64 * kRows) void k_layer_norm(LnArgs a) {
    using L = Lane<T>;
    constexpr int V = L::V;
    constexpr bool MULTI = G == 0;
    constexpr int kShare = MULTI ? 1 : 64 / G;   // rows of a wave
    __shared__ float2 part[MULTI ? 2 : 1][MULTI ? kMaxWaves : 1];
    const int C = a.C;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t = MULTI ? threadIdx.x : threadIdx.x & (G - 1), lanes = MULTI ? blockDim.x : G;
    const Place<V, NV> at(C, t, lanes);
    const float n = (float)C;
    float w[NV][V], b[NV][V];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        load_w<V>(a.w, at.c[k], 1.f, w[k]);
        load_w<V>(a.b, at.c[k], 0.f, b[k]);
    }
    const long long step = (long long)gridDim.x * (MULTI ? 1 : kRows * kShare);
    long long row = (long long)blockIdx.x * (MULTI ? 1 : kRows * kShare) + (MULTI ? 0 : wave * kShare);
    if (kShare > 1) row += (threadIdx.x & 63) / (MULTI ? 64 : G);
    rvec nx[NV], nr[RES ? NV : 1];
    auto fetch = [&](long long r) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            nx[k] = L::load((const T *)a.x + r * C + at.c[k]);
            if constexpr (RES) nr[k] = L::load((const T *)a.res + r * C + at.c[k]);
        }
    };
    // wider lanes have no registers for it (4096 x 16 384 fp32 with checkpoint
    // 225 us, 316 with the next row ahead and its spills; bf16 132 and 135)
    constexpr bool kAhead = NV * V <= 16;
    if (kAhead && row < a.rows) fetch(row);
    for (int flip = 0; row < a.rows; row += step, flip ^= 1) {
        if (!kAhead) fetch(row);
        rvec r[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            r[k] = nx[k];
            if constexpr (RES) {
                float h[V];
#pragma unroll
                for (int j = 0; j < V; ++j) h[j] = L::get(nx[k], j) + L::get(nr[k], j);
                r[k] = L::pack(h);   // the stream is kept in its dtype, and the norm sees what is kept
            }
        }
        if (kAhead && row + step < a.rows) fetch(row + step);
        float m = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < V; ++j) s += L::get(r[k], j);
            if (k == at.kt) {
                s = 0.f;
#pragma unroll
                for (int j = 0; j < V; ++j) s += at.own(k, j, L::get(r[k], j));
            }
            m += at.has[k] ? s : 0.f;
        }
        // this wave's mean (exact for a constant row whose sum is) and squares about it
        const float cnt = MULTI ? at.count : n;
        float mean = lanes_total<G>(m) / fmaxf(cnt, 1.f);
        float q = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float d = L::get(r[k], j) - mean;
                s = fmaf(d, d, s);
            }
            if (k == at.kt) {
                s = 0.f;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float d = at.own(k, j, L::get(r[k], j) - mean);
                    s = fmaf(d, d, s);
                }
            }
            q += at.has[k] ? s : 0.f;
        }
        q = lanes_total<G>(q);
        if constexpr (MULTI) {
            if ((t & 63) == 0) part[flip][wave] = make_float2(mean, q);
            __syncthreads();
            // lane i takes wave i's share; waves hold 64 V elements of each
            // vector but where the row ends
            const int i = t & 63, nw = lanes >> 6;
            float mi = 0.f, qi = 0.f, ci = 0.f;
            if (i < nw) {
                const float2 p = part[flip][i];
                mi = p.x;
                qi = p.y;
#pragma unroll
                for (int k = 0; k < NV; ++k) ci += (float)max(0, min(64 * V, C - (k * lanes + 64 * i) * V));
            }
            mean = wave_total(ci * mi) / n;
            const float d = mi - mean;
            q = wave_total(fmaf(ci * d, d, qi));
        }
        const float rstd = 1.0f / sqrtf(q / n + a.eps);
        T *out = (T *)a.out + row * C;
        T *sum = (T *)a.sum + row * C;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float h[V], o[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                h[j] = L::get(r[k], j);
                o[j] = fmaf((h[j] - mean) * rstd, w[k][j], b[k][j]);
            }
            const bool ok = at.has[k];
            if (ok) {
                L::store(out + at.c[k], L::pack(o));
                if constexpr (RES) L::store(sum + at.c[k], r[k]);
            }
            if constexpr (CK) {
                uint32_t top = 0;
#pragma unroll
                for (int j = 0; j < V; ++j) top = max(top, abs_bits(h[j]));
                if (k == at.kt) {
                    top = 0;
#pragma unroll
                    for (int j = 0; j < V; ++j) top = max(top, abs_bits(at.own(k, j, h[j])));
                }
                top = block_max<32 / V>(ok ? top : 0u);
                uint32_t code[V];
                act8_codes<V>(h, top, code);
                int8_t *cq = a.q + row * C + at.c[k];
                const int skip = k == at.kt ? at.skip : 0;
                if (ok && skip == 0) {
                    Bytes<V>::store(cq, Bytes<V>::pack(code));
                } else if (ok) {
                    // the overlapped elements may lie in another block
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        if (j >= skip) cq[j] = (int8_t)code[j];
                }
                const int c0 = at.c[k] + skip;
                if (ok && (c0 & 31) == 0) a.scale[row * ((C + 31) / 32) + c0 / 32] = (uint8_t)(top >> 23);
            }
        }
        if (t == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
    }
}

// The gradient's workgroups have kBwdWaves waves at least, so that few of them
// (and few rows of partial sums) fill the chip: R rows at a time of W waves
// each, MULTI if W > 1.
constexpr int kBwdWaves = 8;

template <typename T, int NV, int G, bool Q8, bool DSUM>
__global__ __launch_bounds__(64 * kBwdWaves) void k_layer_norm_bwd(LnBwdArgs a, int W, int R) {
    using L = Lane<T>;
    constexpr int V = L::V, E = V * NV;
    constexpr bool MULTI = G == 0;
    constexpr int kShare = MULTI ? 1 : 64 / G;   // rows of a wave
    __shared__ float2 part[MULTI ? 2 : 1][MULTI ? kBwdWaves : 1];
    // sums to join: W E 64 of dw and of db, where R > 1 (then W <= 4)
    __shared__ float sum[E > 16 ? 1 : MULTI ? 2 * E * 256 : 2 * E * 64];
    const int C = a.C;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int sub = MULTI ? wave / W : wave, lanes = MULTI ? 64 * W : G;
    const int t = MULTI ? threadIdx.x - sub * lanes : threadIdx.x & (G - 1);
    const int slot = sub * kShare + (kShare > 1 ? (threadIdx.x & 63) / (MULTI ? 64 : G) : 0);
    const Place<V, NV> at(C, t, lanes);
    const float inv = 1.0f / (float)C;
    const int nblk = (C + 31) / 32;
    float w[NV][V], dw[NV][V], db[NV][V];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        load_w<V>(a.w, at.c[k], 1.f, w[k]);
#pragma unroll
        for (int j = 0; j < V; ++j) dw[k][j] = db[k][j] = 0.f;
    }
    struct Row {
        rvec g[NV], s[DSUM ? NV : 1], x[Q8 ? 1 : NV];
        typename Bytes<V>::type q[Q8 ? NV : 1];
        uint32_t e[Q8 ? NV : 1];
        float mean, rstd;
    };
    auto fetch = [&](Row &o, long long r) {
        o.mean = a.mean[r];
        o.rstd = a.rstd[r];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            o.g[k] = L::load((const T *)a.dout + r * C + at.c[k]);
            if constexpr (Q8) {
                o.q[k] = Bytes<V>::load((const int8_t *)a.x + r * C + at.c[k]);
                // the block of the lane's own elements; overlapped ones are not used
                o.e[k] = a.xscale[r * nblk + (at.c[k] + (k == at.kt ? at.skip : 0)) / 32];
            } else {
                o.x[k] = L::load((const T *)a.x + r * C + at.c[k]);
            }
            if constexpr (DSUM) o.s[k] = L::load((const T *)a.dsum + r * C + at.c[k]);
        }
    };
    // all waves make the same turns (the barrier); one without a row reads the
    // last one and uses nothing of it
    const long long step = (long long)gridDim.x * R, last = a.rows - 1;
    long long base = (long long)blockIdx.x * R;
    // wider lanes have no registers for it (4096 x 16 384 bf16 from a checkpoint
    // 100 us, 166 with the next row ahead and its spills; from the array 113 and
    // 116; what would gain is the array without dsum at 12 000, 68 and 61)
    constexpr bool kAhead = E <= 16;
    Row next;
    if (kAhead) fetch(next, min(base + slot, last));
    for (int flip = 0; base < a.rows; base += step, flip ^= 1) {
        const long long row = base + slot;
        const bool live = row < a.rows;
        if (!MULTI && !live) break;
        if (!kAhead) fetch(next, min(row, last));
        const Row r = next;
        if (kAhead) fetch(next, min(row + step, last));
        float xh[NV][V];
        float t1 = 0.f, t2 = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if constexpr (Q8) {
                Bytes<V>::values(r.q[k], act8_unit(r.e[k]), xh[k]);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) xh[k][j] = L::get(r.x[k], j);
            }
            float s1 = 0.f, s2 = 0.f;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float d = L::get(r.g[k], j);
                xh[k][j] = (xh[k][j] - r.mean) * r.rstd;
                if (!MULTI || live) {
                    db[k][j] += d;
                    dw[k][j] = fmaf(d, xh[k][j], dw[k][j]);
                }
                const float gw = d * w[k][j];
                s1 += gw;
                s2 = fmaf(gw, xh[k][j], s2);
            }
            if (k == at.kt) {
                s1 = s2 = 0.f;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float gw = at.own(k, j, L::get(r.g[k], j) * w[k][j]);
                    s1 += gw;
                    s2 = fmaf(gw, at.own(k, j, xh[k][j]), s2);
                }
            }
            t1 += at.has[k] ? s1 : 0.f;
            t2 += at.has[k] ? s2 : 0.f;
        }
        t1 = lanes_total<G>(t1);
        t2 = lanes_total<G>(t2);
        if constexpr (MULTI) {
            if ((t & 63) == 0) part[flip][wave] = make_float2(t1, t2);
            __syncthreads();
            t1 = t2 = 0.f;
            for (int i = 0; i < W; ++i) {
                const float2 p = part[flip][sub * W + i];
                t1 += p.x;
                t2 += p.y;
            }
            if (!live) continue;
        }
        const float m1 = t1 * inv, m2 = t2 * inv;
        T *dx = (T *)a.dx + row * C;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float o[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float d = fmaf(-xh[k][j], m2, fmaf(L::get(r.g[k], j), w[k][j], -m1));
                if constexpr (DSUM) o[j] = fmaf(r.rstd, d, L::get(r.s[k], j));
                else o[j] = r.rstd * d;
            }
            if (!at.has[k]) continue;
            const rvec p = L::pack(o);
            const int skip = k == at.kt ? at.skip : 0;
            if (!Q8 || skip == 0) {
                L::store(dx + at.c[k], p);
            } else {
                // an overlapped element was decoded with another block's unit
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    if (j < skip) continue;
                    if constexpr (sizeof(T) == 2) dx[at.c[k] + j] = (T)(p[j >> 1] >> (16 * (j & 1)));
                    else dx[at.c[k] + j] = __uint_as_float(p[j]);
                }
            }
        }
    }
    if (!a.part) return;
    // this workgroup's share of dw | db: the sums of the R rows at a time added in order
    float *out = a.part + (size_t)blockIdx.x * 2 * C;
    if constexpr (kShare > 1) {
        // the rows that share a wave first
#pragma unroll
        for (int off = G; off < 64; off *= 2)
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    dw[k][j] += __shfl_xor(dw[k][j], off);
                    db[k][j] += __shfl_xor(db[k][j], off);
                }
    }
    if constexpr (E <= 16) {
        const int n = R / kShare;   // waves, or (G = 0) rows
        for (int s = 0; s < n && n > 1; ++s) {
            if (sub == s) {
#pragma unroll
                for (int k = 0; k < NV; ++k)
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        float *p = sum + (k * V + j) * lanes + t, *q = p + E * lanes;
                        if (s > 0) {
                            dw[k][j] += *p;
                            db[k][j] += *q;
                        }
                        if (s < n - 1) {
                            *p = dw[k][j];
                            *q = db[k][j];
                        }
                    }
            }
            __syncthreads();
        }
        if (sub != n - 1) return;
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int skip = k == at.kt ? at.skip : 0;
        if (!at.has[k]) continue;
        if (skip == 0) {
#pragma unroll
            for (int i = 0; i < V / 4; ++i) {
                Lane<float>::store(out + at.c[k] + 4 * i, Lane<float>::pack(dw[k] + 4 * i));
                Lane<float>::store(out + C + at.c[k] + 4 * i, Lane<float>::pack(db[k] + 4 * i));
            }
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j >= skip) {
                    out[at.c[k] + j] = dw[k][j];
                    out[C + at.c[k] + j] = db[k][j];
                }
        }
    }
}

// How a row is held: G lanes of one wave or (G = 0) `waves` waves, nv vectors
// a lane. Rows of up to 256 channels take the fewest lanes, 8 elements each
// (kernel times, bf16: 60 000 x 64 5.6 us, with residual and checkpoint 8.9,
// their gradient 12.4; a wave a row 16.8, 26.9 and 21.8; 60 000 x 128 13.3 and
// 16.0 for 27.2 and 23.4); wider ones `lane` elements a lane, or the fewest
// that kMaxWaves waves can do with.
struct Form {
    int nv, waves, G;
};
template <typename T>
Form row_form(int C, int lane) {
    const int V = 16 / (int)sizeof(T);
    Form f;
    f.nv = 1;
    f.waves = 1;
    f.G = 64;
    if (C <= 256) {
        f.nv = 8 / V;
        f.G = C <= 64 ? 8 : C <= 128 ? 16 : 32;
        return f;
    }
    const int units = (C + 64 * V - 1) / (64 * V);          // vectors of a row, in waves
    while (f.nv * V < lane && f.nv < units) f.nv *= 2;
    while (f.nv * kMaxWaves < units) f.nv *= 2;
    f.waves = (units + f.nv - 1) / f.nv;
    if (f.waves > 1) f.G = 0;
    return f;
}
template <typename T>
Form bwd_form(int C) { return row_form<T>(C, 8); }
// rows that a workgroup of the gradient takes at a time
inline int bwd_rows(const Form &f) {
    return f.G ? kBwdWaves * (64 / f.G) : f.waves >= kBwdWaves ? 1 : kBwdWaves / f.waves;
}
template <typename T>
int bwd_wgs(long long rows, int C) {
    const Form f = bwd_form<T>(C);
    // two workgroups of 8 waves a CU, or the one that its registers allow
    const int r = bwd_rows(f), most = f.nv * (16 / (int)sizeof(T)) > 8 ? 256 : 512;
    const long long wgs = (rows + r - 1) / r;
    return (int)(wgs < most ? wgs : most);
}

template <typename T, bool RES, bool CK>
hipError_t launch_fwd(const LnArgs &a, hipStream_t s) {
    const Form f = row_form<T>(a.C, 16);
    const long long per = f.G ? kRows * (64 / f.G) : 1, wgs = (a.rows + per - 1) / per;
    // two turns a workgroup, more only if that leaves too few or makes a grid
    // beyond the largest
    const long long half = (wgs + 1) / 2, most = 1 << 20;
    const dim3 grid((unsigned)(wgs < 2048 ? wgs : half < 2048 ? 2048 : half < most ? half : most));
    const dim3 block(64 * (f.G ? kRows : f.waves));
#define GO(NV, G_)                                                                                          \
    if (f.nv == NV && f.G == G_) {                                                                          \
        BM_LAUNCH("layer_norm", (k_layer_norm<T, NV, G_, RES, CK>), grid, block, 0, s, a);                    \
        return hipGetLastError();                                                                           \
    }
    constexpr int N8 = 8 * sizeof(T) / 16;   // vectors that make 8 elements
    GO(N8, 8) GO(N8, 16) GO(N8, 32)
    GO(N8, 64) GO(2 * N8, 64) GO(2 * N8, 0) GO(4 * N8, 0)
#undef GO
    return hipErrorInvalidValue;
}

template <typename T, bool Q8, bool DSUM>
hipError_t launch_b(const LnBwdArgs &a, hipStream_t s) {
    const Form f = bwd_form<T>(a.C);
    const int R = bwd_rows(f);
    const dim3 grid((unsigned)bwd_wgs<T>(a.rows, a.C)), block(64 * (f.G ? kBwdWaves : f.waves * R));
#define GO(NV, G_)                                                                                       \
    if (f.nv == NV && f.G == G_) {                                                                       \
        BM_LAUNCH("layer_norm_bwd", (k_layer_norm_bwd<T, NV, G_, Q8, DSUM>), grid, block, 0, s, a,         \
                  f.waves, R);                                                                           \
        return hipGetLastError();                                                                        \
    }
    constexpr int N8 = 8 * sizeof(T) / 16;   // vectors that make 8 elements
    GO(N8, 8) GO(N8, 16) GO(N8, 32) GO(N8, 64) GO(N8, 0) GO(2 * N8, 0) GO(4 * N8, 0)
#undef GO
    return hipErrorInvalidValue;
}

template <typename T>
hipError_t launch_fwd_t(const LnArgs &a, hipStream_t s) {
    if (a.res) return a.q ? launch_fwd<T, true, true>(a, s) : launch_fwd<T, true, false>(a, s);
    return a.q ? launch_fwd<T, false, true>(a, s) : launch_fwd<T, false, false>(a, s);
}
template <typename T>
hipError_t launch_b_t(const LnBwdArgs &a, hipStream_t s) {
    if (a.xscale) return a.dsum ? launch_b<T, true, true>(a, s) : launch_b<T, true, false>(a, s);
    return a.dsum ? launch_b<T, false, true>(a, s) : launch_b<T, false, false>(a, s);
}

}  // namespace

hipError_t launch_layer_norm(const LnArgs &a, bool bf16, hipStream_t s) {
    if (a.rows == 0) return hipSuccess;
    return bf16 ? launch_fwd_t<uint16_t>(a, s) : launch_fwd_t<float>(a, s);
}

// workgroups of the gradient: each leaves one row of 2 C partial sums
int layer_norm_bwd_wgs(long long rows, int C, bool bf16) {
    return bf16 ? bwd_wgs<uint16_t>(rows, C) : bwd_wgs<float>(rows, C);
}

hipError_t launch_layer_norm_bwd(const LnBwdArgs &a, bool bf16, hipStream_t s) {
    if (a.rows > 0) {
        hipError_t e = bf16 ? launch_b_t<uint16_t>(a, s) : launch_b_t<float>(a, s);
        if (e != hipSuccess) return e;
    }
    if (!a.dw && !a.db) return hipSuccess;
    const ColSum c{a.part, layer_norm_bwd_wgs(a.rows, a.C, bf16), a.C, 1, 1, a.dw, a.db};
    return launch_col_sum(&c, 1, s);
}

}  // namespace bm
