// kda_attn.hip -- softmax attention of packed new tokens over a paged 8-bit
// key/value cache.
//
// For new token i of a sequence (position p) and query head h, with the cached
// tokens j that the mask leaves (j <= p when causal, j > p - window with a
// window, j < kv_len, their page present):
//     s_j = scale q.k_j,  o = sum_j e^{s_j} v_j / sum_j e^{s_j},  lse = log sum_j e^{s_j}
// in one pass over the keys, with a running maximum m, sum l and output that
// are scaled by 2^(m_old - m_new) when the maximum grows (scores in the log2
// domain).  No keys left: o = 0, lse = -inf.
//
// Products on the matrix cores.  A code times its page's power-of-two scale is
// exact in bf16, so K and V enter as the values they stand for; bf16 queries
// are exact as well, and the only rounding of operands is that of the
// probabilities to bf16 (half an ulp, 2^-9 relative, independent per key).
// With fp32 rows, queries and probabilities enter as three bf16 terms each
// (8 + 8 + 8 bits hold the 24 of fp32), three products instead of one.
//
// Both products are formed transposed, S^T = K Q^T and O^T = V^T P^T, which
// keeps a query row in one lane column throughout: in the result layout of
// S^T (column = row of Q, 4 consecutive tokens per lane group) a lane already
// holds the slots that it supplies to P^T, with the contraction index numbered
// as the layout has it, so no value crosses lanes between the two products.
// V is read row by row (8 bytes: 8 dims of one token); byte permutes pair two
// tokens of a dim before the conversion to bf16.  The dims of V are numbered
// so that a lane's 8 bytes serve the 8 products of its column.

#include <algorithm>

#include "kda_attn_ops.h"

namespace kda {
namespace {

using namespace attn;

constexpr int kShortRows = 64;        // most query rows of a sequence that this kernel takes
constexpr int kSmallCall = 1024;      // query rows of a call that it takes alone
constexpr int kMinShare = 4;          // fewest tiles worth a workgroup of their own

template <int D> struct Codes {
    u32x4 k[4][D / 64];      // 4 groups of 16 tokens: 16 bytes of the lane's token each
    uint32_t v[4][4][D / 64];   // 4 groups, 4 tokens: D / 16 bytes each
    float ks[4], vs[4];
    int ok;                  // groups with a page
};

template <int D>
__device__ __forceinline__ void load_tile(const AttnArgs &a, const Seq &s, int n, int hk, int64_t kb,
                                          int lane, Codes<D> &c) {
    const int col = lane & 15, kg = lane >> 4;
    c.ok = 0;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const int64_t at = kb + 16 * g;
        int pid = -1;
        if (at < s.kvl) pid = a.kv.table[(int64_t)n * a.kv.width + at / a.kv.page];
        pid = __builtin_amdgcn_readfirstlane(pid);
        c.ks[g] = c.vs[g] = 1.f;
        if (pid >= 0 && pid < a.kv.n_pages) {
            c.ok |= 1 << g;
            const int64_t ph = (int64_t)pid * a.kv.Hk + hk;
            const int64_t base = (ph * a.kv.page + at % a.kv.page) * D;
            const uint8_t *kp = a.kv.k_codes + base + col * D + kg * 16;
            const uint8_t *vp = a.kv.v_codes + base + (4 * kg) * D + col * (D / 16);
#pragma unroll
            for (int i = 0; i < D / 64; ++i) c.k[g][i] = *(const u32x4 *)(kp + 64 * i);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (D == 128) {
                    const uint2 w = *(const uint2 *)(vp + i * D);
                    c.v[g][i][0] = w.x;
                    c.v[g][i][1] = w.y;
                } else {
                    c.v[g][i][0] = *(const uint32_t *)(vp + i * D);
                }
            }
            c.ks[g] = a.kv.k_scale[ph];
            c.vs[g] = a.kv.v_scale[ph];
        } else {
#pragma unroll
            for (int i = 0; i < D / 64; ++i) c.k[g][i] = u32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < D / 64; ++j) c.v[g][i][j] = 0;
        }
    }
}

// O^T += V^T P^T for one pair of token groups
template <int D, int NS>
__device__ __forceinline__ void add_pv(const uint32_t (&v0)[4][D / 64], const uint32_t (&v1)[4][D / 64],
                                       float s0, float s1, const Frag<NS> &p, f32x4 *o) {
#pragma unroll
    for (int w = 0; w < D / 64; ++w) {
        const uint32_t t[8] = {v0[0][w], v0[1][w], v0[2][w], v0[3][w],
                               v1[0][w], v1[1][w], v1[2][w], v1[3][w]};
        const bf16x8 f[4] = {v_frag<0>(t, s0, s1), v_frag<1>(t, s0, s1), v_frag<2>(t, s0, s1),
                             v_frag<3>(t, s0, s1)};
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int i = 0; i < NS; ++i)
                o[4 * w + b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[b], p.f[i], o[4 * w + b], 0, 0, 0);
    }
}

// Where every wave's share of a unit meets: D + 2 floats per row and wave.
template <int D> struct Meet {
    float o[kWaves][kRows][D + 4];
    float m[kWaves][kRows], l[kWaves][kRows];
};

// BF: bf16 rows.  One workgroup takes a contiguous share of all (unit, tile)
// pairs, or, with workers = 0, one unit; its waves take the tiles of a unit in
// turn and meet in LDS at the unit's end.
template <int D, bool BF>
__global__ __launch_bounds__(kAttnThreads) void attn_kernel(const AttnArgs a) {
    constexpr int NS = BF ? 1 : 3;
    constexpr int NF = D / 32;                 // contraction steps of Q K^T
    constexpr int NT = D / 16;                 // 16-dim blocks of O
    __shared__ Meet<D> sm;
    __shared__ int64_t s_scan[kWaves];
    __shared__ int64_t s_base;
    __shared__ int s_n;

    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int col = lane & 15, kg = lane >> 4;
    const int G = a.Hq / a.kv.Hk;
    const int N = a.kv.N;

    // this workgroup's share [from, to) of the tiles of all units; n0: the
    // sequence that holds `from`, base: the tiles before that sequence
    int64_t from, to, base = 0;
    int n = 0;
    if (a.workers == 0) {
        // units are numbered like the packed rows: first(n) = cu[n] G / kRows + n
        const int64_t x = blockIdx.x / a.kv.Hk;
        int lo = 0, hi = N - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (a.kv.cu[mid] * G / kRows + mid <= x) lo = mid; else hi = mid - 1;
        }
        n = lo;
        const Seq s = sequence(a, n, G);
        const int64_t r = x - (s.c0 * G / kRows + n);
        if (r < 0 || r >= s.rt) return;
        from = ((int64_t)(blockIdx.x % a.kv.Hk) * s.rt + r) * s.tiles;
        to = from + s.tiles;
    } else {
        // total, then the sequence in which the share starts
        int64_t total = 0;
        for (int n0 = 0; n0 < N; n0 += kAttnThreads) {
            int64_t c = 0;
            if (n0 + tid < N) {
                const Seq s = sequence(a, n0 + tid, G);
                c = (int64_t)a.kv.Hk * s.rt * s.tiles;
            }
#pragma unroll
            for (int off = 32; off >= 1; off >>= 1) c += __shfl_xor(c, off);
            if (lane == 0) s_scan[w] = c;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kWaves; ++i) total += s_scan[i];
            __syncthreads();
        }
        const int64_t share = max((total + a.workers - 1) / a.workers, (int64_t)kMinShare);
        from = share * blockIdx.x;
        to = min(from + share, total);
        if (from >= to) return;
        int64_t before = 0;
        for (int n0 = 0; n0 < N; n0 += kAttnThreads) {
            int64_t c = 0;
            if (n0 + tid < N) {
                const Seq s = sequence(a, n0 + tid, G);
                c = (int64_t)a.kv.Hk * s.rt * s.tiles;
            }
            int64_t inc = c;
#pragma unroll
            for (int off = 1; off < 64; off <<= 1) {
                const int64_t y = __shfl_up(inc, off);
                if (lane >= off) inc += y;
            }
            if (lane == 63) s_scan[w] = inc;
            __syncthreads();
            for (int i = 0; i < kWaves; ++i) {
                if (i < w) inc += s_scan[i];
            }
            inc += before;
            if (inc - c <= from && from < inc) {
                s_n = n0 + tid;
                s_base = inc - c;
            }
            for (int i = 0; i < kWaves; ++i) before += s_scan[i];
            __syncthreads();
            if (before > from) break;
        }
        n = s_n;
        base = s_base;
    }

    for (int64_t at = from; at < to; ++n) {
        const Seq s = sequence(a, n, G);
        const int64_t end = base + (int64_t)a.kv.Hk * s.rt * s.tiles;   // of this sequence
        while (at < to && at < end) {
            const int64_t rel = at - base;
            const int unit = (int)(rel / s.tiles);
            const int64_t ubase = base + (int64_t)unit * s.tiles;
            const int t_lo = s.lo + (int)(at - ubase);
            const int64_t uend = ubase + s.tiles;
            const int t_hi = s.lo + (int)(min(uend, to) - ubase);
            const int hk = unit / s.rt, rb = unit % s.rt;
            const bool whole = ubase >= from && uend <= to;

            // the lane's query row and the keys it sees
            const int R = rb * kRows + col;
            const int tok = min(R / G, s.len - 1), gh = R % G;
            const bool live = R < s.len * G;
            const int64_t pos = s.pos0 + tok;
            const int64_t vis_hi = live ? (a.causal ? min(pos + 1, s.kvl) : s.kvl) : 0;
            const int64_t vis_lo = a.window > 0 ? pos - a.window + 1 : 0;
            Frag<NS> q[NF];
            {
                const int64_t qi = (s.c0 + tok) * a.q_row + (int64_t)(hk * G + gh) * D;
#pragma unroll
                for (int f = 0; f < NF; ++f) {
                    float x[8];
                    mf::IO<BF>::load8(a.q, qi + (f >> 1) * 64 + kg * 16 + (f & 1) * 8, x);
                    q[f] = split8<NS>(x);
                }
            }
            // tiles that some row of the unit sees
            const int tok_last = min((rb * kRows + kRows - 1) / G, s.len - 1);
            const int64_t seen = a.causal ? min(s.pos0 + tok_last + 1, s.kvl) : s.kvl;
            const int64_t all_lo = a.window > 0 ? s.pos0 + tok_last - a.window + 1 : 0;
            const int64_t all_hi = a.causal ? min(s.pos0 + rb * kRows / G + 1, s.kvl) : s.kvl;
            const int t_end = min(t_hi, (int)((max(seen, (int64_t)0) + kTile - 1) / kTile));
            const int64_t first = a.window > 0 ? max(s.pos0 + rb * kRows / G - a.window + 1, (int64_t)0) : 0;
            const int t_beg = max(t_lo, (int)min(first / kTile, (int64_t)INT32_MAX / 2));

            float m = -__builtin_inff(), l = 0.f;
            f32x4 o[NT];
#pragma unroll
            for (int i = 0; i < NT; ++i) o[i] = f32x4{0.f, 0.f, 0.f, 0.f};

            for (int t = t_beg + w; t < t_end; t += kWaves) {
                const int64_t kb = (int64_t)t * kTile;
                Codes<D> c;
                load_tile<D>(a, s, n, hk, kb, lane, c);
                f32x4 sc[4];
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    sc[g] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int f = 0; f < NF; ++f) {
                        const u32x4 x = c.k[g][f >> 1];
                        const uint32_t c0 = (f & 1) ? x[2] : x[0], c1 = (f & 1) ? x[3] : x[1];
                        u32x4 kf;
                        kf[0] = widen<false>(c0, c.ks[g]);
                        kf[1] = widen<true>(c0, c.ks[g]);
                        kf[2] = widen<false>(c1, c.ks[g]);
                        kf[3] = widen<true>(c1, c.ks[g]);
#pragma unroll
                        for (int i = 0; i < NS; ++i)
                            sc[g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                __builtin_bit_cast(bf16x8, kf), q[f].f[i], sc[g], 0, 0, 0);
                    }
                }
                const bool full = c.ok == 15 && kb >= all_lo && kb + kTile <= all_hi;
                float tm = -__builtin_inff();
                bool sees[16];
#pragma unroll
                for (int g = 0; g < 4; ++g)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float x = sc[g][i] * a.scale;
                        if (!full) {
                            const int64_t j = kb + 16 * g + 4 * kg + i;
                            const bool y = j >= vis_lo && j < vis_hi && (c.ok >> g & 1);
                            sees[4 * g + i] = y;
                            x = y ? x : -__builtin_inff();
                        }
                        sc[g][i] = x;
                        tm = fmaxf(tm, x);
                    }
                tm = fmaxf(tm, __shfl_xor(tm, 16));
                tm = fmaxf(tm, __shfl_xor(tm, 32));
                const float mn = fmaxf(m, tm);
                const float ms = mn == -__builtin_inff() ? 0.f : mn;
                const float alpha = mf::ex2(m - ms);
                m = mn;
                float p[16], ps = 0.f;
#pragma unroll
                for (int g = 0; g < 4; ++g)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float y = mf::ex2(sc[g][i] - ms);
                        p[4 * g + i] = y;
                        ps += y;
                    }
                l = l * alpha + ps;
#pragma unroll
                for (int i = 0; i < NT; ++i) o[i] *= alpha;

                if (!full) {
                    // A NaN among the values reaches only the rows that see it: the
                    // products take zeros in its place, and 1 x (row sees it) counts it.
                    uint32_t any = 0;
#pragma unroll
                    for (int g = 0; g < 4; ++g)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int j = 0; j < D / 64; ++j) any |= nan_bytes(c.v[g][i][j]);
                    if (__ballot(any != 0) != 0) {
                        f32x4 cnt[NT];
#pragma unroll
                        for (int i = 0; i < NT; ++i) cnt[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int g = 0; g < 4; g += 2) {
                            uint32_t one[2][4][D / 64];
                            float vis[8];
#pragma unroll
                            for (int h = 0; h < 2; ++h)
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    vis[4 * h + i] = sees[4 * (g + h) + i] ? 1.f : 0.f;
#pragma unroll
                                    for (int j = 0; j < D / 64; ++j) {
                                        uint32_t &x = c.v[g + h][i][j];
                                        const uint32_t b = nan_bytes(x) >> 7;     // 1 per NaN byte
                                        one[h][i][j] = b * 0x38u;                 // the code of 1.0
                                        x &= ~(b * 0xffu);
                                    }
                                }
                            add_pv<D, 1>(one[0], one[1], 1.f, 1.f, split8<1>(vis), cnt);
                        }
#pragma unroll
                        for (int i = 0; i < NT; ++i)
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                if (cnt[i][j] > 0.f) o[i][j] = __builtin_nanf("");
                    }
                }
#pragma unroll
                for (int g = 0; g < 4; g += 2)
                    add_pv<D, NS>(c.v[g], c.v[g + 1], c.vs[g], c.vs[g + 1], split8<NS>(p + 4 * g), o);
            }

            // the waves meet
            l += __shfl_xor(l, 16);
            l += __shfl_xor(l, 32);
            if (kg == 0) { sm.m[w][col] = m; sm.l[w][col] = l; }
#pragma unroll
            for (int i = 0; i < 4; ++i)       // dims (D / 16)(4 kg + i) + j, j < NT
#pragma unroll
                for (int j = 0; j < NT; j += 4)
                    *(f32x4 *)&sm.o[w][col][NT * (4 * kg + i) + j] =
                        f32x4{o[j][i], o[j + 1][i], o[j + 2][i], o[j + 3][i]};
            __syncthreads();
            {
                constexpr int E = kRows * D / kAttnThreads;      // 8 or 4 dims per thread
                const int r = tid / (D / E), d = (tid % (D / E)) * E;
                float M = -__builtin_inff();
#pragma unroll
                for (int i = 0; i < kWaves; ++i) M = fmaxf(M, sm.m[i][r]);
                const float Ms = M == -__builtin_inff() ? 0.f : M;
                float L = 0.f, y[E];
#pragma unroll
                for (int j = 0; j < E; ++j) y[j] = 0.f;
#pragma unroll
                for (int i = 0; i < kWaves; ++i) {
                    const float f = mf::ex2(sm.m[i][r] - Ms);
                    L += f * sm.l[i][r];
#pragma unroll
                    for (int j = 0; j < E; ++j) y[j] += f * sm.o[i][r][d + j];
                }
                const int RR = rb * kRows + r;
                if (whole) {
                    if (RR < s.len * G) {
                        const int64_t row = (s.c0 + RR / G) * a.Hq + hk * G + RR % G;
                        const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
                        for (int j = 0; j < E; ++j) {
                            const float z = y[j] * inv;
                            if (BF) ((bf16_t *)a.o)[row * D + d + j] = (bf16_t)z;
                            else ((float *)a.o)[row * D + d + j] = z;
                        }
                        if (a.lse && d == 0)
                            a.lse[row] = L == 0.f ? -__builtin_inff() : (M + __builtin_amdgcn_logf(L)) * kLn2;
                    }
                } else {
                    // cut at this workgroup's end: its second slot; at its start: the first
                    float *dst = a.part + (2 * (int64_t)blockIdx.x + (ubase >= from ? 1 : 0)) * (kRows * (D + 2));
#pragma unroll
                    for (int j = 0; j < E; ++j) dst[r * D + d + j] = y[j];
                    if (d == 0) { dst[kRows * D + r] = M; dst[kRows * D + kRows + r] = L; }
                }
            }
            __syncthreads();
            at = uend;
        }
        base = end;
    }
}

// Joins the parts of every unit that attn_kernel cut: one workgroup per unit.
template <int D, bool BF>
__global__ __launch_bounds__(kAttnThreads) void join_kernel(const AttnArgs a) {
    __shared__ int64_t s_scan[2][kWaves];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int G = a.Hq / a.kv.Hk, N = a.kv.N;
    const int64_t x = blockIdx.x / a.kv.Hk;
    int lo = 0, hi = N - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.kv.cu[mid] * G / kRows + mid <= x) lo = mid; else hi = mid - 1;
    }
    const int n = lo;
    const Seq s = sequence(a, n, G);
    const int64_t rb = x - (s.c0 * G / kRows + n);
    if (rb < 0 || rb >= s.rt) return;
    const int hk = blockIdx.x % a.kv.Hk;
    int64_t total = 0, base = 0;
    for (int n0 = 0; n0 < N; n0 += kAttnThreads) {
        int64_t c = 0;
        if (n0 + tid < N) {
            const Seq y = sequence(a, n0 + tid, G);
            c = (int64_t)a.kv.Hk * y.rt * y.tiles;
        }
        int64_t b = n0 + tid < n ? c : 0;
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) {
            c += __shfl_xor(c, off);
            b += __shfl_xor(b, off);
        }
        if (lane == 0) { s_scan[0][w] = c; s_scan[1][w] = b; }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kWaves; ++i) { total += s_scan[0][i]; base += s_scan[1][i]; }
        __syncthreads();
    }
    const int64_t share = max((total + a.workers - 1) / a.workers, (int64_t)kMinShare);
    const int64_t ubase = base + ((int64_t)hk * s.rt + rb) * s.tiles;
    const int64_t w0 = ubase / share, w1 = (ubase + s.tiles - 1) / share;
    if (w0 == w1) return;                     // written whole
    constexpr int E = kRows * D / kAttnThreads;
    const int r = tid / (D / E), d = (tid % (D / E)) * E;
    const int64_t R = rb * kRows + r;
    if (R >= (int64_t)s.len * G) return;
    float M = -__builtin_inff(), L = 0.f, y[E];
#pragma unroll
    for (int j = 0; j < E; ++j) y[j] = 0.f;
    for (int64_t i = w0; i <= w1; ++i) {
        const float *src = a.part + (2 * i + (ubase >= i * share ? 1 : 0)) * (kRows * (D + 2));
        const float m = src[kRows * D + r], l = src[kRows * D + kRows + r];
        const float mn = fmaxf(M, m), ms = mn == -__builtin_inff() ? 0.f : mn;
        const float f0 = mf::ex2(M - ms), f1 = mf::ex2(m - ms);
        M = mn;
        L = L * f0 + l * f1;
#pragma unroll
        for (int j = 0; j < E; ++j) y[j] = y[j] * f0 + src[r * D + d + j] * f1;
    }
    const int64_t row = (s.c0 + R / G) * a.Hq + hk * G + R % G;
    const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
    for (int j = 0; j < E; ++j) {
        const float z = y[j] * inv;
        if (BF) ((bf16_t *)a.o)[row * D + d + j] = (bf16_t)z;
        else ((float *)a.o)[row * D + d + j] = z;
    }
    if (a.lse && d == 0)
        a.lse[row] = L == 0.f ? -__builtin_inff() : (M + __builtin_amdgcn_logf(L)) * kLn2;
}

template <int D, bool BF>
hipError_t launch(const AttnArgs &a, hipStream_t s) {
    const int G = a.Hq / a.kv.Hk;
    // units over all sequences: at most first(N) of them per kv head
    const int64_t units = (a.kv.T * G / kRows + a.kv.N) * a.kv.Hk;
    if (units > INT32_MAX) return hipErrorInvalidValue;
    const dim3 block(kAttnThreads);
    hipLaunchKernelGGL((attn_kernel<D, BF>), dim3((unsigned)(a.workers ? a.workers : units)), block, 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.workers == 0) return e;
    hipLaunchKernelGGL((join_kernel<D, BF>), dim3((unsigned)units), block, 0, s, a);
    return hipGetLastError();
}

}  // namespace

void attn_plan(int cus, int N, int64_t T, int Hq, int Hk, int64_t max_kv, AttnArgs *a) {
    const int G = Hq / Hk;
    const int64_t rows = T * G;
    a->workers = -1;
    a->row_units = 0;
    a->row_splits = 1;
    // A single sequence and small calls are of one kind; in others the lengths,
    // which only the device knows, decide sequence by sequence.
    const bool all_short = rows <= kShortRows || (N > 1 && rows <= kSmallCall);
    const bool all_long = N == 1 && !all_short;
    a->short_rows = all_short ? INT32_MAX : kShortRows;
    if (!all_long) a->workers = max_kv <= 8 * kTile ? 0 : 2 * cus;
    if (!all_short) {
        a->row_units = (int32_t)(rows / kRowTile + N);
        const int64_t units = (int64_t)a->row_units * Hk;
        if (units < 2 * cus) {
            const int64_t want = (4 * (int64_t)cus + units - 1) / units;
            a->row_splits = (int32_t)std::max<int64_t>(1, std::min<int64_t>({want, 16, max_kv / 1024}));
        }
    }
}

size_t attn_partial_bytes(int D, const AttnArgs &a) {
    const size_t one = a.workers > 0 ? (size_t)a.workers * 2 * kRows * (D + 2) : 0;
    const size_t rows = a.row_splits > 1 ? (size_t)a.row_units * a.kv.Hk * a.row_splits * kRowTile * (D + 2) : 0;
    return std::max(one, rows) * sizeof(float);
}

hipError_t launch_attn(bool bf16, int D, const AttnArgs &a, hipStream_t s) {
    if (D == 128) return bf16 ? launch<128, true>(a, s) : launch<128, false>(a, s);
    if (D == 64) return bf16 ? launch<64, true>(a, s) : launch<64, false>(a, s);
    return hipErrorInvalidValue;
}

}  // namespace kda
