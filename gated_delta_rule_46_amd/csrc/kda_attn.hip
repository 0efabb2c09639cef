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
// probabilities to bf16 (at most 2^-8 of each, to either side; outputs, 0.0017 off the
// exact ones by their own rounding, are 0.0018 off for one token over 257 keys and 0.0020
// to 0.0021 for prompts, relative in the 2-norm, where a second term would cost half as
// many matrix products again).
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
//
// Bound by reading the codes once: 64 sequences of 512 to 32,768 tokens, one new one each,
// at 32 / 8 heads of 128 with bf16 rows 231 us (5.5 TB/s; reads of shuffled 8 KiB pages
// alone reach 6.8), 131,072 keys 62 us (4.3), 257 keys 10.6 (one chain of memory latencies).
// Hence all of the card on any mix of lengths (shares of equal steps, joined after), loads
// of one step ahead without a branch, and few registers, for three waves per SIMD.

#include <algorithm>

#include "kda_attn_ops.h"

namespace kda {
namespace {

using namespace attn;

// Which kernel: units of 16 or 32 rows read their keys once each, units of 128 rows (kda_attn_rows.hip)
// less often, but they start later and wait for their tiles.  us per call at 32 / 8 heads of 128, here /
// there, sequences x keys x rows per kv head: bf16 64 x 8,000 x 20 184 / 416, x 32 185 / 273, x 64
// 366 / 432; 8 x 8,000 x 20 46 / 67, x 64 67 / 76; 1 x 100,000 x 32 55 / 96; fp32 64 x 8,000 x 32
// 365 / 747, x 64 750 / 1,121; 8 x 8,000 x 64 110 / 152, x 128 195 / 136.
constexpr int kShortRows = 64;        // most query rows of a sequence that come here ...
// ... unless all units x keys are no more than this: 1 x 2,000 x 128 with bf16 rows 18 / 21, 4 x 2,000 x 128
// 32 / 36, 1 x 4,000 x 256 39 / 31; with fp32 rows 3 x 3,000 x 140 46 / 76, 1 x 1,000 x 1,024 23 / 42; with
// heads of 64 and bf16 rows 3 x 1,900 x 140 16 / 24, 1 x 1,000 x 1,024 14 / 22.
static int64_t small_call(bool bf16, int D) { return bf16 && D == 128 ? 1 << 18 : 1 << 20; }
// Rows of a unit: 32 where a sequence has more than 16 (bf16 64 x 8,000 x 20 185 us in units of 32, 378 in
// units of 16; x 64 366 / 720).  In a small call 16, which are twice as many workgroups (6 x 500 x 32 13.1 / 12.3), and with
// fp32 rows, whose three terms for two blocks of rows would not fit a wave's registers at two waves per SIMD.

// One workgroup per unit, without parts and their launch, up to this many keys, twice as
// many from 64 units on.  us per call, unit by unit / in shares, head_dim 128: 1 sequence
// of 1,000 keys at 1 kv head 10.7 / 11.8, 64 at 8 heads 36 / 46; of 2,000 keys 18.7 / 12.1
// and 64 / 69; of 4,000 28 / 12 and 119 / 115.
constexpr int kDirect = 1024;
constexpr int kMinShare = 8;          // fewest steps worth a workgroup of their own (two per wave)

// A step's codes in a wave's registers, as the products read them.
template <int D> struct Codes {
    u32x4 k[2][D / 64];         // 2 groups of 16 tokens: 16 bytes of the lane's token each
    uint32_t v[2][4][D / 64];   // 2 groups, 4 tokens: D / 16 bytes each
    float scale;                // lane 2 x + g: the group's scale of keys (x = 0), values (1)
    int ok;                     // groups with a page
};

// The pages of a wave's next steps.  Memory answers vector loads in order, so a step's
// lookup is issued before the codes of the step ahead of it, and waiting for it leaves
// those codes in flight.  (Scalar loads would not do: any wait for one is a wait for
// all, the lookups on their way among them.)
struct Lookup {
    const int32_t *table;
    int shift, kvl, page;       // page: lanes 0..31 and 32..63 hold group 0's and 1's

    __device__ __forceinline__ void ask(int t, int lane) {
        const int at = min(t * kStep + 16 * (lane >> 5), kvl - 1);
        page = __builtin_nontemporal_load(table + (at >> shift));
    }
};

// kvl > 0.  Groups without a page (or behind the last key) read page 0 and are masked.
template <int D>
__device__ __forceinline__ void load_step(const AttnArgs &a, const Lookup &pg, int hk, int t, int lane, Codes<D> &c) {
    const int col = lane & 15, kg = lane >> 4;
    int64_t ph[2];
    c.ok = 0;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        int pid = __builtin_amdgcn_readlane(pg.page, 32 * g);
        const bool ok = pid >= 0 && pid < a.kv.n_pages && t * kStep + 16 * g < pg.kvl;
        c.ok |= ok << g;
        pid = ok ? pid : 0;
        ph[g] = (int64_t)pid * a.kv.Hk + hk;
        const int64_t base = (ph[g] * a.kv.page + ((t * kStep + 16 * g) & (a.kv.page - 1))) * D;
        const uint8_t *kp = a.kv.k_codes + base, *vp = a.kv.v_codes + base;
        const uint32_t ko = col * D + kg * 16, vo = 4 * kg * D + col * (D / 16);
#pragma unroll
        for (int i = 0; i < D / 64; ++i) c.k[g][i] = __builtin_nontemporal_load((const u32x4 *)(kp + ko + 64 * i));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (D == 128) {
                const u32x2 w = __builtin_nontemporal_load((const u32x2 *)(vp + vo + i * D));
                c.v[g][i][0] = w[0];
                c.v[g][i][1] = w[1];
            } else {
                c.v[g][i][0] = __builtin_nontemporal_load((const uint32_t *)(vp + vo + i * D));
            }
        }
    }
    c.scale = ((lane & 2) ? a.kv.v_scale : a.kv.k_scale)[(lane & 1) ? ph[1] : ph[0]];
}

// O^T += V^T P^T for one pair of token groups
template <int D, int NS, int RB>
__device__ __forceinline__ void add_pv(const uint32_t (&v0)[4][D / 64], const uint32_t (&v1)[4][D / 64],
                                       float s0, float s1, const Frag<NS> (&p)[RB], f32x4 (&o)[RB][D / 16]) {
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
#pragma unroll
                for (int r = 0; r < RB; ++r)
                    o[r][4 * w + b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[b], p[r].f[i], o[r][4 * w + b], 0, 0, 0);
    }
}

// Steps per workgroup when `workers` of them share all.
__device__ __forceinline__ int64_t share_of(int64_t total, int workers) {
    return max((total + workers - 1) / workers, (int64_t)kMinShare);
}

// x / y, the usual case in 32 bits
__device__ __forceinline__ uint32_t quotient(int64_t x, int y) {
    return x >> 32 ? (uint32_t)(x / y) : (uint32_t)x / (uint32_t)y;
}

// Where every wave's share of a unit meets: D + 2 floats per row and wave.
template <int D, int RB> struct Meet {
    float o[kWaves][kRows * RB][D + 4];
    float m[kWaves][kRows * RB], l[kWaves][kRows * RB];
};

// The lane's query rows of a unit (16 apart) and the keys they see.
template <int D, int NS, int RB> struct Rows {
    Frag<NS> q[RB][D / 32];
    int lo[RB], num[RB];      // keys lo <= j < lo + num
    int all_lo, all_hi;       // keys that every row of the unit sees

    // end: the keys from there on are another share's
    __device__ void load(const AttnArgs &a, const Seq &s, int rb, int hk, int G, int end, int lane) {
        constexpr int UR = kRows * RB;
        const int kg = lane >> 4;
#pragma unroll
        for (int b = 0; b < RB; ++b) {
            const int R = rb * UR + kRows * b + (lane & 15);
            const int tok = min(R / G, s.len - 1), gh = R % G;
            const int64_t qi = (s.c0 + tok) * a.q_row + (int64_t)(hk * G + gh) * D;
#pragma unroll
            for (int f = 0; f < D / 32; ++f) {
                float x[8];
                mf::IO<NS == 1>::load8(a.q, qi + (f >> 1) * 64 + kg * 16 + (f & 1) * 8, x);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] *= a.q_sign;     // exact
                q[b][f] = split_query8<NS>(x);
            }
            lo[b] = s.begin_of(a, tok);
            num[b] = R < s.len * G ? max(min(s.end_of(a, tok), end) - lo[b], 0) : 0;
        }
        // The loads end here: were they still on their way at the loop's first entry, its
        // waits would count them in every pass.
#pragma unroll
        for (int b = 0; b < RB; ++b)
#pragma unroll
            for (int f = 0; f < D / 32; ++f)
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    u32x4 x = __builtin_bit_cast(u32x4, q[b][f].f[i]);
                    asm volatile("" : "+v"(x));
                    q[b][f].f[i] = __builtin_bit_cast(bf16x8, x);
                }
        const int t0 = rb * UR / G, t1 = min((rb * UR + UR - 1) / G, s.len - 1);
        all_hi = min(s.end_of(a, t0), end);
        all_lo = s.begin_of(a, t1);
    }
};

// One step of 32 keys for the rows of a unit.  True: values that were NaN are left out,
// see_nans() is to follow.
template <int D, int NS, int RB>
__device__ __forceinline__ bool one_step(const Rows<D, NS, RB> &row, Codes<D> &c, int t, float scale, int lane,
                                          float (&m)[RB], float (&l)[RB], f32x4 (&o)[RB][D / 16]) {
    constexpr int NT = D / 16;
    const int kg = lane >> 4, kb = t * kStep;
    const uint32_t sv = f32_bits(c.ok >> (lane & 1) & 1 ? c.scale : 1.f);
    float ks[2], vs[2];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        ks[g] = bits_f32(__builtin_amdgcn_readlane(sv, g));
        vs[g] = bits_f32(__builtin_amdgcn_readlane(sv, 2 + g));
    }
    f32x4 sc[RB][2];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
#pragma unroll
        for (int b = 0; b < RB; ++b) sc[b][g] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int f = 0; f < D / 32; ++f) {
            const u32x4 x = c.k[g][f >> 1];
            const uint32_t c0 = (f & 1) ? x[2] : x[0], c1 = (f & 1) ? x[3] : x[1];
            u32x4 kf;
            kf[0] = widen<false>(c0, ks[g]);
            kf[1] = widen<true>(c0, ks[g]);
            kf[2] = widen<false>(c1, ks[g]);
            kf[3] = widen<true>(c1, ks[g]);
#pragma unroll
            for (int i = 0; i < NS; ++i)
#pragma unroll
                for (int b = 0; b < RB; ++b)
                    sc[b][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, kf),
                                                                       row.q[b][f].f[i], sc[b][g], 0, 0, 0);
        }
    }
    const bool full = c.ok == 3 && kb >= row.all_lo && kb + kStep <= row.all_hi;
    if (!full) {
        asm volatile("");             // a branch: whole steps are the rule
#pragma unroll
        for (int b = 0; b < RB; ++b)
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const uint32_t n = c.ok >> g & 1 ? row.num[b] : 0;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if ((uint32_t)(kb + 16 * g + 4 * kg + i - row.lo[b]) >= n) sc[b][g][i] = -__builtin_inff();
            }
    }
    float p[RB][8];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
        float tm = -__builtin_inff();
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i) tm = fmaxf(tm, sc[b][g][i]);
        tm = max_16(tm);
        tm = tm == -__builtin_inff() ? tm : tm * scale;
        if (__ballot(tm > m[b]) != 0) {
            const float mn = fmaxf(m[b], tm);
            const float alpha = mf::ex2(m[b] - (mn == -__builtin_inff() ? 0.f : mn));
            m[b] = mn;
            l[b] *= alpha;
#pragma unroll
            for (int i = 0; i < NT; ++i) o[b][i] *= alpha;
        }
        const float ms = m[b] == -__builtin_inff() ? 0.f : m[b];
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i) p[b][4 * g + i] = mf::ex2(__builtin_fmaf(sc[b][g][i], scale, -ms));
    }

    bool repair = false;
    if (!full) {
        // a NaN among the values would reach rows that do not see it (0 x NaN)
        uint32_t any = 0;
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < D / 64; ++j) {
                    const uint32_t b = nan_bytes(c.v[g][i][j]);
                    any |= b;
                    c.v[g][i][j] &= ~((b >> 7) * 0xffu);
                }
        repair = __ballot(any != 0) != 0;
    }
    Frag<NS> pf[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
#pragma unroll
        for (int i = 0; i < 8; ++i) l[b] += p[b][i];
        pf[b] = split8<NS>(p[b]);
    }
    add_pv<D, NS, RB>(c.v[0], c.v[1], vs[0], vs[1], pf, o);
    return repair;
}

// NaN into the outputs of the lane's row whose values are NaN at a key lo <= j < hi.
template <int D>
__device__ __forceinline__ void see_nans(const AttnArgs &a, const int32_t *table, int shift, int hk, int lo, int hi, int kg,
                                         f32x4 *o) {
    constexpr int NT = D / 16;
#pragma unroll 1
    for (int j = lo; j < hi; ++j) {
        const int pid = table[j >> shift];
        if (pid < 0 || pid >= a.kv.n_pages) continue;
        const int64_t row = ((int64_t)pid * a.kv.Hk + hk) * a.kv.page + (j & (a.kv.page - 1));
        const uint32_t *p = (const uint32_t *)(a.kv.v_codes + row * D + kg * (D / 4));
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {            // dims (D / 16)(4 kg + i) + j of the lane
            const uint32_t b = nan_bytes(p[x]);
#pragma unroll
            for (int y = 0; y < 4; ++y)
                o[(4 * x + y) % NT][(4 * x + y) / NT] += nan_or_zero(b, y);
        }
    }
}

template <bool BF, int E>
__device__ __forceinline__ void store_row(void *o, int64_t at, const float *y, float f) {
    float z[E];
#pragma unroll
    for (int j = 0; j < E; ++j) z[j] = y[j] * f;
    if constexpr (E == 8) {
        mf::IO<BF>::store8(o, at, z);
    } else if constexpr (BF) {
        *(mf::bf16x4 *)((bf16_t *)o + at) = mf::Ops<true>::cvt4(f32x4{z[0], z[1], z[2], z[3]});
    } else {
        *(f32x4 *)((float *)o + at) = f32x4{z[0], z[1], z[2], z[3]};
    }
}

// The steps of all units in a row: their number, and where sequence `of` (>= 0) or the
// share of workgroup `block` (of < 0) starts; n: that sequence, base: the steps before it.
struct Place { int64_t total, base; int n; };

__device__ __forceinline__ Place place(const AttnArgs &a, int G, int of, int block, int tid) {
    __shared__ int64_t s_sum[kWaves];
    __shared__ int64_t s_base;
    __shared__ int s_n;
    const int lane = tid & 63, w = tid >> 6, N = a.kv.N;
    // first: up to 256 sequences at a time, in order; the usual call ends after one
    int64_t mine = 0, inc = 0, total = 0;
    for (int n0 = 0; n0 < N; n0 += kAttnThreads) {
        int64_t c = 0;
        if (n0 + tid < N) c = sequence(a, n0 + tid, G).cost(a);
        int64_t x = c;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int64_t y = __shfl_up(x, off);
            if (lane >= off) x += y;
        }
        if (n0 > 0) __syncthreads();
        if (lane == 63) s_sum[w] = x;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kWaves; ++i) {
            if (i < w) x += s_sum[i];
        }
        mine = c;
        inc = total + x;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) total += s_sum[i];
        if (of >= n0 && of < n0 + kAttnThreads && tid == of - n0) { s_base = inc - c; s_n = of; }
    }
    Place p;
    p.total = total;
    if (of < 0) {
        const int64_t from = share_of(total, a.workers) * block;
        if (N <= kAttnThreads) {
            if (inc - mine <= from && from < inc) { s_base = inc - mine; s_n = tid; }
        } else if (from < total) {          // again, now that the total is known
            int64_t before = 0;
            for (int n0 = 0; n0 < N && before <= from; n0 += kAttnThreads) {
                int64_t c = 0;
                if (n0 + tid < N) c = sequence(a, n0 + tid, G).cost(a);
                int64_t x = c;
#pragma unroll
                for (int off = 1; off < 64; off <<= 1) {
                    const int64_t y = __shfl_up(x, off);
                    if (lane >= off) x += y;
                }
                __syncthreads();
                if (lane == 63) s_sum[w] = x;
                __syncthreads();
                x += before;
#pragma unroll
                for (int i = 0; i < kWaves; ++i) {
                    if (i < w) x += s_sum[i];
                    before += s_sum[i];
                }
                if (x - c <= from && from < x) { s_base = x - c; s_n = n0 + tid; }
            }
        }
    }
    __syncthreads();
    p.base = s_base;
    p.n = s_n;
    return p;
}

// The sequence and unit of number x of host_units(): where all sequences are here, in the
// order of the packed rows, sequence n's starting at first(n) = cu[n] G / unit_rows + n (at
// least as many apart as it has); else the same number for each, enough for a short one.
__device__ __forceinline__ bool packed_unit(const AttnArgs &a, int64_t x, int G, int &n, Seq &s, int &rb) {
    if (a.short_rows <= kShortRows) {
        n = (int)x / (kShortRows / a.unit_rows);
        rb = (int)x % (kShortRows / a.unit_rows);
        s = sequence(a, n, G);
        return rb < s.rt;
    }
    n = last_not_above(a.kv.N, x, [&](int i) { return a.kv.cu[i] * G / a.unit_rows + i; });
    s = sequence(a, n, G);
    const int64_t r = x - (s.c0 * G / a.unit_rows + n);
    rb = (int)r;
    return r >= 0 && r < s.rt;
}

// BF: bf16 rows.  One workgroup takes a contiguous share of all (unit, step)
// pairs, or, with workers = 0, one unit; its waves take the steps of a unit in
// turn, each with its next step on the way from HBM, and meet in LDS at the end.
template <int D, bool BF, int RB>
__global__ __launch_bounds__(kAttnThreads, BF && RB == 1 ? 3 : 2) void attn_kernel(const AttnArgs a) {
    constexpr int NS = BF ? 1 : 3;
    constexpr int UR = kRows * RB;             // rows of a unit
    constexpr int NT = D / 16;                 // 16-dim blocks of O
    __shared__ Meet<D, RB> sm;

    const int tid = threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, kg = lane >> 4;
    const int G = a.Hq / a.kv.Hk;
    const int shift = __builtin_ctz(a.kv.page);

    // this workgroup's share [from, to) of the steps
    int64_t from, to, base = 0;
    int n = 0;
    Seq s;
    if (a.workers == 0) {
        int rb;
        if (!packed_unit(a, blockIdx.x / a.kv.Hk, G, n, s, rb)) return;
        from = (int64_t)((int)(blockIdx.x % a.kv.Hk) * s.rt + rb) * s.steps;
        to = from + s.steps;
    } else {
        const Place p = place(a, G, -1, blockIdx.x, tid);
        const int64_t share = share_of(p.total, a.workers);
        from = share * blockIdx.x;
        to = min(from + share, p.total);
        if (from >= to) return;
        n = p.n;
        base = p.base;
        s = sequence(a, n, G);
    }

    for (int64_t at = from; at < to; s = sequence(a, ++n, G)) {
        const int64_t end = base + s.cost(a);  // of this sequence
        const int32_t *table = a.kv.table + (int64_t)n * a.kv.width;
        while (at < to && at < end) {
            const uint32_t unit = quotient(at - base, s.steps);
            const int64_t ubase = base + (int64_t)unit * s.steps, uend = ubase + s.steps;
            const int hk = (int)(unit / (uint32_t)s.rt), rb = (int)(unit % (uint32_t)s.rt);
            const bool whole = ubase >= from && uend <= to;
            // its steps here, less those that no row of the unit sees
            const int t0 = min(rb * UR / G, s.len - 1), t1 = min((rb * UR + UR - 1) / G, s.len - 1);
            const int beg = max(s.lo + (int)(at - ubase), s.begin_of(a, t0) / kStep);
            const int stop = min(s.lo + (int)(min(uend, to) - ubase), (s.end_of(a, t1) + kStep - 1) / kStep);

            float m[RB], l[RB];
            f32x4 o[RB][NT];
#pragma unroll
            for (int b = 0; b < RB; ++b) {
                m[b] = -__builtin_inff();
                l[b] = 0.f;
#pragma unroll
                for (int i = 0; i < NT; ++i) o[b][i] = f32x4{0.f, 0.f, 0.f, 0.f};
            }
            Rows<D, NS, RB> row;
            Codes<D> c0, c1;
            int t = beg + w;
            if (t < stop) {
                // In flight from here on: the codes of the next step, the lookup of the one
                // after.  Past the last step they are the last one's again: a load that
                // might not be issued would make every wait one for all loads.
                const int last = stop - 1;
                Lookup pg{table, shift, s.kvl, 0};
                pg.ask(t, lane);
                row.load(a, s, rb, hk, G, stop * kStep, lane);
                Lookup next = pg;
                next.ask(min(t + kWaves, last), lane);
                load_step<D>(a, pg, hk, t, lane, c0);
                auto step = [&](Codes<D> &c, Codes<D> &ahead) {
                    pg = next;
                    next.ask(min(t + 2 * kWaves, last), lane);
                    load_step<D>(a, pg, hk, min(t + kWaves, last), lane, ahead);
                    if (one_step<D, NS, RB>(row, c, t, a.scale, lane, m, l, o)) {
#pragma unroll
                        for (int b = 0; b < RB; ++b)
                            see_nans<D>(a, table, shift, hk, max(row.lo[b], t * kStep), min(row.lo[b] + row.num[b], (t + 1) * kStep),
                                        kg, o[b]);
                    }
                    t += kWaves;
                };
                // Two steps a pass with one way out, so that the waits of a pass know what is
                // on its way; the second of an odd last pair sees no key.
                do {
                    step(c0, c1);
                    step(c1, c0);
                } while (t < stop);
            }

            // the waves meet
#pragma unroll
            for (int b = 0; b < RB; ++b) {
                const float sum = sum_16(l[b]);
                if (kg == 0) { sm.m[w][kRows * b + col] = m[b]; sm.l[w][kRows * b + col] = sum; }
#pragma unroll
                for (int i = 0; i < 4; ++i)       // dims (D / 16)(4 kg + i) + j, j < NT
#pragma unroll
                    for (int j = 0; j < NT; j += 4)
                        *(f32x4 *)&sm.o[w][kRows * b + col][NT * (4 * kg + i) + j] =
                            f32x4{o[b][j][i], o[b][j + 1][i], o[b][j + 2][i], o[b][j + 3][i]};
            }
            __syncthreads();
#pragma unroll
            for (int b = 0; b < RB; ++b) {
                constexpr int E = kRows * D / kAttnThreads;      // 8 or 4 dims per thread
                const int r = kRows * b + tid / (D / E), d = (tid % (D / E)) * E;
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
                const int R = rb * UR + r;
                if (whole) {
                    if (R < s.len * G) {
                        const int64_t at_row = (s.c0 + R / G) * a.Hq + hk * G + R % G;
                        store_row<BF, E>(a.o, at_row * D + d, y, L == 0.f ? 0.f : 1.f / L);
                        if (a.lse && d == 0) a.lse[at_row] = lse_of(M, L);
                    }
                } else {
                    // cut at this workgroup's end: its second slot; at its start: the first
                    float *dst = a.part + (2 * (int64_t)blockIdx.x + (ubase >= from ? 1 : 0)) * (UR * (D + 2));
                    store_row<false, E>(dst, r * D + d, y, 1.f);
                    if (d == 0) { dst[UR * D + r] = M; dst[UR * D + UR + r] = L; }
                }
            }
            __syncthreads();
            at = uend;
        }
        base = end;
        if (at >= to) break;
    }
}

// Joins the parts of every unit that attn_kernel cut.  A workgroup takes RW rows
// of a unit; 256 / RW threads share a row: D / E of them its dims, the rest its parts.
template <int D, bool BF, int RB, int RW>
__global__ __launch_bounds__(kAttnThreads) void join_kernel(const AttnArgs a) {
    constexpr int UR = kRows * RB;
    constexpr int E = kRows * D / kAttnThreads;
    constexpr int TD = D / E;                           // 16 threads over the dims
    constexpr int SL = kAttnThreads / (RW * TD);        // slices of the parts
    __shared__ float s_o[SL][RW][D + 4];
    __shared__ float s_m[SL][RW], s_l[SL][RW];
    const int tid = threadIdx.x;
    const int G = a.Hq / a.kv.Hk;
    const uint32_t u = blockIdx.x / (UR / RW);
    const int hk = u % a.kv.Hk;
    int n, rb;
    Seq s;
    if (!packed_unit(a, u / a.kv.Hk, G, n, s, rb)) return;
    const Place p = place(a, G, n, 0, tid);
    const int64_t share = share_of(p.total, a.workers);
    const int64_t ubase = p.base + (int64_t)(hk * s.rt + rb) * s.steps;
    const int64_t w0 = ubase / share, w1 = (ubase + s.steps - 1) / share;
    if (w0 == w1) return;                               // written whole
    const int d = (tid % TD) * E, sl = tid / TD % SL, rr = tid / (TD * SL);
    const int r = (blockIdx.x % (UR / RW)) * RW + rr;
    float M = -__builtin_inff(), L = 0.f, y[E];
#pragma unroll
    for (int j = 0; j < E; ++j) y[j] = 0.f;
    for (int64_t i = w0 + sl; i <= w1; i += SL) {
        const float *src = a.part + (2 * i + (ubase >= i * share ? 1 : 0)) * (UR * (D + 2));
        const float m = src[UR * D + r], l = src[UR * D + UR + r];
        float v[E];
#pragma unroll
        for (int j = 0; j < E; j += 4) *(f32x4 *)(v + j) = *(const f32x4 *)(src + r * D + d + j);
        const float mn = fmaxf(M, m), ms = mn == -__builtin_inff() ? 0.f : mn;
        const float f0 = mf::ex2(M - ms), f1 = mf::ex2(m - ms);
        M = mn;
        L = L * f0 + l * f1;
#pragma unroll
        for (int j = 0; j < E; ++j) y[j] = y[j] * f0 + v[j] * f1;
    }
    if constexpr (SL > 1) {
#pragma unroll
        for (int j = 0; j < E; ++j) s_o[sl][rr][d + j] = y[j];
        if (d == 0) { s_m[sl][rr] = M; s_l[sl][rr] = L; }
        __syncthreads();
        if (sl != 0) return;
        M = -__builtin_inff();
        for (int i = 0; i < SL; ++i) M = fmaxf(M, s_m[i][rr]);
        const float ms = M == -__builtin_inff() ? 0.f : M;
        L = 0.f;
#pragma unroll
        for (int j = 0; j < E; ++j) y[j] = 0.f;
        for (int i = 0; i < SL; ++i) {
            const float f = mf::ex2(s_m[i][rr] - ms);
            L += s_l[i][rr] * f;
#pragma unroll
            for (int j = 0; j < E; ++j) y[j] += s_o[i][rr][d + j] * f;
        }
    }
    const int R = rb * UR + r;
    if (R >= s.len * G) return;
    const int64_t row = (s.c0 + R / G) * a.Hq + hk * G + R % G;
    store_row<BF, E>(a.o, row * D + d, y, L == 0.f ? 0.f : 1.f / L);
    if (a.lse && d == 0) a.lse[row] = lse_of(M, L);
}

// Units over all sequences at most, per kv head.
int64_t host_units(int64_t T, int G, int N, const AttnArgs &a) {
    return a.short_rows <= kShortRows ? (int64_t)N * (kShortRows / a.unit_rows) : T * G / a.unit_rows + N;
}

template <int D, bool BF, int RB>
hipError_t launch(const AttnArgs &a, hipStream_t s) {
    constexpr int UR = kRows * RB;
    const int64_t units = host_units(a.kv.T, a.Hq / a.kv.Hk, a.kv.N, a) * a.kv.Hk;
    if (units > INT32_MAX / UR) return hipErrorInvalidValue;
    const dim3 block(kAttnThreads);
    hipLaunchKernelGGL((attn_kernel<D, BF, RB>), dim3((unsigned)(a.workers ? a.workers : units)), block, 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.workers == 0) return e;
    // few units have many parts each: more workgroups per unit and threads per row
    if (units < a.workers / 8)
        hipLaunchKernelGGL((join_kernel<D, BF, RB, 1>), dim3((unsigned)(units * UR)), block, 0, s, a);
    else
        hipLaunchKernelGGL((join_kernel<D, BF, RB, kRows>), dim3((unsigned)(units * RB)), block, 0, s, a);
    return hipGetLastError();
}

}  // namespace

// Workgroups of attn_kernel that a compute unit holds (by their registers).  The shares
// are cut for just these: half as many take 258 us for 64 sequences of 512 to 32,768
// tokens at 32 / 8 heads of 128, these 231, twice as many 256 (more parts to write and
// join).  Counting a unit's start and end as kUnitCost steps evens out shares of many
// short units and of few long ones (246 us without).
static int resident(bool bf16, int D, int unit_rows) {
    if (unit_rows > kRows) return 2;
    return D == 64 ? (bf16 ? 4 : 3) : (bf16 ? 3 : 2);
}

void attn_plan(int cus, bool bf16, int D, int N, int64_t T, int Hq, int Hk, int64_t max_kv, AttnArgs *a) {
    const int G = Hq / Hk;
    const int64_t rows = T * G;
    a->workers = -1;
    a->row_units = 0;
    a->row_splits = a->split_tiles = 1;
    // keys that a unit can see: the table's, or its window's
    const int64_t keys = a->window > 0 ? std::min<int64_t>(max_kv, (int64_t)a->window + 2 * kRows + 2 * kStep) : max_kv;
    // The lengths are known on the device only.  A call goes to this kernel alone where it is small, or
    // where equal lengths would be short (a decode step, equally many drafted tokens); a single long
    // sequence to the other; else each sequence goes to its own, and a kernel that has none costs 5 us,
    // its join as much.  Lengths that could be equal and are not: a long sequence then reads its keys
    // once for each 32 rows, in shares on all of the card beside the short ones, instead of for each 128
    // after them.  us for T = a multiple of N / one row more (32 / 8 heads of 128, bf16, decoding
    // sequences over 2,000 keys and a chunk): 63 and 449 tokens over 4,000 keys 160 / 193, over 16,000
    // 390 / 488; 255 and 1,793 over 0 273 / 354, over 4,000 686 / 424, over 16,000 1,491 / 783, over 60,000
    // 4,558 / 2,045 (the worst found).  And lengths that are equal but for a padded row: 64 decoding
    // sequences over 2,000 keys 62, 63 in 64 rows 91; 64 of 5 tokens 58, with one more row 84.
    const bool small = std::max<int64_t>(rows / kRows, N) * Hk * keys <= small_call(bf16, D);
    const int64_t most = T % N == 0 ? rows / N : rows;      // rows of a sequence if they are equally long
    const bool all_short = small || most <= (N == 1 ? kShortRows : 2 * kRows);
    const bool all_long = N == 1 && !all_short;
    a->unit_rows = bf16 && !small && most > kRows ? 2 * kRows : kRows;
    // (alone, it also takes a sequence that padding made look long)
    a->short_rows = all_short ? INT32_MAX : all_long ? 0 : kShortRows;
    if (!all_long) {
        const int64_t units = host_units(T, G, N, *a) * Hk;
        const bool direct = keys <= kDirect || (keys <= 2 * kDirect && units >= 64);
        a->workers = direct ? 0 : cus * resident(bf16, D, a->unit_rows);
    }
    if (!all_short) {
        a->row_units = a->row_fold = (int32_t)(rows / kRowTile + N);
        const int64_t units = std::max<int64_t>((rows + kRowTile - 1) / kRowTile, N) * Hk;
        if (units < 2 * cus) {
            // Two workgroups for every compute unit; the more units, the more their parts cost against
            // what sharing the keys gains.  us whole / 2 / 4 / 8 parts at 32 / 8 heads of 128: 64 units,
            // 2,000 keys 53 / 39 / 33 / 38, 15,000 329 / 180 / 102 / 86; 128 units, 512 keys
            // 21 / 23 / 23 / 23, 4,000 94 / 64 / 59 / 71; 256 units, 1,024 keys 32 / 37 / 49 / 49, 4,000
            // 96 / 83 / 98 / 125; 384 units, 1,536 keys 46 / 53 / 73 / 74, 6,144 177 / 188 / 185 / 225 (2 are taken).
            a->split_tiles = units < cus / 4 ? 4 : units < cus ? 8 : 16;
            const int64_t want = (2 * (int64_t)cus + units - 1) / units;
            a->row_splits =
                (int32_t)std::max<int64_t>(1, std::min<int64_t>({want, 32, max_kv / (a->split_tiles * kTile)}));
        }
        if (a->row_splits == 1 && units <= 2 * cus) a->row_fold = (a->row_units + 1) / 2;
    }
}

size_t attn_partial_bytes(int D, const AttnArgs &a) {
    const size_t one = a.workers > 0 ? (size_t)a.workers * 2 * a.unit_rows * (D + 2) : 0;
    const size_t rows = a.row_splits > 1 ? (size_t)a.row_units * a.kv.Hk * a.row_splits * kRowTile * (D + 2) : 0;
    return std::max(one, rows) * sizeof(float);
}

hipError_t launch_attn(bool bf16, int D, const AttnArgs &a, hipStream_t s) {
    if (a.unit_rows > kRows) {
        if (bf16 && D == 128) return launch<128, true, 2>(a, s);
        if (bf16 && D == 64) return launch<64, true, 2>(a, s);
        return hipErrorInvalidValue;
    }
    if (D == 128) return bf16 ? launch<128, true, 1>(a, s) : launch<128, false, 1>(a, s);
    if (D == 64) return bf16 ? launch<64, true, 1>(a, s) : launch<64, false, 1>(a, s);
    return hipErrorInvalidValue;
}

}  // namespace kda
