// kda_attn_rows.hip -- attention of long runs of new tokens (prompts and their
// chunks) over the 8-bit cache: the formulas of kda_attn.hip with the keys
// shared by 128 query rows, bound by the matrix cores.
//
// A workgroup takes 128 rows (token, head of the group) of one sequence and kv
// head; each of its four waves owns 32 and keeps their queries, maxima, sums and
// outputs in registers.  64 keys at a time are staged through LDS, two buffers:
// while a tile is computed the next one is on its way from HBM in registers.
// Wave w stages the 16 tokens of group w, so one page lookup serves a wave.
//
// Both are staged as bf16 operand fragments, a lane's 16 bytes in lane order (no
// bank conflicts), the values transposed by byte permutes: the conversions are
// done once per workgroup.  (Keys left as codes halve their LDS traffic, 28% of
// the cycles, but every wave converts them again: the vector pipe is the busier
// one, 60%.)  The 8-bit matrix instruction would take codes as they are, with a
// bf16 query as two e4m3 terms (4 + 4 bits), but it sums its products with fewer
// bits than fp32: scores came out off by 2^-17 of sum |q k|, so it is not used.
// With fp32 rows queries and probabilities are three bf16 terms, as in
// kda_attn.hip.
//
// The maximum is followed lazily: outputs are scaled only when some row's
// maximum grew by more than 2^8 since (probabilities stay below 2^8, which
// costs neither fp32 sums nor bf16 operands any precision).
//
// A prompt of 8,192 tokens at 32 / 8 heads of 128 with bf16 rows takes 555 us (990 TFLOP/s;
// an 8192^3 product of the library 1,210 to 1,240), four chunks of 300 to 1,024 over up to
// 15,000 keys 461 (958).  The matrix cores are busy 43% of the cycles and the
// vector pipe 47%, at 2.0 to 2.2 GHz.  Two workgroups per compute unit, each at its own
// place in a tile, overlap the two better than one of 256 rows: as eight waves of 32 rows
// (half the conversions and LDS writes) 578, as four of 64, each computing the next tile's
// scores beside this one's exponentials, 558.

#include "kda_attn_ops.h"

namespace kda {
namespace {

using namespace attn;

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kWaveRows = 32;
constexpr float kLag = 8.f;           // growth of a maximum (log2) that rescales

// The unit of a workgroup: rows [row0, row0 + 128) of sequence n, and the tiles
// [beg, end) that some of them see, shared by `splits` workgroups.
struct Unit {
    Seq s;
    int n, row0, beg, end, splits;
};

__device__ __forceinline__ bool find_unit(const AttnArgs &a, int64_t x, int G, Unit &u) {
    // units of sequence n start at first(n) = cu[n] G / 128 + n
    u.n = last_not_above(a.kv.N, x, [&](int n) { return a.kv.cu[n] * G / kRowTile + n; });
    u.s = sequence(a, u.n, G);
    const int64_t rows = (int64_t)u.s.len * G;
    const int64_t r = (x - (u.s.c0 * G / kRowTile + u.n)) * kRowTile;
    if (rows <= a.short_rows || r < 0 || r >= rows) return false;
    u.row0 = (int)r;
    const int t0 = u.row0 / G, t1 = min((u.row0 + kRowTile - 1) / G, u.s.len - 1);
    u.end = (u.s.end_of(a, t1) + kTile - 1) / kTile;
    u.beg = min(u.s.begin_of(a, t0) / kTile, u.end);
    u.splits = min(a.row_splits, max((u.end - u.beg + a.split_tiles - 1) / a.split_tiles, 1));
    return true;
}

template <int D> struct Stage {
    u32x4 k[2][D / 16][64];           // 32 tokens: steps of 16 dims, (token, 8 dims) per lane
    u32x4 v[4][D / 32][64];           // 16 tokens: 32 dims, (dim, 8 tokens) per lane
    int ok[4];                        // group of 16 tokens has a page and starts before the last key
    int nan, hole;                    // the tile if it held a NaN value, a group that is not ok
};

__device__ __forceinline__ f32x16 mma(u32x4 a, bf16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), b, c, 0, 0, 0);
}

// Queries of a lane's row as operand fragments, NS bf16 terms each.
template <int D, int NS> struct Query {
    Frag<NS> f[D / 16];               // step i: dims 16 i + 8 kg + 0..7
    __device__ void load(const void *q, int64_t at, int kg, float sign) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            float x[8];
            mf::IO<NS == 1>::load8(q, at + 16 * i + 8 * kg, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] *= sign;       // exact
            f[i] = split_query8<NS>(x);
        }
    }
    // S^T of both halves of a tile: fragments are read two steps ahead, and other(i) is
    // work for the vector pipe beside step i of D / 16.
    template <typename F>
    __device__ __forceinline__ void scores(const Stage<D> &st, int lane, f32x16 (&c)[2], F other) const {
        constexpr int N = D / 16;
        c[0] = c[1] = f32x16{};
        u32x4 x[3][2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) x[i][tt] = st.k[tt][i][lane];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (i + 2 < N) {
#pragma unroll
                for (int tt = 0; tt < 2; ++tt) x[(i + 2) % 3][tt] = st.k[tt][i + 2][lane];
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int t = 0; t < NS; ++t) {
                c[0] = mma(x[i % 3][0], f[i].f[t], c[0]);
                c[1] = mma(x[i % 3][1], f[i].f[t], c[1]);
            }
            other(i);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
};

// A tile on its way from HBM: wave w holds group w (16 tokens).
template <int D> struct Flight {
    u32x4 k[D / 64];
    uint32_t v[8];
    float ks, vs;
    int ok;

    __device__ void load(const AttnArgs &a, int pid, int hk, int at, int lane) {
        ok = pid >= 0 && pid < a.kv.n_pages;
        ks = vs = 1.f;
        if (ok) {
            const int64_t ph = (int64_t)pid * a.kv.Hk + hk;
            const int64_t base = (ph * a.kv.page + (at & (a.kv.page - 1))) * D;
            const uint8_t *kp = a.kv.k_codes + base + (lane & 15) * D + (lane >> 4) * 16;
            const uint8_t *vp = a.kv.v_codes + base + 4 * (lane >> 5) * D + (lane & 31) * (D / 32);
#pragma unroll
            for (int r = 0; r < D / 64; ++r) k[r] = *(const u32x4 *)(kp + r * 64);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint8_t *p = vp + ((i >> 2) * 8 + (i & 3)) * D;
                if constexpr (D == 128) v[i] = *(const uint32_t *)p;
                else v[i] = *(const uint16_t *)p;
            }
            ks = a.kv.k_scale[ph];
            vs = a.kv.v_scale[ph];
        } else {
#pragma unroll
            for (int r = 0; r < D / 64; ++r) k[r] = u32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = 0;
        }
    }

    // Values that must not take part, out; what the tile is, noted.  left: tokens of the
    // group that the sequence has (16 for a whole one); what lies behind them on the page
    // is anything.  part: some rows of the unit do not see all of the tile; NaN values are
    // then left out (0 x NaN is a NaN) and see_nans() follows.
    __device__ void settle(Stage<D> &st, int t, int w, int lane, int left, bool part) {
        if (left < 16) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if ((i >> 2) * 8 + 4 * (lane >> 5) + (i & 3) >= left) v[i] = 0;
        }
        if (part) {
            uint32_t bad = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t b = nan_bytes(v[i]);
                bad |= b;
                v[i] &= ~((b >> 7) * 0xffu);
            }
            if (bad) st.nan = t;      // every writer stores the same value
        }
        if (!ok) st.hole = t;
        if (lane == 0) st.ok[w] = ok;
    }

    // Part i of kParts of the operand fragments.
    static constexpr int kParts = D / 16;
    u32x4 kf[D / 32], vf[D / 32];
    __device__ __forceinline__ void widen_part(int i) {
        if (i < D / 32) {
            const uint32_t c0 = i & 1 ? k[i >> 1][2] : k[i >> 1][0], c1 = i & 1 ? k[i >> 1][3] : k[i >> 1][1];
            kf[i] = u32x4{widen<false>(c0, ks), widen<true>(c0, ks), widen<false>(c1, ks), widen<true>(c1, ks)};
        } else {
            const int j = i - D / 32;
            const bf16x8 f = j == 0 ? v_frag<0>(v, vs, vs) : j == 1 ? v_frag<1>(v, vs, vs)
                           : j == 2 ? v_frag<2>(v, vs, vs) : v_frag<3>(v, vs, vs);
            vf[j] = __builtin_bit_cast(u32x4, f);
        }
    }
    __device__ __forceinline__ void store(Stage<D> &st, int w, int lane) const {
        // group w: tokens 16 (w & 1) + .. of half w >> 1; piece p: dims 16 p + 0..15
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            st.k[w >> 1][4 * (i >> 1) + (lane >> 4)][16 * (w & 1) + (lane & 15) + 32 * (i & 1)] = kf[i];
            st.v[w][i][lane] = vf[i];
        }
    }
};

// NaN into the outputs of the lane's row whose values are NaN at a key lo <= j < hi.
template <int D>
__device__ __forceinline__ void see_nans(const AttnArgs &a, const int32_t *table, int shift, int hk, int lo, int hi, int kg,
                                         f32x16 *o) {
    constexpr int NJ = D / 32, E = D / 8;
#pragma unroll 1
    for (int j = lo; j < hi; ++j) {
        const int pid = table[j >> shift];
        if (pid < 0 || pid >= a.kv.n_pages) continue;
        const int64_t row = ((int64_t)pid * a.kv.Hk + hk) * a.kv.page + (j & (a.kv.page - 1));
        const uint8_t *p = a.kv.v_codes + row * D + E * kg;
#pragma unroll
        for (int e = 0; e < 4; ++e)                   // dims 2 E e + E kg + NJ i + j of the lane
#pragma unroll
            for (int x = 0; x < E / 4; ++x) {
                const uint32_t b = nan_bytes(*(const uint32_t *)(p + 2 * E * e + 4 * x));
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    o[(4 * x + y) % NJ][4 * e + (4 * x + y) / NJ] += nan_or_zero(b, y);
            }
    }
}

template <int D, bool BF>
__global__ __launch_bounds__(kAttnThreads, BF ? 2 : 1) void rows_kernel(const AttnArgs a) {
    constexpr int NS = BF ? 1 : 3;
    constexpr int NJ = D / 32;
    __shared__ __align__(16) Stage<D> stage[2];

    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 31, kg = lane >> 5;
    const int G = a.Hq / a.kv.Hk;
    const int hk = blockIdx.x % a.kv.Hk;
    // the last rows see the most keys: they go first; where all units fit the card at once, the second
    // half in turn (a long one and a short one on each compute unit)
    const int64_t y = blockIdx.x / a.kv.Hk, z = y / a.row_splits;
    const int split = (int)(y % a.row_splits);
    Unit u;
    if (!find_unit(a, z < a.row_fold ? a.row_units - 1 - z : z - a.row_fold, G, u) || split >= u.splits) return;
    const Seq &s = u.s;
    const int tiles = u.end - u.beg;
    const int t0 = u.beg + (int)((int64_t)tiles * split / u.splits);
    const int t1 = u.beg + (int)((int64_t)tiles * (split + 1) / u.splits);

    // the lane's row, the keys it sees, and what all / any rows of the wave see
    const int R = u.row0 + kWaveRows * w + col;
    const bool live = R < s.len * G;
    const int tok = min(R / G, s.len - 1);
    const int vis_hi = live ? s.end_of(a, tok) : 0, vis_lo = s.begin_of(a, tok);
    const int first = u.row0 + kWaveRows * w;
    const int wt0 = min(first / G, s.len - 1), wt1 = min((first + kWaveRows - 1) / G, s.len - 1);
    const int any_hi = first < s.len * G ? s.end_of(a, wt1) : 0, any_lo = s.begin_of(a, wt0);
    const int all_hi = s.end_of(a, wt0), all_lo = s.begin_of(a, wt1);

    const float sl = a.scale;
    Query<D, NS> q;
    q.load(a.q, (s.c0 + tok) * a.q_row + (int64_t)(hk * G + R % G) * D, kg, a.q_sign);

    float m = -__builtin_inff(), l = 0.f;
    f32x16 o[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) o[j] = f32x16{};
    if (tid < 2) stage[tid].nan = stage[tid].hole = -1;

    const int shift = __builtin_ctz(a.kv.page);
    const int32_t *table = a.kv.table + (int64_t)u.n * a.kv.width;
    // A lane's copy of the wave's page: made uniform where it is used, one tile later, so
    // that nothing waits for the lookup together with the codes on their way.
    const int zero = opaque(0);
    auto page_of = [&](int t) {
        const int at = t * kTile + 16 * w;
        return t < t1 && at < s.kvl ? table[(at >> shift) + zero] : -1;
    };
    // tiles outside [whole_lo, whole_hi) are not seen whole by every row of the unit
    const int u0 = min(u.row0 / G, s.len - 1), u1 = min((u.row0 + kRowTile - 1) / G, s.len - 1);
    const int whole_lo = s.begin_of(a, u1), whole_hi = u.row0 + kRowTile <= s.len * G ? s.end_of(a, u0) : 0;
    auto part = [&](int t) { return t * kTile < whole_lo || (t + 1) * kTile > whole_hi; };
    auto left_of = [&](int t) {
        return min(max(s.kvl - (t * kTile + 16 * w), 0), 16);
    };
    Flight<D> fl;
    auto load = [&](int t, int pid) {
        fl.load(a, __builtin_amdgcn_readfirstlane(pid), hk, t * kTile + 16 * w, lane);
    };
    int pid = page_of(t0);
    if (t0 < t1) {
        load(t0, pid);
        pid = page_of(t0 + 1);
        __syncthreads();                       // nan, hole
        fl.settle(stage[t0 & 1], t0, w, lane, left_of(t0), part(t0));
#pragma unroll
        for (int i = 0; i < Flight<D>::kParts; ++i) fl.widen_part(i);
        fl.store(stage[t0 & 1], w, lane);
        if (t0 + 1 < t1) {
            load(t0 + 1, pid);
            pid = page_of(t0 + 2);
        }
    }
    __syncthreads();

    for (int t = t0; t < t1; ++t) {
        const Stage<D> &st = stage[t & 1];
        const int kb = t * kTile;
        const int nan = st.nan, hole = st.hole;
        if (t + 1 < t1) fl.settle(stage[(t + 1) & 1], t + 1, w, lane, left_of(t + 1), part(t + 1));
        // The next tile's conversions beside this one's products; past the last tile they
        // write what nobody reads.
        f32x16 sc[2];
        // (the two waves of a SIMD: the one that is further, at its exponentials and the
        // product with the values, goes first; 4% on prompt chunks)
        __builtin_amdgcn_s_setprio(0);
        q.scores(st, lane, sc, [&](int i) { fl.widen_part(i); });
        fl.store(stage[(t + 1) & 1], w, lane);
        if (t + 2 < t1) {
            load(t + 2, pid);
            pid = page_of(t + 3);
        }
        if (kb < any_hi && kb + kTile > any_lo) {
            u32x4 vf[2][NJ];                   // values of step k, and of the next
#pragma unroll
            for (int j = 0; j < NJ; ++j) vf[0][j] = st.v[0][j][lane];
            __builtin_amdgcn_sched_barrier(0);
            const bool full = hole != t && kb >= all_lo && kb + kTile <= all_hi;
            if (!full) {
                const int lo = vis_lo - kb, hi = vis_hi - kb;
                const int gm = st.ok[0] | st.ok[1] << 1 | st.ok[2] << 2 | st.ok[3] << 3;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const int j = 32 * (i >> 4) + 8 * ((i >> 2) & 3) + 4 * kg + (i & 3);
                    if (!(j >= lo && j < hi && (gm >> (j >> 4) & 1))) sc[i >> 4][i & 15] = -__builtin_inff();
                }
            }
            __builtin_amdgcn_s_setprio(1);
            float mx = -__builtin_inff();
#pragma unroll
            for (int i = 0; i < 32; ++i) mx = fmaxf(mx, sc[i >> 4][i & 15]);
            mx = max_32(mx);
            mx = mx == -__builtin_inff() ? mx : mx * sl;
            if (__ballot(mx > m + kLag) != 0) {
                const float mn = fmaxf(m, mx);
                const float f = mf::ex2(m - (mn == -__builtin_inff() ? 0.f : mn));
                m = mn;
                l *= f;
#pragma unroll
                for (int j = 0; j < NJ; ++j) o[j] *= f;
            }
            const float ms = m == -__builtin_inff() ? 0.f : m;
            float p[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) p[i] = mf::ex2(__builtin_fmaf(sc[i >> 4][i & 15], sl, -ms));
#pragma unroll
            for (int i = 0; i < 32; ++i) l += p[i];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (k < 3) {
#pragma unroll
                    for (int j = 0; j < NJ; ++j) vf[(k + 1) & 1][j] = st.v[k + 1][j][lane];
                }
                const Frag<NS> pf = split8<NS>(p + 8 * k);
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int i = 0; i < NS; ++i)
                        o[j] = mma(vf[k & 1][j], pf.f[i], o[j]);
            }
            if (nan == t)
                see_nans<D>(a, table, shift, hk, max(vis_lo, kb), min(vis_hi, kb + kTile), kg, o);
        }
        __syncthreads();
    }

    l = sum_32(l);
    if (!live) return;
    constexpr int E = D / 8;                   // contiguous dims per group of 4 results
    if (u.splits == 1) {
        const int64_t row = (s.c0 + tok) * a.Hq + hk * G + R % G;
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float z[E];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < NJ; ++j) z[NJ * i + j] = o[j][4 * e + i] * inv;
#pragma unroll
            for (int i = 0; i < E; i += 8) mf::IO<BF>::store8(a.o, row * D + 2 * E * e + E * kg + i, z + i);
        }
        if (a.lse && kg == 0) a.lse[row] = lse_of(m, l);
    } else {
        float *dst = a.part + (int64_t)blockIdx.x * (kRowTile * (D + 2));
        const int r = kWaveRows * w + col;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float z[E];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < NJ; ++j) z[NJ * i + j] = o[j][4 * e + i];
#pragma unroll
            for (int i = 0; i < E; i += 8) mf::IO<false>::store8(dst, r * D + 2 * E * e + E * kg + i, z + i);
        }
        if (kg == 0) { dst[kRowTile * D + r] = m; dst[kRowTile * (D + 1) + r] = l; }
    }
}

// Joins the splits of a unit: D / 8 threads take a row.
template <int D, bool BF>
__global__ __launch_bounds__(kAttnThreads) void join_rows_kernel(const AttnArgs a) {
    constexpr int RP = kAttnThreads / (D / 8);          // rows per workgroup
    const int G = a.Hq / a.kv.Hk;
    const int64_t x = blockIdx.x / (kRowTile / RP);
    const int hk = (int)(x % a.kv.Hk);
    const int64_t y = x / a.kv.Hk;
    Unit u;
    if (!find_unit(a, a.row_units - 1 - y, G, u) || u.splits == 1) return;
    const int r = (int)(blockIdx.x % (kRowTile / RP)) * RP + threadIdx.x / (D / 8), d = threadIdx.x % (D / 8) * 8;
    const int R = u.row0 + r;
    if (R >= u.s.len * G) return;
    float M = -__builtin_inff(), L = 0.f, z[8] = {};
#pragma unroll 4
    for (int i = 0; i < u.splits; ++i) {
        const float *src = a.part + ((y * a.row_splits + i) * a.kv.Hk + hk) * (kRowTile * (D + 2));
        const float m = src[kRowTile * D + r], l = src[kRowTile * (D + 1) + r];
        const float mn = fmaxf(M, m), ms = mn == -__builtin_inff() ? 0.f : mn;
        const float f0 = mf::ex2(M - ms), f1 = mf::ex2(m - ms);
        float v[8];
        mf::load8f(src + r * D + d, v);
        M = mn;
        L = L * f0 + l * f1;
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = z[j] * f0 + v[j] * f1;
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] *= inv;
    const int64_t row = (u.s.c0 + R / G) * a.Hq + hk * G + R % G;
    mf::IO<BF>::store8(a.o, row * D + d, z);
    if (a.lse && d == 0) a.lse[row] = lse_of(M, L);
}

template <int D, bool BF>
hipError_t launch(const AttnArgs &a, hipStream_t s) {
    const int64_t units = (int64_t)a.row_units * a.kv.Hk;
    const int64_t per = kRowTile / (kAttnThreads / (D / 8));
    if (units * a.row_splits > INT32_MAX || units * per > INT32_MAX) return hipErrorInvalidValue;
    hipLaunchKernelGGL((rows_kernel<D, BF>), dim3((unsigned)(units * a.row_splits)), dim3(kAttnThreads), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.row_splits == 1) return e;
    hipLaunchKernelGGL((join_rows_kernel<D, BF>), dim3((unsigned)(units * per)), dim3(kAttnThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_rows(bool bf16, int D, const AttnArgs &a, hipStream_t s) {
    if (D == 128) return bf16 ? launch<128, true>(a, s) : launch<128, false>(a, s);
    if (D == 64) return bf16 ? launch<64, true>(a, s) : launch<64, false>(a, s);
    return hipErrorInvalidValue;
}

}  // namespace kda
