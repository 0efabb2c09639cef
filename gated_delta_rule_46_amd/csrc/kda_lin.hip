// kda_lin.hip -- linear attention with one decay per head, chunked prefill.
//
//     S_t = e^{g_t} S_{t-1} + k_t v_t^T,    o_t = scale S_t^T q_t
//
// With G_i the log decays summed over a chunk's tokens up to i, a chunk of C
// tokens that starts from the state S is
//     P_ij = scale e^{G_i - G_j} q_i.k_j  (j <= i),
//     o_i  = scale e^{G_i} S^T q_i + sum_j P_ij v_j,
//     S   <- e^{G_C} S + sum_j e^{G_C - G_j} k_j v_j^T.
// Every exponent is a difference that is at most zero (g <= 0), so no decay
// overflows or needs a floor; G is summed in fp64 and kept as two floats, so that
// a difference keeps its 24 bits behind a decay of any size.
//
// One workgroup takes a unit (a sequence, or a segment of a long one) and value head
// from its first chunk to its last; a wave owns 16 of the value columns (32 of bf16 heads of 128 in one
// workgroup) and keeps their part of S in the accumulators of the state product.  As the rows of S that a
// lane accumulates are chosen to be 8 consecutive ones of a 32-row block, the registers are
// the operand of S^T q as they stand.  The three tiles of P (C x C, its lower triangle) are formed by the
// first three waves and exchanged through LDS.
//
// With bf16 rows P and the state as an operand of S^T q are rounded to bf16, by half a step each.  A second
// term of that operand takes 4 to 15% of prompts (131,072 tokens 1,140 -> 1,307 us) and changes their outputs'
// distance from the exact ones in no digit (0.0017, the outputs' own rounding); where a large state is resumed it is
// 0.0022 without and 0.0017 with it (64 x 5 drafted tokens, 63.6 -> 64.9 us).  The product that forms the
// state takes its weighted values in three terms, which hold 24 bits.
//
// Chunks are a pipeline with one barrier each.  Before it the waves form P of the chunk, S^T q and the new
// state, and put the next chunk's q, k, v (loaded into registers a chunk earlier) into the other half of
// LDS; behind it they add P v (v is an operand in registers by then).  So a wave can be a whole chunk behind
// another one, and two buffers of everything are enough.
//
// A long sequence is cut into segments where there are too few units for the card: a first
// launch forms what each segment (but the last) adds to the state, from its end backwards
// and only as far as its decays leave anything; a second one carries the states over the
// segments; then all segments run as units of their own.
//
// Bound by HBM with 4 waves of 32 columns and two workgroups a compute unit: 64 x 2,048 tokens at 32
// heads of 128 x 128, bf16, 946 us (4.3 GB, 4.5 TB/s; a large copy 5.15).  Chunks of 64 tokens on 8 waves of 16
// columns took 25% longer: q and k^T are
// read from LDS by every wave, and one barrier keeps all waves of a compute unit in step.  131,072 tokens of
// one sequence 1,130 to 1,176 us: 930 for the segments, 196 for what they add (a head that remembers is read
// twice: 1,390 us in all if no head forgets), 30 for the rest.

#include <algorithm>
#include <cmath>

#include "kda_attn.h"
#include "kda_lin.h"
#include "kda_mfma.h"

namespace kda {
namespace {

using mf::bf16_t;
using mf::bf16x4;
using mf::bf16x8;
using mf::f32x4;
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr float kLeastGate = -1e4f;   // e^-10000 is zero; sums of it stay exact to 2^-30 in fp64

// HV: value columns of a head; DV: those of a workgroup.
template <int DK_, int HV_, bool BF_, int DV_ = HV_>
struct Shape {
    static constexpr int DK = DK_, HV = HV_, DV = DV_;
    static constexpr bool BF = BF_;
    using O = mf::Ops<BF>;
    using T = typename O::T;
    static constexpr int C = 32, NT = C / 16;       // tokens per chunk, tiles of 16
    static constexpr int NW = BF ? 4 : DV / 16, THREADS = 64 * NW;
    static constexpr int NB = DV / 16 / NW;         // column tiles of a wave
    static_assert(NB == 1 || NB == 2);
    static constexpr int NKB = DK / 32;
    static constexpr int TERMS = BF ? 3 : 1;        // operand terms that hold an fp32 value
    static constexpr int E = 16 / sizeof(T);        // elements of a 16-byte piece
    static constexpr int NPK = C * DK / E / THREADS, NPV = C * DV / E / THREADS;
    static constexpr int KB = C * DK * sizeof(T), VB = C * DV * sizeof(T), PB = C * C * sizeof(T);
    static constexpr int DB = (4 * C + 4 + 2 * NW) * sizeof(float);   // decays of a chunk, and its rows that are not finite
    // At most two workgroups a compute unit, which is what the calls are cut for: where three or four fit they are dealt
    // out unevenly among few units (heads of 64, two / three: 32 of 8 x 2,048 tokens 101 / 120 us; 128 x 64, 8 / 32 of 64
    // ragged sequences to 8,000 tokens 475 / 517, but 32 of 200 x 700 64 x 64 612 / 597).  Of fp32 heads with dk 128
    // one fits (91 and 108 KB).
    static constexpr int LDS = std::max(4 * KB + 2 * VB + 2 * PB + 2 * DB, 56 * 1024);
    static constexpr int LDS_STATES = 2 * (KB + VB + DB);    // of the launch that forms the segments' states
    static_assert(C * DK % (E * THREADS) == 0 && C * DV % (E * THREADS) == 0);
    static_assert(LDS <= 160 * 1024);
};

// The wave's number, in a scalar register: branches on it change no lane masks.
__device__ __forceinline__ int wave_of() { return __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)); }

// Element x of row r of an LDS tile of W columns.  Its 16-byte pieces are permuted by the row so
// that neither 16 rows at one piece (operands along a row) nor 4 rows at 4 pieces (transposed
// ones) meet in a bank.
template <typename T, int W>
__device__ __forceinline__ int at(int r, int x) {
    constexpr int E = 16 / sizeof(T), PIECES = W / E;
    const int f = PIECES == 8 ? ((r & 2) << 1 | ((r >> 2) & 3)) : sizeof(T) == 2 ? ((r & 3) << 2 | ((r >> 2) & 3)) : r & 15;
    return r * W + ((x / E) ^ (PIECES == 4 ? f & 3 : f)) * E + x % E;
}

// A chunk's decays in LDS.
template <class X>
struct Decays {
    float *hi, *lo, *out, *keep;      // G / 2 in log2 (two floats), scale e^G, e^{G_C - G}
    float *all;                       // e^{G_C}
    uint32_t *odd_k, *odd_v;          // per wave: which rows of k and v that it put there hold infinities or NaN
    __device__ explicit Decays(char *p) {
        hi = (float *)p;
        lo = hi + X::C;
        out = lo + X::C;
        keep = out + X::C;
        all = keep + X::C;
        odd_k = (uint32_t *)(all + 4);
        odd_v = odd_k + X::NW;
    }
    // what any wave has set, the same for every thread
    static __device__ __forceinline__ uint32_t any(const uint32_t *waves) {
        uint32_t r = 0;
#pragma unroll
        for (int i = 0; i < X::NW; ++i) r |= waves[i];
        return __builtin_amdgcn_readfirstlane((int)r);
    }
};

// Transposed operand fragment from a row-major LDS tile of W columns: lane (m, g) gets
// one column of rows r0 + 8 g .. + 7.  STEP 4: column x0 + m; STEP 8: column x0 + 8 (m / 4) + m % 4.
// bf16: a 16-lane group loads 4 rows of 4 times 4 columns, and each lane gets one column of them.
template <class X, int W, int STEP>
__device__ __forceinline__ typename X::O::F8 ld_t(const typename X::T *tile, int r0, int x0) {
    const int lane = threadIdx.x & 63, m = lane & 15, r = r0 + 8 * (lane >> 4);
    if constexpr (X::BF) {
        typedef short s16x4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) s16x4 lds_t;
        const int x = x0 + STEP * (m & 3);
        const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t *)(tile + at<typename X::T, W>(r + (m >> 2), x)));
        const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t *)(tile + at<typename X::T, W>(r + 4 + (m >> 2), x)));
        return X::O::cat(__builtin_bit_cast(bf16x4, a), __builtin_bit_cast(bf16x4, b));
    } else {
        const int x = x0 + STEP * (m >> 2) + (m & 3);
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = tile[at<typename X::T, W>(r + e, x)];
        return X::O::cvt8(y);
    }
}

// Operand fragment along a row: elements x .. x + 7.
template <class X, int W>
__device__ __forceinline__ typename X::O::F8 ld_r(const typename X::T *tile, int r, int x) {
    using T = typename X::T;
    if constexpr (X::BF) return X::O::ld8(tile + at<T, W>(r, x));
    else return X::O::ld44(tile + at<T, W>(r, x), tile + at<T, W>(r, x + 4));
}

__device__ __forceinline__ bool not_finite(float x) { return (f32_bits(x) & 0x7f800000u) == 0x7f800000u; }

template <typename V>
__device__ __forceinline__ u32x4 words(V v) { return __builtin_bit_cast(u32x4, v); }

template <class X> struct Terms { typename X::O::F8 t[X::TERMS]; };

// Finite fp32 values as operand terms.  bf16: three times the upper half of what is left, which holds all
// 24 bits.
template <class X>
__device__ __forceinline__ Terms<X> terms8(const float *x) {
    Terms<X> r;
    if constexpr (X::BF) {
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = x[j];
#pragma unroll
        for (int t = 0; t < X::TERMS; ++t) {
            u32x4 u;
#pragma unroll
            for (int j = 0; j < 4; ++j) u[j] = __builtin_amdgcn_perm(f32_bits(y[2 * j + 1]), f32_bits(y[2 * j]), 0x07060302u);
            r.t[t] = __builtin_bit_cast(bf16x8, u);
            if (t + 1 < X::TERMS) {
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] -= bits_f32(f32_bits(y[j]) & 0xffff0000u);
            }
        }
    } else {
        r.t[0] = X::O::cvt8(x);
    }
    return r;
}

// Puts zeros in place of infinities and NaN.
template <class X>
__device__ __forceinline__ void clean(typename X::O::F8 *f) {
    float x[8];
    X::O::unpack8(*f, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = not_finite(x[e]) ? 0.f : x[e];
    *f = X::O::cvt8(x);
}

// 2^x of an fp64 x <= 0 or so, to about an ulp of fp32.  (The exponential instruction gives zeros below 2^-126.)
__device__ __forceinline__ float exp2_of(double x) {
    const float hi = (float)x;
    const float lo = (float)(x - (double)hi);
    const bool small = hi < -126.f;
    const float e = mf::ex2(small ? hi + 64.f : hi);
    const float r = e + e * (lo * 0.6931471805599453f);
    return hi < -150.f ? 0.f : small ? r * 0x1p-64f : r;
}

// Lane l - off of x in its row of 16 lanes, 0 before the row.
template <int OFF>
__device__ __forceinline__ double row_before(double x) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, 0x110 | OFF, 0xF, 0xF, true);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), 0x110 | OFF, 0xF, 0xF, true);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double lane_of(double x, int l) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)b, l), hi = __builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), l);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ double log2_decay(float g) {
    return (double)(g < kLeastGate ? kLeastGate : g) * 1.4426950408889634;   // NaN stays
}

// Log decays of a chunk's tokens (lane = token, zero behind the end) summed up to each, in log2.
template <class X>
__device__ __forceinline__ double summed(float g, double *all) {
    const int lane = threadIdx.x & 63;
    double x = log2_decay(g);
    x += row_before<1>(x);
    x += row_before<2>(x);
    x += row_before<4>(x);
    x += row_before<8>(x);
    double sum = lane_of(x, 15);
#pragma unroll
    for (int row = 1; row < X::C / 16; ++row) {
        if (lane >> 4 == row) x += sum;
        sum = lane_of(x, 16 * row + 15);
    }
    *all = sum;
    return x;
}

// The factor 2^x of a state.  A head with one decay for all tokens would have the same factor in every chunk, and its
// rounding would add up over some 1 / (1 - factor) of them (16,384 tokens at a decay of e^-0.00003: 10^-5).  So what the
// rounding of a factor near one left out goes into the next one.
__device__ __forceinline__ float state_factor(double x, float *left_out) {
    const float t = (float)(x * 0.6931471805599453) + *left_out;
    if (t > kSlow && t < 0x1p-20f) {
        const float m = expm1_small(t), f = 1.f + m;
        *left_out = m - (f - 1.f);
        return f;
    }
    *left_out = 0.f;
    return exp2_of(x);
}

// The decays of a chunk, by one wave.
template <class X>
__device__ __forceinline__ void write_decays(char *p, float g, float scale, float *left_out) {
    const int lane = threadIdx.x & 63;
    const Decays<X> s(p);
    double all;
    const double x = summed<X>(g, &all);
    if (lane < X::C) {
        const double half = 0.5 * x;
        s.hi[lane] = (float)half;
        s.lo[lane] = (float)(half - (double)(float)half);
        s.out[lane] = scale * exp2_of(x);
        s.keep[lane] = exp2_of(all - x);
    }
    const float f = state_factor(all, left_out);
    if (lane == 0) *s.all = f;
}

// 2^((G_i - G_j) / 2) of halves of G: its square reaches below the smallest normal number
template <class X>
__device__ __forceinline__ float decay_between(float hi_i, float lo_i, float hi_j, float lo_j) {
    const float d = hi_i - hi_j;
    if constexpr (X::BF) return mf::ex2(d + (lo_i - lo_j));   // P is rounded to bf16
    const float b = d - hi_i;                                 // what the subtraction rounded off
    const float e = mf::ex2(d);
    return e + e * (((hi_i - (d - b)) + (-hi_j - b) + (lo_i - lo_j)) * 0.6931471805599453f);
}

// Global memory from a uniform address on, `bytes` of it: loads behind them give zeros, stores are
// dropped.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t window(const char *p, int bytes) {
    const uint64_t u = (uint64_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)u), hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)(u >> 32));
    return __builtin_amdgcn_make_buffer_rsrc((void *)((uint64_t)hi << 32 | lo), 0, __builtin_amdgcn_readfirstlane(bytes), 0x00027000);
}
// `rows` rows of `width` bytes, `distance` apart (31 bits in all)
__device__ __forceinline__ __amdgpu_buffer_rsrc_t window(const char *p, int rows, int distance, int width) {
    return window(p, rows > 0 ? (rows - 1) * distance + width : 0);
}

// A tensor's rows of a unit, W columns of them, chunk after chunk.
template <class X, int W>
struct Source {
    using T = typename X::T;
    static constexpr int PIECES = W / X::E, N = X::C * PIECES / X::THREADS, STEP = X::THREADS / PIECES;
    static_assert(X::THREADS % PIECES == 0);
    const char *p;                    // the chunk's first row
    int row;                          // bytes between rows
    int offset;                       // of the thread's first piece
    __device__ __forceinline__ Source(const void *base, int64_t t, int64_t distance, int64_t off)
        : p((const char *)((const T *)base + t * distance + off)), row((int)distance * (int)sizeof(T)),
          offset(threadIdx.x / PIECES * row + threadIdx.x % PIECES * 16) {}
    __device__ __forceinline__ void step(int chunks) { p += (int64_t)row * (chunks * X::C); }
};

// Nothing that loads or stores global memory is moved across, so that the loads of all chunks leave in one order (where
// those before a loop had another one, waiting for a load in the loop waited for outputs too).
__device__ __forceinline__ void in_order() { __builtin_amdgcn_sched_barrier(0x78f); }

// A chunk's 16-byte pieces on their way from global memory to LDS.
template <class X, int W>
struct Rows {
    using S = Source<X, W>;
    u32x4 r[S::N];
    // `valid` rows (all of the chunk's at most), zeros behind them
    __device__ __forceinline__ void fetch(const S &s, int valid) {
        const auto w = window(s.p, valid, s.row, W * (int)sizeof(typename X::T));
#pragma unroll
        for (int i = 0; i < S::N; ++i) r[i] = __builtin_amdgcn_raw_buffer_load_b128(w, s.offset, i * S::STEP * s.row, 0);
        in_order();
    }
    __device__ __forceinline__ void put(typename X::T *tile) const {
#pragma unroll
        for (int i = 0; i < S::N; ++i) {
            const int q = threadIdx.x + i * X::THREADS;
            *(u32x4 *)(tile + at<typename X::T, W>(q / S::PIECES, q % S::PIECES * X::E)) = r[i];
        }
    }
    // Sets the wave's word to the rows of its pieces that hold infinities or NaN (which leave a NaN times zero).
    __device__ __forceinline__ void mark(uint32_t *waves) const {
        constexpr int ROWS = 64 / S::PIECES;                  // of a wave
        uint32_t rows = 0;
#pragma unroll
        for (int i = 0; i < S::N; ++i) {
            float x = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t u = r[i][j];
                x = fmaf(bits_f32(X::BF ? u & 0xffff0000u : u), 0.f, x);
                if (X::BF) x = fmaf(bits_f32(u << 16), 0.f, x);
            }
            const uint64_t lanes = __ballot(x != x);
#pragma unroll
            for (int l = 0; l < ROWS; ++l)
                if (lanes >> (l * S::PIECES) & ((1ull << S::PIECES) - 1)) rows |= 1u << (i * S::STEP + wave_of() * ROWS + l);
        }
        if ((threadIdx.x & 63) == 0) waves[wave_of()] = rows;
    }
};

// x, for the compiler another one in each turn of a loop: what follows from it is formed there and takes no registers
// elsewhere.
__device__ __forceinline__ int in_loop(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

// A wave's columns of the state: s[b][kb][hf][i] is row 32 kb + 8 gq + 4 hf + i, column col(b), of
// lane (m, gq).
template <class X>
struct State {
    static constexpr int SIZE = X::DK * X::HV;
    // With two tiles a wave's columns alternate by 4, so that a lane of the transposed outputs
    // holds 8 in a row.
    static constexpr int STEP = 4 * X::NB;
    f32x4 s[X::NB][X::NKB][2];
    static __device__ __forceinline__ int first() {
        const int lane = threadIdx.x & 63, m = lane & 15;
        return 8 * (lane >> 4) * X::HV + 16 * X::NB * wave_of() + STEP * (m >> 2) + (m & 3);
    }
    template <typename F>
    __device__ __forceinline__ void each(F f) {
        const int at = first();
#pragma unroll
        for (int b = 0; b < X::NB; ++b)
#pragma unroll
            for (int kb = 0; kb < X::NKB; ++kb)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) f(s[b][kb][hf], at + (32 * kb + 4 * hf) * X::HV + 4 * b);
    }
    __device__ __forceinline__ void load(const float *src) {   // null: zeros
        each([&](f32x4 &x, int) { x = f32x4{0.f, 0.f, 0.f, 0.f}; });
        if (src)
            each([&](f32x4 &x, int at) {
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = src[at + i * X::HV];
            });
    }
    __device__ __forceinline__ void store(float *dst) {
        each([&](f32x4 &x, int at) {
#pragma unroll
            for (int i = 0; i < 4; ++i) dst[at + i * X::HV] = x[i];
        });
    }
    // Whether k or v may have had an infinity or a NaN, the same for every thread: one of k leaves none of its row's
    // values finite and one of v none of its column's, and neither ever leaves the state again.
    __device__ __forceinline__ bool odd(uint32_t *waves) {
        float x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = i < X::NB ? s[i][0][0][0] * 0.f : 0.f;
#pragma unroll
        for (int kb = 0; kb < X::NKB; ++kb)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = fmaf(s[0][kb][hf][i], 0.f, x[i]);
        const float sum = (x[0] + x[1]) + (x[2] + x[3]);
        const bool mine = __any(sum != sum);
        if ((threadIdx.x & 63) == 0) waves[wave_of()] = mine;
        __syncthreads();
        return Decays<X>::any(waves);
    }
    // v^T of the wave's columns
    __device__ __forceinline__ static void values(const typename X::T *v, typename X::O::F8 *vf) {
#pragma unroll
        for (int b = 0; b < X::NB; ++b) vf[b] = ld_t<X, X::DV, STEP>(v, 0, 16 * X::NB * wave_of() + 4 * b);
    }
    // s += k^T (weights v) token by token: all of a token whose k has an infinity or a NaN (bits of odd_k), and columns of
    // one whose v has.
    __device__ __forceinline__ void add_rare(const typename X::T *k, const typename X::T *v, const float *keep, uint32_t odd_k,
                                             uint32_t odd_v) {
        for (uint32_t left = odd_k | odd_v; left; left &= left - 1) {
            const int j = __builtin_ctz(left), lane = in_loop(threadIdx.x & 63), m = lane & 15, gq = lane >> 4;
            const bool whole = odd_k >> j & 1;
            float x[X::NB];
            bool there[X::NB];
#pragma unroll
            for (int b = 0; b < X::NB; ++b) {
                x[b] = (float)v[at<typename X::T, X::DV>(j, 16 * X::NB * wave_of() + STEP * (m >> 2) + (m & 3) + 4 * b)];
                there[b] = whole || not_finite(x[b]);
                x[b] *= keep[j];
            }
#pragma unroll
            for (int kb = 0; kb < X::NKB; ++kb) {
                float y[8];
                X::O::unpack8(ld_r<X, X::DK>(k, j, 32 * kb + 8 * gq), y);
#pragma unroll
                for (int b = 0; b < X::NB; ++b)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        f32x4 &z = s[b][kb][e / 4];
                        const float t = z[e % 4] + y[e] * x[b];
                        z[e % 4] = there[b] ? t : z[e % 4];
                    }
            }
        }
    }
    // s += k^T (weights v), both finite: an infinite k that meets a term of v that is zero, or the zero that stands in for
    // an infinite v, would leave a NaN where k v is an infinity
    __device__ __forceinline__ void add(const typename X::T *k, const typename X::O::F8 *v, const float *keep) {
        float wt[8];
        mf::load8f(keep + 8 * ((threadIdx.x & 63) >> 4), wt);
        Terms<X> wv[X::NB];
#pragma unroll
        for (int b = 0; b < X::NB; ++b) {
            float x[8];
            X::O::unpack8(v[b], x);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= wt[e];
            wv[b] = terms8<X>(x);
        }
#pragma unroll
        for (int kb = 0; kb < X::NKB; ++kb)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const typename X::O::F8 kf = ld_t<X, X::DK, 8>(k, 0, 32 * kb + 4 * hf);
#pragma unroll
                for (int t = 0; t < X::TERMS; ++t)
#pragma unroll
                    for (int b = 0; b < X::NB; ++b) s[b][kb][hf] = X::O::mma32(s[b][kb][hf], kf, wv[b].t[t]);
            }
    }
};

// A sequence, and how it is cut.
struct Seq {
    int64_t c0;
    int len, segs;
    int first;        // c0 / seg
    __device__ __forceinline__ Seq(const LinArgs &a, int n) {
        const int begin = (int)min(max(a.cu[n], (int64_t)0), a.T), end = (int)min(max(a.cu[n + 1], (int64_t)0), a.T);
        c0 = __builtin_amdgcn_readfirstlane(begin);
        len = __builtin_amdgcn_readfirstlane(max(end - begin, 0));
        segs = 1;
        first = 0;
        if (a.seg) {
            first = (int)((uint32_t)c0 / (uint32_t)a.seg);
            segs = max((int)(((uint32_t)len + a.seg - 1) / (uint32_t)a.seg), 1);
        }
    }
};
__device__ __forceinline__ int seg_of(const LinArgs &a, int n) {
    return (int)((uint32_t)min(max(a.cu[n], (int64_t)0), a.T) / (uint32_t)a.seg);
}

template <int DK, int HV, bool BF, int DV>
__global__ __launch_bounds__((Shape<DK, HV, BF, DV>::THREADS), 2) void lin_kernel(const LinArgs a) {
    using X = Shape<DK, HV, BF, DV>;
    using O = typename X::O;
    using T = typename X::T;
    using F8 = typename O::F8;
    constexpr int C = X::C, NT = X::NT, NB = X::NB, NKB = X::NKB;
    extern __shared__ __align__(16) char lds[];
    T *const sq = (T *)lds, *const sk = (T *)(lds + 2 * X::KB), *const sv = (T *)(lds + 4 * X::KB);
    T *const sp = (T *)(lds + 4 * X::KB + 2 * X::VB);
    char *const sd = lds + 4 * X::KB + 2 * X::VB + 2 * X::PB;

    const int tid = threadIdx.x, lane = tid & 63, w = wave_of();
    const int m = lane & 15, gq = lane >> 4;
    const int x0 = blockIdx.x % (HV / DV) * DV;          // first of the workgroup's columns
    const int item = blockIdx.x / (HV / DV), unit = item / a.Hv, h = item - unit * a.Hv;
    const int hk = h / (a.Hv / a.Hk);
    const bool last = unit >= a.stretches;
    int n = unit - a.stretches;
    if (!last) n = last_not_above(a.N, unit, [&](int i) { return (int64_t)seg_of(a, i); });
    else if (a.order) n = a.order[n];
    const Seq seq(a, n);
    const int seg = last ? seq.segs - 1 : unit - seq.first;
    if (!last && (seg < 0 || seg + 1 >= seq.segs)) return;
    const int skip = seg * a.seg;                        // tokens before the unit
    const int len = last ? seq.len - skip : a.seg;
    const int64_t t0 = seq.c0 + skip;

    const float *src = seq.segs > 1 ? a.carry + (int64_t)(2 * seq.first + seg) * a.Hv * State<X>::SIZE
                                    : slot_of(a, a.read_idx, n, State<X>::SIZE);
    if (src) src += h * State<X>::SIZE + x0;
    State<X> S;

    // The unit from its first chunk to its last.  careful: infinities and NaN of k and v are added token by token.
    // A unit whose state ends with any is run once more so, from the same state and over the same outputs: a look at
    // k and v of every chunk took 5 to 12% of short prompts.
    auto pass = [&](auto careful) {
        constexpr bool CAREFUL = decltype(careful)::value;
        S.load(src);
        Source<X, DK> fq(a.q, t0, a.q_row, hk * DK), fk(a.k, t0, a.k_row, hk * DK);
        Source<X, DV> fv(a.v, t0, a.v_row, (int64_t)h * HV + x0);
        const char *fg = (const char *)(a.g + t0 * a.g_row + h);
        const int g_row = (int)a.g_row * 4, g_at = lane % C * g_row;
        struct Chunk { Rows<X, DK> q, k; Rows<X, DV> v; float g; };
        // the next chunk that has not been fetched; always as many loads, so that waiting for them waits for
        // nothing else
        auto fetch = [&](Chunk &r, int c) {
            const int valid = min(len - c * C, C);
            r.q.fetch(fq, valid);
            r.k.fetch(fk, valid);
            r.v.fetch(fv, valid);
            r.g = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(window(fg, valid, g_row, 4), g_at, 0, 0));
            fq.step(1);
            fk.step(1);
            fv.step(1);
            fg += (int64_t)g_row * C;
        };
        float left_out = 0.f;
        auto put = [&](const Chunk &r, int c) {
            r.q.put(sq + c % 2 * C * DK);
            r.k.put(sk + c % 2 * C * DK);
            r.v.put(sv + c % 2 * C * DV);
            if constexpr (CAREFUL) {
                const Decays<X> s(sd + c % 2 * X::DB);
                r.k.mark(s.odd_k);
                r.v.mark(s.odd_v);
            }
            if (w == X::NW - 1) write_decays<X>(sd + c % 2 * X::DB, lane % C < len - c * C ? r.g : 0.f, a.scale, &left_out);
        };

        const int col = 16 * NB * w + S.STEP * gq;           // first of the columns that the lane stores
        const int o_row = a.Hv * HV * (int)sizeof(T), o_at = m * o_row + col * (int)sizeof(T);
        const char *out = (const char *)((T *)a.o + (t0 * a.Hv + h) * HV + x0);
        // chunk c, whose rows are in LDS; `next` holds those of the one behind it, and takes those of the one further
        auto chunk = [&](int c, Chunk &next) {
            const int valid = min(len - c * C, C);
            const T *const q = sq + c % 2 * C * DK, *const v = sv + c % 2 * C * DV;
            T *const k = sk + c % 2 * C * DK, *const pt = sp + c % 2 * C * C;
            const Decays<X> s(sd + c % 2 * X::DB);

            F8 vf[NB];
            S.values(v, vf);

            // P^T tiles (rows j, columns i) of the first three waves (the last one has the decays of the next chunk to
            // form): lane holds 4 consecutive j of its i
            if (w < 3) {
                const int it = w > 0, jt = w > 1;
                const int i = 16 * it + m, j = 16 * jt + 4 * gq;
                f32x4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int kb = 0; kb < NKB; ++kb)
                    p = O::mma32(p, ld_r<X, DK>(k, 16 * jt + m, 32 * kb + 8 * gq), ld_r<X, DK>(q, i, 32 * kb + 8 * gq));
                const f32x4 hj = *(const f32x4 *)(s.hi + j), lj = *(const f32x4 *)(s.lo + j);
                const float hi = s.hi[i], li = s.lo[i];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float e = decay_between<X>(hi, li, hj[r], lj[r]);
                    p[r] = j + r <= i ? a.scale * (p[r] * e * e) : 0.f;
                }
                O::st4(pt + at<T, C>(i, j), p);
            }

            // o^T = e^G S^T q^T: lane holds token 16 it + m, four columns of each tile
            f32x4 acc[NT][NB];
#pragma unroll
            for (int it = 0; it < NT; ++it)
#pragma unroll
                for (int b = 0; b < NB; ++b) acc[it][b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb) {
                F8 sf[NB];
#pragma unroll
                for (int b = 0; b < NB; ++b) sf[b] = O::cvt44(S.s[b][kb][0], S.s[b][kb][1]);
#pragma unroll
                for (int it = 0; it < NT; ++it) {
                    const F8 qf = ld_r<X, DK>(q, 16 * it + m, 32 * kb + 8 * gq);
#pragma unroll
                    for (int b = 0; b < NB; ++b) acc[it][b] = O::mma32(acc[it][b], sf[b], qf);
                }
            }
#pragma unroll
            for (int it = 0; it < NT; ++it)
#pragma unroll
                for (int b = 0; b < NB; ++b) acc[it][b] *= s.out[16 * it + m];

            // S <- e^{G_C} S + k^T (weights v)
            const float all = *s.all;
            S.each([&](f32x4 &x, int) { x *= all; });
            uint32_t odd_k = 0, odd_v = 0;
            if constexpr (CAREFUL) {
                odd_k = s.any(s.odd_k);
                odd_v = s.any(s.odd_v);
            }
            if (odd_k | odd_v) {
                // They are added token by token, then zeros stand in for them: infinite values must not meet the zeros of P
                // above its diagonal, nor infinite keys the zero terms of a value.
                __syncthreads();
                for (uint32_t left = odd_k | odd_v; left; left &= left - 1) {
                    const int j = __builtin_ctz(left), i = in_loop(m), x0 = in_loop(col);
                    const bool whole = odd_k >> j & 1;
                    float y[NT];
#pragma unroll
                    for (int it = 0; it < NT; ++it) y[it] = (float)pt[at<T, C>(16 * it + i, j)];
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const float x = (float)v[at<T, DV>(j, x0 + 4 * b + r)];
                            const bool there = whole || not_finite(x);
#pragma unroll
                            for (int it = 0; it < NT; ++it) {
                                f32x4 &z = acc[it][b];
                                const float t = z[r] + y[it] * x;
                                z[r] = there && j <= 16 * it + i ? t : z[r];
                            }
                        }
                }
                S.add_rare(k, v, s.keep, odd_k, odd_v);
#pragma unroll
                for (int b = 0; b < NB; ++b) clean<X>(&vf[b]);
                __syncthreads();
                for (uint32_t left = odd_k; left; left &= left - 1) {
                    const int j = __builtin_ctz(left);
                    if (tid < DK) k[at<T, DK>(j, tid)] = (T)0.f;
                    if (tid < C) pt[at<T, C>(tid, j)] = (T)0.f;
                }
                __syncthreads();
            }
            S.add(k, vf, s.keep);

            if constexpr (CAREFUL) fetch(next, c + 1);   // no sooner: its registers are needed above
            put(next, c + 1);
            if constexpr (!CAREFUL) fetch(next, c + 2);
            __syncthreads();   // P and the next chunk are there

#pragma unroll
            for (int it = 0; it < NT; ++it) {
                const F8 pf = ld_r<X, C>(pt, 16 * it + m, 8 * gq);
#pragma unroll
                for (int b = 0; b < NB; ++b) acc[it][b] = O::mma32(acc[it][b], vf[b], pf);
            }
            const auto ow = window(out, valid, o_row, DV * (int)sizeof(T));
            out += (int64_t)o_row * C;
#pragma unroll
            for (int it = 0; it < NT; ++it) {
                if constexpr (!BF) {
                    __builtin_amdgcn_raw_buffer_store_b128(words(acc[it][0]), ow, o_at, 16 * it * o_row, 0);
                } else if constexpr (NB == 2) {
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, O::cvt44(acc[it][0], acc[it][1])), ow, o_at,
                                                           16 * it * o_row, 0);
                } else {
                    __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, O::cvt4(acc[it][0])), ow, o_at, 16 * it * o_row, 0);
                }
            }

            const int end = (c + 1) * C;
            if (valid == C && a.interval && (skip + end) % a.interval == 0)
                S.store(a.ckpt + (((a.ckpt_off ? a.ckpt_off[n] : 0) + (skip + end) / a.interval - 1) * a.Hv + h) * S.SIZE + x0);
        };

        if (w == 3) {                                        // P's upper tile, of both buffers
#pragma unroll
            for (int i = 0; i < 2; ++i) O::st4(sp + i * C * C + at<T, C>(m, 16 + 4 * gq), f32x4{0.f, 0.f, 0.f, 0.f});
        }
        if (len > 0) {
            Chunk next;
            fetch(next, 0);
            put(next, 0);
            if constexpr (!CAREFUL) fetch(next, 1);
            __syncthreads();
            for (int c = 0; c * C < len; ++c) chunk(c, next);
        }
    };
    pass(std::false_type());
    if (S.odd(Decays<X>(sd).odd_k)) {
        __syncthreads();                                 // all have read it
        pass(std::true_type());
    }

    if (last) {
        float *dst = slot_of(a, a.write_idx, n, S.SIZE);
        if (dst) S.store(dst + h * S.SIZE + x0);
    }
}

// Log2 decays of every 64 tokens of the segments that are formed in pieces.  One workgroup a
// block of tokens; a row of lanes takes a token's heads.
constexpr int kSum = 64, kSumThreads = 256;
__global__ __launch_bounds__(kSumThreads) void lin_sums_kernel(const LinArgs a) {
    __shared__ double s_sum[kSumThreads];
    const int blocks = a.seg / kSum;
    const int stretch = blockIdx.x / blocks, block = blockIdx.x - stretch * blocks;
    const int n = last_not_above(a.N, stretch, [&](int i) { return (int64_t)seg_of(a, i); });
    const Seq seq(a, n);
    const int seg = stretch - seq.first;
    if (seg < 0 || seg + 1 >= seq.segs) return;
    const int64_t t0 = seq.c0 + (int64_t)seg * a.seg + block * kSum;
    int row = 64;                     // lanes of a token: the smallest power of two that holds its heads
    while (row > 1 && row / 2 >= a.Hv) row /= 2;
    const int rows = kSumThreads / row, r = threadIdx.x / row;
    for (int h0 = 0; h0 < a.Hv; h0 += row) {
        const int h = h0 + threadIdx.x % row;
        double sum = 0.0;
        if (h < a.Hv) {
#pragma unroll 8
            for (int t = r; t < kSum; t += rows) sum += log2_decay(a.g[(t0 + t) * a.g_row + h]);
        }
        s_sum[threadIdx.x] = sum;
        __syncthreads();
        if (r == 0 && h < a.Hv) {
            for (int i = 1; i < rows; ++i) sum += s_sum[threadIdx.x + i * row];
            a.sums[(int64_t)blockIdx.x * a.Hv + h] = sum;
        }
        __syncthreads();
    }
}

// What a piece of a segment adds to the state at the segment's end, and the segment's decay.
// The weights count from that end, so the piece's chunks are walked backwards until nothing
// is left of a token (weights below 2^-150 are zero), and a piece of which nothing is left ends at once.
constexpr double kGone = -150.0;

template <int DK, int DV, bool BF>
__global__ __launch_bounds__((Shape<DK, DV, BF>::THREADS), BF ? 3 : 2) void lin_states_kernel(const LinArgs a) {
    using X = Shape<DK, DV, BF>;
    using T = typename X::T;
    constexpr int C = X::C;
    extern __shared__ __align__(16) char lds[];
    __shared__ double s_rest[2];      // log2 decay behind the chunk
    __shared__ double s_sum[X::NW];
    T *const sk = (T *)lds, *const sv = (T *)(lds + 2 * X::KB);
    char *const sd = lds + 2 * (X::KB + X::VB);

    const int lane = threadIdx.x & 63, w = wave_of();
    // heads that remember longest take most of the time: they come at another place in each unit's row, as
    // workgroups are dealt out to the compute units in turn
    const int unit = blockIdx.x / a.Hv, h = (blockIdx.x - unit * a.Hv + unit) % a.Hv;
    const int stretch = unit / a.pieces, piece = unit - stretch * a.pieces;
    const int hk = h / (a.Hv / a.Hk);
    // only the last sequence that starts in or before a stretch can have a segment here
    const int n = last_not_above(a.N, stretch, [&](int i) { return (int64_t)seg_of(a, i); });
    const Seq seq(a, n);
    const int seg = stretch - seq.first;
    if (seg < 0 || seg + 1 >= seq.segs) return;
    const int64_t t1 = seq.c0 + (int64_t)(seg + 1) * a.seg;   // the segment's end
    const int64_t t0 = t1 - a.seg + (int64_t)piece * a.piece;
    const int len = min(a.piece, (int)(t1 - t0));             // a multiple of 64

    // decay of the tokens behind the piece
    double rest = 0.0;
    if (piece + 1 < a.pieces) {
        const double *sums = a.sums + (int64_t)stretch * (a.seg / kSum) * a.Hv + h;
        for (int i = (piece + 1) * (a.piece / kSum) + threadIdx.x; i < a.seg / kSum; i += X::THREADS) rest += sums[(int64_t)i * a.Hv];
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) rest += __shfl_xor(rest, off);
        if (lane == 0) s_sum[w] = rest;
        __syncthreads();
        rest = 0.0;
#pragma unroll
        for (int i = 0; i < X::NW; ++i) rest += s_sum[i];
    }
    const int64_t kept = (int64_t)stretch * a.Hv + h, slot = (int64_t)unit * a.Hv + h;
    const bool gone = rest < kGone;
    if (threadIdx.x == 0) a.live[slot] = !gone;
    if (gone) {
        if (threadIdx.x == 0 && piece == 0) a.kept[kept] = 0.f;
        return;
    }
    const double behind = rest;

    State<X> S;
    // As in lin_kernel, but one body: the registers of two would leave room for two workgroups a compute unit, not three.
    bool careful = false;
    auto pass = [&]() {
        S.load(nullptr);
        rest = behind;
        const int chunks = len / C;
        Source<X, DK> fk(a.k, t0 + len - C, a.k_row, hk * DK);
        Source<X, DV> fv(a.v, t0 + len - C, a.v_row, (int64_t)h * DV);
        const char *fg = (const char *)(a.g + (t0 + len - C) * a.g_row + h);
        const int g_row = (int)a.g_row * 4, g_at = lane % C * g_row;
        struct Chunk { Rows<X, DK> k; Rows<X, DV> v; float g; };
        auto fetch = [&](Chunk &r, int c) {         // the c-th chunk from the end
            const int valid = c < chunks ? C : 0;
            r.k.fetch(fk, valid);
            r.v.fetch(fv, valid);
            r.g = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(window(fg, valid, g_row, 4), g_at, 0, 0));
            fk.step(-1);
            fv.step(-1);
            fg -= (int64_t)g_row * C;
        };
        auto put = [&](const Chunk &r, int c) {
            r.k.put(sk + c % 2 * C * DK);
            r.v.put(sv + c % 2 * C * DV);
            if (careful) {
                const Decays<X> s(sd + c % 2 * X::DB);
                r.k.mark(s.odd_k);
                r.v.mark(s.odd_v);
            }
            if (c % X::NW == w) {
                const Decays<X> s(sd + c % 2 * X::DB);
                double all;
                const double x = summed<X>(r.g, &all);
                const double after = c ? s_rest[(c - 1) % 2] : behind;
                if (lane < C) s.keep[lane] = exp2_of(after + (all - x));
                if (lane == 0) s_rest[c % 2] = after + all;
            }
        };

        Chunk next;
        fetch(next, 0);
        put(next, 0);
        fetch(next, 1);
        bool more = true;
        for (int c = 0; more; ++c) {
            __syncthreads();
            rest = s_rest[c % 2];
            more = c + 1 < chunks && !(rest < kGone);
            if (more) put(next, c + 1);
            fetch(next, c + 2);
            __builtin_amdgcn_sched_barrier(0);   // the loads leave before the products, which take long
            T *const k = sk + c % 2 * C * DK;
            const T *const v = sv + c % 2 * C * DV;
            const Decays<X> s(sd + c % 2 * X::DB);
            typename X::O::F8 vf[X::NB];
            S.values(v, vf);
            uint32_t odd_k = 0, odd_v = 0;
            if (careful) {
                odd_k = s.any(s.odd_k);
                odd_v = s.any(s.odd_v);
            }
            if (odd_k | odd_v) {
                S.add_rare(k, v, s.keep, odd_k, odd_v);
#pragma unroll
                for (int b = 0; b < X::NB; ++b) clean<X>(&vf[b]);
                __syncthreads();
                for (uint32_t left = odd_k; left; left &= left - 1)
                    if (threadIdx.x < DK) k[at<T, DK>(__builtin_ctz(left), threadIdx.x)] = (T)0.f;
                __syncthreads();
            }
            S.add(k, vf, s.keep);
        }
    };
    for (;;) {
        pass();
        if (careful || !S.odd(Decays<X>(sd).odd_k)) break;
        careful = true;
        __syncthreads();
    }
    S.store(a.part + slot * S.SIZE);
    if (threadIdx.x == 0 && piece == 0) {
        const float t = (float)(rest * 0.6931471805599453);
        a.kept[kept] = t > kSlow && t <= 0.f ? -fabsf(expm1_small(t)) : exp2_of(rest);
    }
}

// The incoming states of a split sequence's segments: four elements a thread, one segment
// after the other.
constexpr int kCarryThreads = 256, kMaxPieces = 4;
__global__ __launch_bounds__(kCarryThreads) void lin_carry_kernel(const LinArgs a, int size) {
    const int blocks = size / (4 * kCarryThreads);
    const int at = (blockIdx.x % blocks * kCarryThreads + threadIdx.x) * 4;
    const int stretch = blockIdx.x / blocks / a.Hv, h = blockIdx.x / blocks % a.Hv;
    const int n = last_not_above(a.N, stretch, [&](int i) { return (int64_t)seg_of(a, i); });
    const Seq seq(a, n);
    if (seq.first != stretch || seq.segs < 2) return;
    const float *src = slot_of(a, a.read_idx, n, size);
    f32x4 S = {0.f, 0.f, 0.f, 0.f};
    if (src) S = *(const f32x4 *)(src + (int64_t)h * size + at);
    float *dst = a.carry + ((int64_t)2 * stretch * a.Hv + h) * size + at;
    *(f32x4 *)dst = S;
    constexpr int G = 4;              // segments whose parts are on their way at once
    float kept[G];
    int live[G][kMaxPieces];
    auto look = [&](int s0) {
#pragma unroll
        for (int i = 0; i < G; ++i) {
            const int s = stretch + min(s0 + i, seq.segs - 2);
            kept[i] = a.kept[(int64_t)s * a.Hv + h];
#pragma unroll
            for (int p = 0; p < kMaxPieces; ++p)
                live[i][p] = p < a.pieces ? a.live[((int64_t)s * a.pieces + p) * a.Hv + h] : 0;
        }
    };
    look(0);
    for (int s0 = 0; s0 + 1 < seq.segs; s0 += G) {
        float keep[G];
        f32x4 part[G][kMaxPieces];
#pragma unroll
        for (int i = 0; i < G; ++i) {
            const int64_t s = stretch + min(s0 + i, seq.segs - 2);
            keep[i] = bits_f32(in_loop(f32_bits(kept[i])));   // its sign is not asked for in look(), which would wait
#pragma unroll
            for (int p = 0; p < kMaxPieces; ++p) {
                part[i][p] = f32x4{0.f, 0.f, 0.f, 0.f};
                if (live[i][p]) part[i][p] = *(const f32x4 *)(a.part + ((s * a.pieces + p) * a.Hv + h) * size + at);
            }
        }
        look(s0 + G);
        auto carry = [&](auto careful) {      // careful: with infinities
            f32x4 x = S;
#pragma unroll
            for (int i = 0; i < G; ++i) {
                const bool slow = f32_bits(keep[i]) >> 31;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    x[j] = decltype(careful)::value ? decayed(x[j], keep[i], slow) : fmaf(x[j], keep[i], slow ? x[j] : 0.f);
#pragma unroll
                for (int p = 0; p < kMaxPieces; ++p) x += part[i][p];
                if (s0 + i + 1 < seq.segs) *(f32x4 *)(dst + (i + 1) * (int64_t)a.Hv * size) = x;
            }
            return x;
        };
        f32x4 x = carry(std::false_type());
        const f32x4 none = x * 0.f;           // NaN where it is not finite
        const float sum = (none[0] + none[1]) + (none[2] + none[3]);
        if (sum != sum) x = carry(std::true_type());
        S = x;
        dst += G * (int64_t)a.Hv * size;
    }
}

template <typename K>
hipError_t start(K *kernel, int64_t grid, int threads, int lds, const LinArgs &a, hipStream_t s) {
    const hipError_t e = hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(threads), lds, s, a);
    return hipGetLastError();
}

// Sequences by the length of their last segment, the longest first: workgroups start in this
// order, and the short ones fill up what the long ones leave.
constexpr int kOrderThreads = 1024;
__global__ __launch_bounds__(kOrderThreads) void lin_order_kernel(const LinArgs a) {
    __shared__ int s_len[kOrderThreads];
    const int n = threadIdx.x;
    int len = 0;
    if (n < a.N) {
        const int begin = (int)min(max(a.cu[n], (int64_t)0), a.T), end = (int)min(max(a.cu[n + 1], (int64_t)0), a.T);
        len = max(end - begin, 0);
        if (a.seg && len > a.seg) len -= (len - 1) / a.seg * a.seg;
    }
    s_len[n] = len;
    __syncthreads();
    if (n >= a.N) return;
    int rank = 0;
    for (int i = 0; i < a.N; ++i) rank += s_len[i] > len || (s_len[i] == len && i < n);
    a.order[rank] = n;
}

template <int DK, int DV, bool BF>
hipError_t launch(const LinArgs &a, hipStream_t s) {
    using X = Shape<DK, DV, BF>;
    if (a.order) {
        hipLaunchKernelGGL(lin_order_kernel, dim3(1), dim3(kOrderThreads), 0, s, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (a.seg) {
        hipError_t e = hipSuccess;
        if (a.pieces > 1) {
            const int64_t blocks = (int64_t)a.stretches * (a.seg / kSum);
            hipLaunchKernelGGL(lin_sums_kernel, dim3((unsigned)blocks), dim3(kSumThreads), 0, s, a);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }
        e = start(lin_states_kernel<DK, DV, BF>, (int64_t)a.stretches * a.pieces * a.Hv, X::THREADS, X::LDS_STATES, a, s);
        if (e != hipSuccess) return e;
        const int64_t grid = (int64_t)a.stretches * a.Hv * (DK * DV / (4 * kCarryThreads));
        hipLaunchKernelGGL(lin_carry_kernel, dim3((unsigned)grid), dim3(kCarryThreads), 0, s, a, DK * DV);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    const int64_t heads = ((int64_t)a.stretches + a.N) * a.Hv;
    if constexpr (BF && DV == 128)
        if (a.narrow) {
            using Y = Shape<DK, DV, BF, 64>;
            return start(lin_kernel<DK, DV, BF, 64>, heads * 2, Y::THREADS, Y::LDS, a, s);
        }
    return start(lin_kernel<DK, DV, BF, DV>, heads, X::THREADS, X::LDS, a, s);
}

// Pieces of fewer tokens cost more than they save: 32 heads, segments of 1,024 tokens in one piece / two 198 / 212 us (16,384
// tokens).  Of longer ones they cost where heads remember and save where they forget: one / two to four, 65,536 tokens
// 695 / 754 and 653 / 633 us, 131,072 1,367 / 1,414 and 1,276 / 1,168.
constexpr int kLeastPiece = 1024;
// Tokens of a sequence on average from which the order pays for its launch: 200 ragged sequences of 100 to 3,000 tokens at
// 32 heads 1,238 us as they come, 1,158 in order; 64 of 64 to 512 125.5 / 124.2; 64 of 60 61 / 65.
constexpr int kLeastOrdered = 128;

}  // namespace

namespace {
void cut(int cus, bool bf16, int dv, LinArgs *a) {
    a->seg = a->slots = a->stretches = a->piece = a->pieces = 0;
    a->order = nullptr;
    a->ordered = a->N > 1 && a->N <= kOrderThreads && (int64_t)a->N * a->Hv > 2 * cus && a->T / a->N >= kLeastOrdered;
    // Where it pays to cut, the segments give every compute unit its two workgroups, but:
    //  - at least 2 sqrt(T) tokens: a segment takes about 4 us per 32 tokens in its two launches, and each
    //    one lengthens the carry by about 0.5 us (one head, 4,096 tokens: 41 us with segments of 64, 34 of 128,
    //    41 of 256; 16,384: 114, 71, 59);
    //  - at least 4 tokens a head: a segment's state is written and read twice (32 heads, 1,024 tokens: 44 us with
    //    segments of 64, 39 of 128);
    //  - six of the shortest ones at least for bf16 heads of 128 columns, or the additional launches cost what they
    //    save (in one / cut: 32 heads, 512 tokens 25 / 31 us, 768 35 / 35, 1,024 47 / 42; one head, 384 19 / 20, 512
    //    24 / 20), four for the others, whose states are smaller or chunks slower (32 heads of 64 x 64, 512 tokens:
    //    20 / 20; fp32 heads of 128 x 128: 100 / 56), and three of any (256 heads leave each compute unit one
    //    workgroup in one piece, and halves take as long);
    //  - among several sequences the longest one may have from T / N to T tokens: half as many again of those halfway
    //    (32 heads, 2 x 512 tokens 26 / 43 us, but 47 / 42 if one has all; 8 x 512 42 / 81, but 163 / 75);
    //  - none where the sequences are shorter than a quarter of one on average, so that few can be longer than one (32
    //    heads, 64 x 60 tokens 61 us whole, 73 cut); those between pay for one that may be long (8 heads, 64 x 60 18.6 /
    //    25.7, but 234 / 54 if one has 3,777 of the tokens).
    // Fp32 heads with dk 128, one workgroup a compute unit, are cut for two as well (for two / one, dv 128: 8 heads of
    // 8,192 tokens 149 / 154 us, 32 of 2,048 118 / 98).
    const int64_t per_head = std::max(2 * cus / a->Hv, 1);
    const int64_t least = std::max((int64_t)4 * a->Hv, (int64_t)std::ceil(2.0 * std::sqrt((double)a->T)));
    const int64_t seg = (std::max((a->T + per_head - 1) / per_head, least) + 63) / 64 * 64;
    const int64_t longest = (a->T + a->T / a->N) / 2, fewest = (bf16 && dv == 128 ? 6 : 4) * (a->N > 1 ? 3 : 2);
    if (2 * longest < fewest * ((least + 63) / 64 * 64) || a->T < 3 * seg || a->T / a->N < seg / 4) return;
    a->seg = (int32_t)seg;
    a->stretches = (int32_t)(a->T / seg);
    a->slots = 2 * a->stretches;
    const int32_t pieces = (int32_t)std::max<int64_t>(std::min<int64_t>(kMaxPieces, seg / kLeastPiece), 1);
    a->piece = ((a->seg + pieces - 1) / pieces + 63) / 64 * 64;
    a->pieces = (a->seg + a->piece - 1) / a->piece;
}

}  // namespace

void lin_plan(int cus, bool bf16, int dv, LinArgs *a) {
    cut(cus, bf16, dv, a);
    // A workgroup alone on its compute unit takes 28% less time for half of the columns (32 heads, 257 tokens: 22.6 ->
    // 16.3 us); where there are enough, q and k would be read and multiplied twice for nothing.
    a->narrow = (int64_t)(a->stretches + a->N) * a->Hv * 2 <= cus;
}

// The buffers, from the largest alignment to the smallest.
size_t lin_buffers(int dk, int dv, char *ws, LinArgs *a) {
    const size_t state = (size_t)dk * dv * sizeof(float) * a->Hv, pieces = (size_t)a->stretches * a->pieces;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char *const p = ws + at;
        at += bytes;
        return p;
    };
    a->carry = (float *)take(a->slots * state);
    a->part = (float *)take(pieces * state);
    a->sums = (double *)take(a->pieces > 1 ? (size_t)a->stretches * (a->seg / kSum) * a->Hv * sizeof(double) : 0);
    a->kept = (float *)take((size_t)a->stretches * a->Hv * sizeof(float));
    a->live = (int32_t *)take(pieces * a->Hv * sizeof(int32_t));
    char *const order = take(a->ordered ? a->N * sizeof(int32_t) : 0);
    if (a->ordered) a->order = (int32_t *)order;
    return at;
}

bool lin_supported(int dk, int dv) { return (dk == 64 || dk == 128) && (dv == 64 || dv == 128); }

hipError_t launch_lin(bool bf16, int dk, int dv, const LinArgs &a, hipStream_t s) {
    if (a.N <= 0) return hipSuccess;
#define KDA_LIN(DK_, DV_)                                                                  \
    if (dk == DK_ && dv == DV_) return bf16 ? launch<DK_, DV_, true>(a, s) : launch<DK_, DV_, false>(a, s);
    KDA_LIN(64, 64)
    KDA_LIN(64, 128)
    KDA_LIN(128, 64)
    KDA_LIN(128, 128)
#undef KDA_LIN
    return hipErrorInvalidValue;
}

}  // namespace kda
