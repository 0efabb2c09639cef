// kda_attn_ops.h -- what the attention kernels share (kda_attn.hip,
// kda_attn_rows.hip): a sequence as they see it, codes to bf16, fp32 as bf16 terms.
#pragma once

#include "kda_attn.h"
#include "kda_mfma.h"

namespace kda {
namespace attn {

using mf::bf16_t;
using mf::bf16x8;
using mf::f32x4;
typedef bf16_t bf16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kAttnThreads = 256;
constexpr int kWaves = kAttnThreads / 64;
constexpr int kTile = 64;             // keys per step of kda_attn_rows.hip
constexpr int kStep = 32;             // and of kda_attn.hip
constexpr int kUnitCost = 12;         // steps that starting and ending a unit there costs
constexpr int kRows = 16;             // query rows (token, head of the group) of a block; kda_attn.hip: 1 or 2 a unit
constexpr int kRowTile = 128;         // and of kda_attn_rows.hip
constexpr float kLn2 = 0.6931471805599453f;

// bf16 pairs of bytes (0, 1) or (2, 3) of four codes, times 2^(scale's exponent)
template <bool HI>
__device__ __forceinline__ uint32_t widen(uint32_t c, float scale) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, scale, HI));
}

// A sequence as the kernels see it.  Positions are clamped to what the table can
// hold (31 bits), on the far side of every key.
struct Seq {
    int64_t c0;       // first packed token
    int64_t pos0;     // position of the first new token
    int kvl;          // cached tokens that the table can hold
    int len;
    int rt;           // units of unit_rows rows per kv head (0: the other kernel's)
    int lo, steps;    // first step that some row sees; steps of a unit, kUnitCost among them

    // keys that new token i sees: begin_of(i) <= j < end_of(i)
    __device__ __forceinline__ int end_of(const AttnArgs &a, int i) const {
        return a.causal ? (int)max(min(pos0 + i + 1, (int64_t)kvl), (int64_t)0) : kvl;
    }
    __device__ __forceinline__ int begin_of(const AttnArgs &a, int i) const {
        return a.window > 0 ? (int)max(min(pos0 + i + 1 - a.window, (int64_t)kvl), (int64_t)0) : 0;
    }
    // (unit, step) pairs of the sequence
    __device__ __forceinline__ int64_t cost(const AttnArgs &a) const { return (int64_t)a.kv.Hk * rt * steps; }
};

__device__ __forceinline__ Seq sequence(const AttnArgs &a, int n, int G) {
    Seq s = {};
    if (n >= a.kv.N) return s;
    s.c0 = a.kv.cu[n];
    const int64_t c1 = min(a.kv.cu[n + 1], a.kv.T);
    const int64_t kv = a.kv.kv_len[n];
    s.len = s.c0 < 0 ? 0 : (int)max(c1 - s.c0, (int64_t)0);
    s.pos0 = kv - s.len;
    s.kvl = (int)max(min(kv, (int64_t)a.kv.width * a.kv.page), (int64_t)0);
    s.rt = (int64_t)s.len * G <= a.short_rows ? (s.len * G + a.unit_rows - 1) / a.unit_rows : 0;
    s.lo = s.begin_of(a, 0) / kStep;
    s.steps = (s.kvl + kStep - 1) / kStep - s.lo + kUnitCost;
    return s;
}

// Over lanes l and l ^ 32, and over the four groups of 16 lanes.
__device__ __forceinline__ float max_32(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(f32_bits(x), f32_bits(x), false, false);
    return fmaxf(bits_f32(r[0]), bits_f32(r[1]));
}
__device__ __forceinline__ float sum_32(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(f32_bits(x), f32_bits(x), false, false);
    return bits_f32(r[0]) + bits_f32(r[1]);
}
__device__ __forceinline__ float max_16(float x) {
    const auto r = __builtin_amdgcn_permlane16_swap(f32_bits(x), f32_bits(x), false, false);
    return max_32(fmaxf(bits_f32(r[0]), bits_f32(r[1])));
}
__device__ __forceinline__ float sum_16(float x) {
    const auto r = __builtin_amdgcn_permlane16_swap(f32_bits(x), f32_bits(x), false, false);
    return sum_32(bits_f32(r[0]) + bits_f32(r[1]));
}

// log sum exp from a maximum (log2) and a sum
__device__ __forceinline__ float lse_of(float m, float l) {
    return l == 0.f ? -__builtin_inff() : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

// A operand of V^T for dims (D / 16) m + 4 w + b of token groups g, g + 1.
template <int B>
__device__ __forceinline__ bf16x8 v_frag(const uint32_t (&t)[8], float s0, float s1) {
    // byte B of two tokens side by side: the low pair for even B, the high one for odd
    constexpr uint32_t sel = B < 2 ? 0x05010400u : 0x07030602u;
    constexpr bool HI = B & 1;
    u32x4 r;
    r[0] = widen<HI>(__builtin_amdgcn_perm(t[1], t[0], sel), s0);
    r[1] = widen<HI>(__builtin_amdgcn_perm(t[3], t[2], sel), s0);
    r[2] = widen<HI>(__builtin_amdgcn_perm(t[5], t[4], sel), s1);
    r[3] = widen<HI>(__builtin_amdgcn_perm(t[7], t[6], sel), s1);
    return __builtin_bit_cast(bf16x8, r);
}

template <int NS> struct Frag { bf16x8 f[NS]; };

// fp32 values as NS bf16 terms
template <int NS>
__device__ __forceinline__ Frag<NS> split8(const float *x) {
    Frag<NS> r;
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = x[j];
#pragma unroll
    for (int t = 0; t < NS; ++t)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const bf16_t h = (bf16_t)y[j];
            r.f[t][j] = h;
            if (t + 1 < NS) y[j] -= (float)h;
        }
    return r;
}

// The same for queries, which can be infinite, or so large that the first term would be
// rounded to an infinity (what is left of x would then be a NaN): an infinity is its
// first term alone, and the largest values are cut instead of rounded.
template <int NS>
__device__ __forceinline__ Frag<NS> split_query8(const float *x) {
    if constexpr (NS == 1) return split8<1>(x);
    Frag<NS> r;
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t b = f32_bits(x[j]), mag = b & 0x7fffffffu;
        const bool cut = mag >= 0x7f7f8000u && mag <= 0x7f800000u;
        const bf16_t h = (bf16_t)(cut ? bits_f32(b & 0xffff0000u) : x[j]);
        r.f[0][j] = h;
        y[j] = mag == 0x7f800000u ? 0.f : x[j] - (float)h;
    }
    if constexpr (NS > 1) {
        const Frag<NS - 1> rest = split8<NS - 1>(y);
#pragma unroll
        for (int t = 1; t < NS; ++t) r.f[t] = rest.f[t - 1];
    }
    return r;
}

__device__ __forceinline__ uint32_t nan_bytes(uint32_t c) {   // 0x80 in every byte that is a NaN code
    return ((c & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

// NaN if byte y of nan_bytes() is set, else 0 (no comparison: those would hold a
// lane mask each).
__device__ __forceinline__ float nan_or_zero(uint32_t b, int y) {
    return bits_f32((uint32_t)((int32_t)(b << (24 - 8 * y)) >> 31) & 0x7fc00000u);
}

}  // namespace attn
}  // namespace kda
