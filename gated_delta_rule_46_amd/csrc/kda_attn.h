// Internal interfaces of the attention-layer operators with the C ABI
// (kda_api.hip): q/k norm with rotation (kda_rotate.hip), the 8-bit key/value
// cache (kda_kv.hip) and attention over it (kda_attn.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda_internal.h"

namespace kda {

// RMS norm of every head of q and k with the rotation (kda_rotate.hip).
struct RotateArgs {
    const void *q, *k;           // rows of Hq (Hk) heads of D, I/O dtype
    void *q_out, *k_out;
    int64_t q_row, k_row, q_out_row, k_out_row;   // elements from token to token
    const float *q_weight, *k_weight;             // [D] (nullable: ones)
    const float *table;          // [n_pos, rot]: cosines, then sines (nullable: no rotation)
    const int64_t *positions;    // [T] (nullable without a table)
    int64_t T, n_pos;
    int32_t Hq, Hk, rot;
    float eps;
};
hipError_t launch_rotate(bool bf16, int D, bool pairs, const RotateArgs &a, hipStream_t s);

// A paged key/value cache and the tokens of a call: sequence n's are the last
// cu[n+1] - cu[n] of its kv_len[n] cached tokens, and the token at position p
// lives in row p % page of page table[n * width + p / page].
struct KvArgs {
    uint8_t *k_codes, *v_codes;  // [n_pages, Hk, page, D] e4m3
    float *k_scale, *v_scale;    // [n_pages, Hk]
    const int32_t *table;        // [N, width]
    int64_t n_pages;
    int32_t page, width;
    const int64_t *cu, *kv_len;  // [N+1], [N]
    int32_t N, Hk;
    int64_t T;
    const void *k, *v;           // kda_kv_write: rows of Hk heads, I/O dtype
    int64_t k_row, v_row;
    void *k_out, *v_out;         // kda_kv_read: [T, Hk, D], I/O dtype
};
hipError_t launch_kv_write(bool bf16, int D, const KvArgs &a, hipStream_t s);
hipError_t launch_kv_read(bool bf16, int D, const KvArgs &a, hipStream_t s);

// Attention over the cache (kda_attn.hip).
struct AttnArgs {
    KvArgs kv;
    const void *q;               // rows of Hq heads, I/O dtype
    int64_t q_row;
    void *o;                     // [T, Hq, D], I/O dtype
    float *lse;                  // [T, Hq] (nullable)
    float *part;                 // partial results of split units
    int32_t Hq;
    float scale;                 // of the scores, times log2(e): its size, at least the smallest normal
    float q_sign;                // its sign, which the queries take: -1, 0 or 1
    int32_t causal, window;
    // sequences of at most short_rows query rows per kv head go to kda_attn.hip,
    // the others to kda_attn_rows.hip
    int32_t short_rows;
    int32_t unit_rows;           // kda_attn.hip: rows per unit, 16 or 32
    int32_t workers;             // kda_attn.hip: workgroups that share the tiles; 0: one per
                                 // unit; -1: not launched
    int32_t row_units;           // kda_attn_rows.hip: units per kv head, 0: not launched
    int32_t row_splits;          // workgroups per unit at most
    int32_t split_tiles;         // one for each so many tiles of 64 keys
    int32_t row_fold;            // units from the last one that start in order, the others after them
};
// The plan of a call (short_rows, workers, row_units, row_splits) and the bytes
// of its partial results.
void attn_plan(int cus, bool bf16, int D, int N, int64_t T, int Hq, int Hk, int64_t max_kv, AttnArgs *a);
size_t attn_partial_bytes(int D, const AttnArgs &a);
hipError_t launch_attn(bool bf16, int D, const AttnArgs &a, hipStream_t s);
hipError_t launch_attn_rows(bool bf16, int D, const AttnArgs &a, hipStream_t s);

// Two fp32 values per half word of e4m3 codes (round to nearest even).
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
    uint32_t r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return __builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
}

__device__ __forceinline__ void uncode4(uint32_t c, float *out) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(c, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(c, true);
    out[0] = a[0]; out[1] = a[1]; out[2] = b[0]; out[3] = b[1];
}

// 8 consecutive elements that are not read again, past the caches (6 to 8% of the time
// of a call that streams its rows; such stores cost 20%).
template <bool BF> __device__ __forceinline__ void load8_once(const void *base, int64_t i, float *out) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    if (BF) {
        const u32x4 w = __builtin_nontemporal_load((const u32x4 *)((const uint16_t *)base + i));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            out[2 * j] = bits_f32(w[j] << 16);
            out[2 * j + 1] = bits_f32(w[j] & 0xffff0000u);
        }
    } else {
        typedef float f32x4 __attribute__((ext_vector_type(4)));
        const f32x4 a = __builtin_nontemporal_load((const f32x4 *)((const float *)base + i));
        const f32x4 b = __builtin_nontemporal_load((const f32x4 *)((const float *)base + i + 4));
#pragma unroll
        for (int j = 0; j < 4; ++j) { out[j] = a[j]; out[4 + j] = b[j]; }
    }
}
// The last n in [0, N) with first(n) <= x, 0 if there is none, for a first that does
// not decrease: 64 probes at a time by the whole wave (x the same in all lanes).
template <typename F>
__device__ __forceinline__ int last_not_above(int N, int64_t x, F first) {
    const int lane = threadIdx.x & 63;
    int lo = 0;
    for (int size = N; size > 1;) {
        const int step = (size + 63) / 64, at = lane * step;
        const bool le = at < size && first(lo + at) <= x;
        const int k = max(__popcll(__ballot(le)), 1) - 1;
        lo += k * step;
        size = min(step, size - k * step);
    }
    return lo;
}

}  // namespace kda
