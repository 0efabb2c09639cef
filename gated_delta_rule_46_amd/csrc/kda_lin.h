// kda_lin.h -- internal interfaces of the linear-attention layer (one decay per
// head): prefill (kda_lin.hip), one-token step (kda_lin_step.hip) and the
// norm of the heads (kda_headnorm.hip) with the C ABI (kda_api.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda_internal.h"

namespace kda {

struct LinArgs {
    const void *q, *k, *v;       // rows of Hk heads of dk, Hk of dk, Hv of dv, io dtype
    int64_t q_row, k_row, v_row; // distance between tokens, elements
    const float *g;              // log decays: g[t * g_row + h] (g_row = 0: one per head)
    int64_t g_row;
    void *o;                     // [T,Hv,dv]
    const int64_t *cu;           // [N+1]
    int64_t T;
    int32_t N, Hk, Hv;
    float scale;
    float *pool;                 // [n_slots,Hv,dk,dv] (nullable)
    int64_t n_slots;
    const int32_t *read_idx, *write_idx;   // [N] (nullable)
    int32_t interval;            // checkpoint interval in tokens, 0 = none
    const int64_t *ckpt_off;     // first rung row per sequence (nullable for N = 1)
    float *ckpt;                 // rung rows
    // Sequences longer than `seg` tokens in segments of so many (0: none is split).  Segment s of a
    // sequence that starts at token c lies in stretch c / seg + s: no two segments with another behind
    // them share one, whatever the lengths are.  A unit is such a stretch, or the last segment of a sequence.
    // A split sequence's segment finds its incoming state at slot 2 (c / seg) + s.  What a segment adds to the
    // state is formed in `pieces` pieces of `piece` tokens.
    int32_t seg, slots, stretches;          // slots: 2 (T / seg); stretches: T / seg
    int32_t piece, pieces;
    bool ordered;                // whether there is an order
    bool narrow;                 // whether a head's columns are shared out over two workgroups
    int32_t *order;              // [N] sequences by the length of their last segment (null: as they come)
    float *carry;                // [slots,Hv,dk,dv]
    float *part;                 // [stretches,pieces,Hv,dk,dv]
    float *kept;                 // [stretches,Hv] decay over a segment: e^G, or e^G - 1 with its sign where G is near 0
    int32_t *live;               // [stretches,pieces,Hv] whether the piece adds anything
    double *sums;                // [stretches,seg/64,Hv] log2 decays of 64 tokens (with more than one piece)
};
// The plan of a call on a device of `cus` compute units; its buffers at ws, and their bytes.
void lin_plan(int cus, bool bf16, int dv, LinArgs *a);
size_t lin_buffers(int dk, int dv, char *ws, LinArgs *a);
bool lin_supported(int dk, int dv);
hipError_t launch_lin(bool bf16, int dk, int dv, const LinArgs &a, hipStream_t s);
// one token per sequence: T and cu unused
hipError_t launch_lin_step(bool bf16, int dk, int dv, const LinArgs &a, hipStream_t s);

// Norm of every head with an activation.
struct HeadNormArgs {
    const void *x, *gate;        // rows of H heads of D, io dtype (gate nullable)
    void *y;
    int64_t x_row, gate_row, y_row;
    const float *weight, *bias;  // [D], or [H,D] with per_head (nullable)
    int64_t T;
    int32_t H, D;
    int32_t per_head, center, act;
    float eps;
};
constexpr int kHeadNormMaxDim = 1024;
hipError_t launch_head_norm(bool bf16, const HeadNormArgs &a, hipStream_t s);

// Slot of the state pool that sequence n reads (writes); null if it has none.
__device__ __forceinline__ float *slot_of(const LinArgs &a, const int32_t *idx, int n, int64_t state) {
    if (!idx) return nullptr;
    const int64_t i = idx[n];
    return i >= 0 && i < a.n_slots ? a.pool + i * a.Hv * state : nullptr;
}

// e^t - 1 for t within 1/8 of zero: the terms left out are below 2^-30 of it.  (e^t as a float keeps few bits of it where
// t is near zero, and one decay for all tokens would add up the same error with every one of them.)
constexpr float kSlow = -0.125f;
__device__ __forceinline__ float expm1_small(float t) {
    return t + t * t * (1.f / 2 + t * (1.f / 6 + t * (1.f / 24 + t * (1.f / 120 + t * (1.f / 720)))));
}

// A state's value behind a decay: keep is e^g, or e^g - 1 where slow (an infinity stays one).
__device__ __forceinline__ float decayed(float s, float keep, bool slow) {
    const float r = fmaf(s, keep, slow ? s : 0.f);
    return slow && fabsf(s) == __builtin_inff() ? s : r;
}

}  // namespace kda
