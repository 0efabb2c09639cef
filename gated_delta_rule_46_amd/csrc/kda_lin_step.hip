// kda_lin_step.hip -- linear attention with one decay per head, one token of each
// sequence against a pool of states:
//     S <- e^g S + k v^T,    o = scale S^T q
//
// The state is read and written once (64 KiB of fp32 a head at dk = dv = 128) and all
// else is small beside it: bound by HBM.  One workgroup of four waves takes 64 columns
// of a (sequence, head): lane (cq, ro) of wave w owns columns 4 cq .. 4 cq + 3 and rows
// 16 j + 4 w + ro, in registers from the read to the write, so that a wave's load covers
// four 256-byte row segments.  The rows are asked for before anything else; q and k go
// through LDS, as each lane needs them at its rows.  64 sequences at 32 heads of 128 x 128: 54 us
// (270 MB, 5.0 TB/s; a large copy 5.15); one sequence 4 us, the launch.

#include "kda_lin.h"
#include "kda_mfma.h"

namespace kda {
namespace {

using mf::f32x4;

constexpr int kStepThreads = 256;
constexpr int kStepCols = 64;

template <bool BF>
__device__ __forceinline__ float load1(const void *p, int64_t i) {
    if (BF) return bits_f32((uint32_t)((const uint16_t *)p)[i] << 16);
    return ((const float *)p)[i];
}

template <bool BF>
__device__ __forceinline__ f32x4 load4(const void *p, int64_t i) {
    if (BF) {
        const uint2 w = *(const uint2 *)((const uint16_t *)p + i);
        return f32x4{bits_f32(w.x << 16), bits_f32(w.x & 0xffff0000u), bits_f32(w.y << 16), bits_f32(w.y & 0xffff0000u)};
    }
    return *(const f32x4 *)((const float *)p + i);
}

template <int DK, int DV, bool BF>
__global__ __launch_bounds__(kStepThreads) void step_kernel(const LinArgs a) {
    constexpr int NCB = DV / kStepCols;
    constexpr int NS = DK / 16;   // row steps of a lane
    constexpr int64_t state = (int64_t)DK * DV;
    __shared__ float s_q[DK], s_k[DK];
    __shared__ __align__(16) float s_o[4][kStepCols];

    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int cq = lane & 15, ro = lane >> 4;
    const int cb = blockIdx.x % NCB, item = blockIdx.x / NCB;
    const int n = item / a.Hv, h = item - n * a.Hv;
    const int col = cb * kStepCols + 4 * cq;
    const float *src = slot_of(a, a.read_idx, n, state);
    float *dst = slot_of(a, a.write_idx, n, state);

    f32x4 S[NS];
#pragma unroll
    for (int j = 0; j < NS; ++j) S[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (src) {
        src += h * state + col;
#pragma unroll
        for (int j = 0; j < NS; ++j) S[j] = *(const f32x4 *)(src + (16 * j + 4 * w + ro) * DV);
    }
    const int64_t t = n;
    const int hk = h / (a.Hv / a.Hk);
    const f32x4 v = load4<BF>(a.v, t * a.v_row + (int64_t)h * DV + col);
    const float g = a.g[t * a.g_row + h];
    bool slow = g > kSlow && g <= 0.f;                   // S + S (e^g - 1), but for infinities
    float keep = slow ? expm1_small(g) : expf(g);
    if (tid < DK) {
        s_q[tid] = a.scale * load1<BF>(a.q, t * a.q_row + hk * DK + tid);
        s_k[tid] = load1<BF>(a.k, t * a.k_row + hk * DK + tid);
    }
    __syncthreads();

    float top = 0.f;
#pragma unroll
    for (int j = 0; j < NS; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) top = fmaxf(top, fabsf(S[j][c]));
    if (slow && __any(top == __builtin_inff())) {
#pragma unroll
        for (int j = 0; j < NS; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c) S[j][c] = decayed(S[j][c], keep, slow);
        keep = 1.f;
        slow = false;
    }

    f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NS; ++j) {
        const int row = 16 * j + 4 * w + ro;
#pragma unroll
        for (int c = 0; c < 4; ++c) S[j][c] = fmaf(S[j][c], keep, slow ? S[j][c] : 0.f);
        S[j] += s_k[row] * v;
        o += s_q[row] * S[j];
    }
    if (dst) {
        dst += h * state + col;
#pragma unroll
        for (int j = 0; j < NS; ++j) *(f32x4 *)(dst + (16 * j + 4 * w + ro) * DV) = S[j];
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {   // over the lanes that share the columns
        o[c] += __shfl_xor(o[c], 16);
        o[c] += __shfl_xor(o[c], 32);
    }
    if (ro == 0) *(f32x4 *)&s_o[w][4 * cq] = o;
    __syncthreads();
    if (tid < 16) {
        o = *(const f32x4 *)&s_o[0][4 * tid] + *(const f32x4 *)&s_o[1][4 * tid] + *(const f32x4 *)&s_o[2][4 * tid] +
            *(const f32x4 *)&s_o[3][4 * tid];
        mf::Ops<BF>::st4((typename mf::Ops<BF>::T *)a.o + (t * a.Hv + h) * DV + col, o);
    }
}

template <int DK, int DV, bool BF>
hipError_t launch(const LinArgs &a, hipStream_t s) {
    const dim3 grid((unsigned)(a.N * a.Hv * (DV / kStepCols)));
    hipLaunchKernelGGL((step_kernel<DK, DV, BF>), grid, dim3(kStepThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_lin_step(bool bf16, int dk, int dv, const LinArgs &a, hipStream_t s) {
    if (a.N <= 0) return hipSuccess;
#define KDA_STEP(DK_, DV_)                                                                 \
    if (dk == DK_ && dv == DV_) return bf16 ? launch<DK_, DV_, true>(a, s) : launch<DK_, DV_, false>(a, s);
    KDA_STEP(64, 64)
    KDA_STEP(64, 128)
    KDA_STEP(128, 64)
    KDA_STEP(128, 128)
#undef KDA_STEP
    return hipErrorInvalidValue;
}

}  // namespace kda
