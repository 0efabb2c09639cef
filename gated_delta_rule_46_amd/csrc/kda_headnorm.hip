// kda_headnorm.hip -- norm of every head (a group of D channels, channels last) with an
// activation, the step between a linear layer's outputs and its projection:
//     y = (x - mean) w / sqrt(var + eps) + b   (mean = 0 and var = mean(x^2) without centering)
//     y <- y act(gate), or act(y) without a gate
//
// One read and one write per element: bound by HBM.  A head is taken by the smallest
// power of two of lanes that holds it in 16-byte pieces (64 lanes with up to 4 pieces
// each for the widest), stays in registers, and its sums go through lane exchanges; the
// variance is summed from the centered values.  All arithmetic in fp32, one rounding
// at the store.  A head whose mean square leaves fp32's range is scaled by a power of
// two first.

#include "kda_attn.h"
#include "kda_lin.h"
#include "kda.h"
#include "kda_mfma.h"

namespace kda {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kNormThreads = 256;

// Least mean square (eps in it) that is used as it stands: what its squares lost below
// fp32's smallest normal, 2^-126 each, is less than 2^-24 of it.
constexpr float kLeastSquare = 0x1p-100f;

template <bool BF>
__device__ __forceinline__ void unpack(u32x4 w, float *x) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (BF) {
            x[2 * j] = bits_f32(w[j] << 16);
            x[2 * j + 1] = bits_f32(w[j] & 0xffff0000u);
        } else {
            x[j] = bits_f32(w[j]);
        }
    }
}

template <int L>
__device__ __forceinline__ float sum_of(float x) {
#pragma unroll
    for (int off = 1; off < L; off <<= 1) x += __shfl_xor(x, off);
    return x;
}

__device__ __forceinline__ float activation(float x, int act) {
    if (act == KDA_ACT_NONE) return x;
    return (act == KDA_ACT_SILU ? x : 1.f) / (1.f + expf(-x));
}

// V pieces of E values in each of L lanes; pieces behind the head's end hold zeros.
template <int L, int V, bool BF>
struct Head {
    static constexpr int E = BF ? 8 : 4, NX = V * E;
    float x[NX];
    // subtracts the mean where asked for; returns the mean square
    __device__ __forceinline__ float squares(const HeadNormArgs &a, int l, float inv) {
        if (a.center) {
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < NX; ++j) s += x[j];
            s = sum_of<L>(s) * inv;
#pragma unroll
            for (int j = 0; j < NX; ++j) x[j] = (l + L * (j / E)) * E < a.D ? x[j] - s : 0.f;
        }
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < NX; ++j) ss += x[j] * x[j];
        return sum_of<L>(ss) * inv;
    }
};

template <int L, int V, bool BF>
__global__ __launch_bounds__(kNormThreads) void norm_kernel(const HeadNormArgs a) {
    constexpr int E = BF ? 8 : 4, NX = V * E;
    using T = typename mf::Ops<BF>::T;
    const int l = threadIdx.x % L;
    const int64_t head = (int64_t)blockIdx.x * (kNormThreads / L) + threadIdx.x / L;
    const bool live = head < a.T * a.H;
    const int64_t t = live ? head / a.H : 0;
    const int h = live ? (int)(head - t * a.H) : 0;
    const float inv = 1.f / (float)a.D;

    u32x4 rx[V], rz[V];
    Head<L, V, BF> y;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int d = (l + L * i) * E;
        rx[i] = rz[i] = u32x4{0, 0, 0, 0};
        if (live && d < a.D) {
            rx[i] = *(const u32x4 *)((const T *)a.x + t * a.x_row + (int64_t)h * a.D + d);
            if (a.gate) rz[i] = *(const u32x4 *)((const T *)a.gate + t * a.gate_row + (int64_t)h * a.D + d);
        }
        unpack<BF>(rx[i], y.x + i * E);
    }
    const float ms = y.squares(a, l, inv) + a.eps;
    float r = rsqrtf(ms);
    if (!(ms >= kLeastSquare && ms < __builtin_inff())) {   // the same in a head's lanes
        // x and sqrt(eps) as multiples of 2^k, the larger of them within [1/2, 1);
        // infinities and NaN stay as they are
        float top = sqrtf(a.eps);
#pragma unroll
        for (int i = 0; i < V; ++i) unpack<BF>(rx[i], y.x + i * E);
#pragma unroll
        for (int j = 0; j < NX; ++j) top = fmaxf(top, fabsf(y.x[j]));
#pragma unroll
        for (int off = 1; off < L; off <<= 1) top = fmaxf(top, __shfl_xor(top, off));
        const int k = top > 0.f && top < __builtin_inff() ? __builtin_amdgcn_frexp_expf(top) : 0;
#pragma unroll
        for (int j = 0; j < NX; ++j) y.x[j] = ldexpf(y.x[j], -k);
        r = rsqrtf(y.squares(a, l, inv) + ldexpf(a.eps, -2 * k));
    }
    if (!live) return;
    const int64_t w0 = a.per_head ? (int64_t)h * a.D : 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int d = (l + L * i) * E;
        if (d >= a.D) break;
        float z[E];
        unpack<BF>(rz[i], z);
#pragma unroll
        for (int j = 0; j < E; ++j) {
            float x = y.x[i * E + j] * r;
            if (a.weight) x *= a.weight[w0 + d + j];
            if (a.bias) x += a.bias[w0 + d + j];
            y.x[i * E + j] = a.gate ? x * activation(z[j], a.act) : activation(x, a.act);
        }
        T *const out = (T *)a.y + t * a.y_row + (int64_t)h * a.D + d;
        if constexpr (BF) mf::Ops<BF>::st8(out, y.x + i * E);
        else *(mf::f32x4 *)out = mf::f32x4{y.x[i * E], y.x[i * E + 1], y.x[i * E + 2], y.x[i * E + 3]};
    }
}

template <int L, int V, bool BF>
hipError_t launch(const HeadNormArgs &a, hipStream_t s) {
    constexpr int per = kNormThreads / L;
    const dim3 grid((unsigned)((a.T * a.H + per - 1) / per));
    hipLaunchKernelGGL((norm_kernel<L, V, BF>), grid, dim3(kNormThreads), 0, s, a);
    return hipGetLastError();
}

template <bool BF>
hipError_t pick(const HeadNormArgs &a, hipStream_t s) {
    const int pieces = (a.D + (BF ? 7 : 3)) / (BF ? 8 : 4);
    if (pieces <= 1) return launch<1, 1, BF>(a, s);
    if (pieces <= 2) return launch<2, 1, BF>(a, s);
    if (pieces <= 4) return launch<4, 1, BF>(a, s);
    if (pieces <= 8) return launch<8, 1, BF>(a, s);
    if (pieces <= 16) return launch<16, 1, BF>(a, s);
    if (pieces <= 32) return launch<32, 1, BF>(a, s);
    if (pieces <= 64) return launch<64, 1, BF>(a, s);
    if (pieces <= 128) return launch<64, 2, BF>(a, s);
    if constexpr (!BF)
        if (pieces <= 256) return launch<64, 4, BF>(a, s);
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_head_norm(bool bf16, const HeadNormArgs &a, hipStream_t s) {
    if (a.T <= 0) return hipSuccess;
    return bf16 ? pick<true>(a, s) : pick<false>(a, s);
}

}  // namespace kda
