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
//
// A lane of bf16 heads has the pieces of four on their way before it waits for the first, and weights that all
// heads share are loaded once: 16,384 tokens of 32 heads of 128 with a gate, bf16, 159 us with one head a
// lane and the weights read for each, 64.5 so (403 MB, 6.2 TB/s; a large copy 5.15).  With the library's
// exponential and a division for the bf16 gates too it takes 80.6.  64 tokens: 4 us, the launch.

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

// e^-|x| neither overflows nor needs a special case.  bf16 outputs take the hardware's exponential and
// reciprocal (an ulp of fp32 each, and |x| 2^-24 from the exponent's scaling).
template <bool BF>
__device__ __forceinline__ float activation(float x, int act) {
    if (act == KDA_ACT_NONE) return x;
    float s;
    if (BF) {
        const float e = mf::ex2(-fabsf(x) * mf::kLog2e), r = __builtin_amdgcn_rcpf(1.f + e);
        s = x < 0.f ? e * r : r;
    } else {
        const float e = expf(-fabsf(x));
        s = (x < 0.f ? e : 1.f) / (1.f + e);
    }
    s = x != x ? x : s;
    return act == KDA_ACT_SILU ? x * s : s;
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
    __device__ __forceinline__ void take(const u32x4 *r) {
#pragma unroll
        for (int i = 0; i < V; ++i) unpack<BF>(r[i], x + i * E);
    }
};

// R heads a lane, whose loads are on their way together.
template <int L, int V, int R, bool BF>
__global__ __launch_bounds__(kNormThreads) void norm_kernel(const HeadNormArgs a) {
    constexpr int E = BF ? 8 : 4, NX = V * E, PER = kNormThreads / L;
    using T = typename mf::Ops<BF>::T;
    const int l = threadIdx.x % L;
    const uint32_t heads = (uint32_t)(a.T * a.H), first = blockIdx.x * (uint32_t)(PER * R) + threadIdx.x / L;
    const float inv = 1.f / (float)a.D;

    int64_t t[R];
    int at[R];                        // the lane's first element in its token's row
    u32x4 rx[R][V], rz[R][V];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const uint32_t head = min(first + r * PER, heads - 1);
        t[r] = head / (uint32_t)a.H;
        at[r] = (int)(head - (uint32_t)t[r] * a.H) * a.D + l * E;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            rx[r][i] = rz[r][i] = u32x4{0, 0, 0, 0};
            if ((l + L * i) * E < a.D) {
                rx[r][i] = __builtin_nontemporal_load((const u32x4 *)((const T *)a.x + t[r] * a.x_row + at[r] + L * i * E));
                if (a.gate)
                    rz[r][i] = __builtin_nontemporal_load((const u32x4 *)((const T *)a.gate + t[r] * a.gate_row + at[r] + L * i * E));
            }
        }
    }
    float w[NX], b[NX];
    auto affine = [&](int from) {
#pragma unroll
        for (int j = 0; j < NX; j += 4) {
            const bool in = (l + L * (j / E)) * E < a.D;
            const int d = from + L * (j / E) * E + j % E;
            const mf::f32x4 one = {1.f, 1.f, 1.f, 1.f}, zero = {0.f, 0.f, 0.f, 0.f};
            const mf::f32x4 x = a.weight && in ? *(const mf::f32x4 *)(a.weight + d) : one;
            const mf::f32x4 y = a.bias && in ? *(const mf::f32x4 *)(a.bias + d) : zero;
#pragma unroll
            for (int i = 0; i < 4; ++i) { w[j + i] = x[i]; b[j + i] = y[i]; }
        }
    };
    if (!a.per_head) affine(l * E);

#pragma unroll
    for (int r = 0; r < R; ++r) {
        Head<L, V, BF> y;
        y.take(rx[r]);
        const float ms = y.squares(a, l, inv) + a.eps;
        float scale = rsqrtf(ms);
        if (!(ms >= kLeastSquare && ms < __builtin_inff())) {   // the same in a head's lanes
            // x and sqrt(eps) as multiples of 2^k, the larger of them within [1/2, 1);
            // infinities and NaN stay as they are
            float top = sqrtf(a.eps);
            y.take(rx[r]);
#pragma unroll
            for (int j = 0; j < NX; ++j) top = fmaxf(top, fabsf(y.x[j]));
#pragma unroll
            for (int off = 1; off < L; off <<= 1) top = fmaxf(top, __shfl_xor(top, off));
            const int k = top > 0.f && top < __builtin_inff() ? __builtin_amdgcn_frexp_expf(top) : 0;
#pragma unroll
            for (int j = 0; j < NX; ++j) y.x[j] = ldexpf(y.x[j], -k);
            scale = rsqrtf(y.squares(a, l, inv) + ldexpf(a.eps, -2 * k));
        }
        if (a.per_head) affine(at[r]);
        const bool live = first + r * PER < heads;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float z[E], out[E];
            unpack<BF>(rz[r][i], z);
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const float x = y.x[i * E + j] * scale * w[i * E + j] + b[i * E + j];
                out[j] = a.gate ? x * activation<BF>(z[j], a.act) : activation<BF>(x, a.act);
            }
            T *const dst = (T *)a.y + t[r] * a.y_row + at[r] + L * i * E;
            if (live && (l + L * i) * E < a.D) {
                if constexpr (BF) mf::Ops<BF>::st8(dst, out);
                else *(mf::f32x4 *)dst = mf::f32x4{out[0], out[1], out[2], out[3]};
            }
        }
    }
}

template <int L, int V, int R, bool BF>
hipError_t launch(const HeadNormArgs &a, hipStream_t s) {
    constexpr int per = kNormThreads / L * R;
    const dim3 grid((unsigned)((a.T * a.H + per - 1) / per));
    hipLaunchKernelGGL((norm_kernel<L, V, R, BF>), grid, dim3(kNormThreads), 0, s, a);
    return hipGetLastError();
}

// One head a lane where there are too few of them to give each of 256 compute units four workgroups (32 heads of 128 with
// a gate, bf16: 1,500 tokens 8.0 us with one, 8.9 with four; 2,048 10.8 / 10.9; 8,192 39.0 / 34.6; two wide ones, 16 of
// 520, fp32: 16,384 tokens 374 / 317), and for fp32 heads of one piece a lane at any number (32 of 128, 16,384 tokens 120
// with one, 134 with four, 119 with two; 32 of 256 261 / 285 / 275).
template <int L, int V, bool BF>
hipError_t launch(const HeadNormArgs &a, hipStream_t s) {
    if constexpr (BF || V > 1) {
        constexpr int R = V == 1 ? 4 : 2;
        if (a.T * a.H >= (int64_t)kNormThreads / L * R * 1024) return launch<L, V, R, BF>(a, s);
    }
    return launch<L, V, 1, BF>(a, s);
}

template <bool BF>
hipError_t pick(const HeadNormArgs &a, hipStream_t s) {
    const int pieces = a.D / (BF ? 8 : 4);
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
