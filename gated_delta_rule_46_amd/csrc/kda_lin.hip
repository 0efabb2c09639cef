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
// One workgroup takes a sequence and value head from its first chunk to its last;
// a wave owns 16 of the value columns and keeps their part of S (dk x 16) in the
// accumulators of the state product for the whole sequence.  As the rows of S that
// a lane accumulates are chosen to be 8 consecutive ones of a 32-row block, the
// registers are the operand of S^T q as they stand.  The tiles of P (C x C, its
// lower triangle) are shared out over the waves and exchanged through LDS.
//
// q, k and v of the next chunk but one are on their way from HBM into registers
// while a chunk is computed, and the next chunk's lie in the other half of LDS.

#include "kda_attn.h"
#include "kda_lin.h"
#include "kda_mfma.h"

namespace kda {
namespace {

using mf::bf16_t;
using mf::bf16x4;
using mf::bf16x8;
using mf::f32x4;
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr float kLeastGate = -1e4f;   // e^-10000 is zero; sums of it stay exact to 2^-30 in fp64

template <int DK_, int DV_, bool BF_>
struct Shape {
    static constexpr int DK = DK_, DV = DV_;
    static constexpr bool BF = BF_;
    using O = mf::Ops<BF>;
    using T = typename O::T;
    static constexpr int C = BF ? 64 : 32;          // tokens per chunk
    static constexpr int NT = C / 16, NJ = C / 32;  // tiles of 16 and blocks of 32 tokens
    static constexpr int NW = DV / 16, THREADS = 64 * NW;
    static constexpr int NKB = DK / 32;
    static constexpr int TERMS = BF ? 3 : 1;        // operand terms that hold an fp32 value
    static constexpr int SK = DK + O::PAD, SV = DV + O::PAD, SP = C + O::PAD;   // LDS rows
    static constexpr int E = 16 / sizeof(T);        // elements of a 16-byte piece
    static constexpr int NPK = C * DK / E / THREADS, NPV = C * DV / E / THREADS;
    static constexpr int QB = C * SK * sizeof(T), VB = C * SV * sizeof(T), PB = C * SP * sizeof(T);
    static constexpr int DECAYS = 4 * C + 4;        // floats: G high, G low, e^G, weights, e^G_C
    static constexpr int STAGE = 2 * QB + VB + DECAYS * 4;
    static constexpr int LDS = 2 * STAGE + PB;
    static_assert(C * DK % (E * THREADS) == 0 && C * DV % (E * THREADS) == 0);
    static_assert(LDS <= 160 * 1024 && QB % 16 == 0 && VB % 16 == 0 && STAGE % 16 == 0);
};

// A chunk's tiles in LDS.
template <class X>
struct Stage {
    typename X::T *q, *k, *v;
    float *hi, *lo, *out, *keep;      // G in log2 (two floats), scale e^G, e^{G_C - G}
    float *all;                       // e^{G_C}
    __device__ explicit Stage(char *p)
        : q((typename X::T *)p), k((typename X::T *)(p + X::QB)), v((typename X::T *)(p + 2 * X::QB)) {
        hi = (float *)(p + 2 * X::QB + X::VB);
        lo = hi + X::C;
        out = lo + X::C;
        keep = out + X::C;
        all = keep + X::C;
    }
};

// Transposed operand fragment from row-major LDS rows: lane (m, g) gets column col(m) of
// rows 8g .. 8g+7.  bf16: p points at row 8g + (m / 4), 4 columns for m % 4 (a 16-lane group
// loads 4 x 16 values and each lane gets one column of 4 rows); fp32: at row 8g, column col(m).
template <class X>
__device__ __forceinline__ typename X::O::F8 ld_t(const typename X::T *p, int stride) {
    if constexpr (X::BF) {
        typedef short s16x4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) s16x4 lds_t;
        const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t *)p);
        const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t *)(p + 4 * stride));
        return X::O::cat(__builtin_bit_cast(bf16x4, a), __builtin_bit_cast(bf16x4, b));
    } else {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = p[e * stride];
        return X::O::cvt8(x);
    }
}

template <class X> struct Terms { typename X::O::F8 t[X::TERMS]; };

// fp32 values as operand terms (an infinity is its first term alone).
template <class X>
__device__ __forceinline__ Terms<X> terms8(const float *x) {
    Terms<X> r;
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = x[j];
#pragma unroll
    for (int t = 0; t < X::TERMS; ++t) {
        r.t[t] = X::O::cvt8(y);
        if (t + 1 < X::TERMS) {
            float z[8];
            X::O::unpack8(r.t[t], z);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = (f32_bits(z[j]) & 0x7fffffffu) == 0x7f800000u ? 0.f : y[j] - z[j];
        }
    }
    return r;
}

__device__ __forceinline__ bool not_finite(float x) { return (f32_bits(x) & 0x7f800000u) == 0x7f800000u; }

// The operand with zeros in place of infinities and NaN.
template <class X>
__device__ __forceinline__ typename X::O::F8 finite_part(typename X::O::F8 f) {
    float x[8];
    X::O::unpack8(f, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = not_finite(x[e]) ? 0.f : x[e];
    return X::O::cvt8(x);
}

// 2^x of an fp64 x <= 0 or so, to about an ulp of fp32.
__device__ __forceinline__ float exp2_of(double x) {
    const float hi = (float)x;
    const float lo = (float)(x - (double)hi);
    const float e = mf::ex2(hi);
    return hi < -150.f ? 0.f : e + e * (lo * 0.6931471805599453f);
}

// The decays of a chunk from its log decays (lane = token; zero behind the end), by one wave.
template <class X>
__device__ __forceinline__ void write_decays(const Stage<X> &s, float g, float scale) {
    const int lane = threadIdx.x & 63;
    double x = (double)(g < kLeastGate ? kLeastGate : g) * 1.4426950408889634;   // NaN stays
#pragma unroll
    for (int off = 1; off < X::C; off <<= 1) {
        const double y = __shfl_up(x, off);
        if (lane >= off) x += y;
    }
    const double all = __shfl(x, X::C - 1);
    if (lane < X::C) {
        s.hi[lane] = (float)x;
        s.lo[lane] = (float)(x - (double)(float)x);
        s.out[lane] = scale * exp2_of(x);
        s.keep[lane] = exp2_of(all - x);
        if (lane == 0) *s.all = exp2_of(all);
    }
}

// 2^(G_i - G_j)
template <class X>
__device__ __forceinline__ float decay_between(float hi_i, float lo_i, float hi_j, float lo_j) {
    const float d = hi_i - hi_j;
    if constexpr (X::BF) return mf::ex2(d + (lo_i - lo_j));   // P is rounded to bf16
    const float b = d - hi_i;                                 // what the subtraction rounded off
    const float e = mf::ex2(d);
    return e + e * (((hi_i - (d - b)) + (-hi_j - b) + (lo_i - lo_j)) * 0.6931471805599453f);
}

template <int DK, int DV, bool BF>
__global__ __launch_bounds__((Shape<DK, DV, BF>::THREADS)) void lin_kernel(const LinArgs a) {
    using X = Shape<DK, DV, BF>;
    using O = typename X::O;
    using T = typename X::T;
    using F8 = typename O::F8;
    constexpr int C = X::C, NT = X::NT, NJ = X::NJ, NKB = X::NKB, E = X::E;
    extern __shared__ __align__(16) char lds[];
    T *const sp = (T *)(lds + 2 * X::STAGE);

    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int m = lane & 15, gq = lane >> 4;
    const int n = blockIdx.x / a.Hv, h = blockIdx.x - n * a.Hv;
    const int hk = h / (a.Hv / a.Hk);
    const int64_t c0 = max(a.cu[n], (int64_t)0);
    const int64_t len64 = min(a.cu[n + 1], a.T) - c0;
    const int len = len64 > 0 ? (int)len64 : 0;
    constexpr int64_t state = (int64_t)DK * DV;

    // S[kb][half]: rows 32 kb + 8 gq + 4 half + i, column 16 w + m
    const int s_at = 8 * gq * DV + 16 * w + m;
    f32x4 S[NKB][2];
    const float *src = slot_of(a, a.read_idx, n, state);
#pragma unroll
    for (int kb = 0; kb < NKB; ++kb)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                S[kb][hf][i] = src ? src[h * state + s_at + (32 * kb + 4 * hf + i) * DV] : 0.f;

    u32x4 rq[X::NPK], rk[X::NPK], rv[X::NPV];
    float rg = 0.f;
    auto fetch = [&](int first) {                       // rows behind the end become zeros
        const int valid = min(C, len - first);
        const int64_t t = c0 + first;
        constexpr int PK = DK / E, PV = DV / E;
#pragma unroll
        for (int i = 0; i < X::NPK; ++i) {
            const int p = tid + i * X::THREADS, row = p / PK, at = p % PK * E;
            rq[i] = rk[i] = u32x4{0, 0, 0, 0};
            if (row < valid) {
                rq[i] = *(const u32x4 *)((const T *)a.q + (t + row) * a.q_row + hk * DK + at);
                rk[i] = *(const u32x4 *)((const T *)a.k + (t + row) * a.k_row + hk * DK + at);
            }
        }
#pragma unroll
        for (int i = 0; i < X::NPV; ++i) {
            const int p = tid + i * X::THREADS, row = p / PV, at = p % PV * E;
            rv[i] = u32x4{0, 0, 0, 0};
            if (row < valid) rv[i] = *(const u32x4 *)((const T *)a.v + (t + row) * a.v_row + (int64_t)h * DV + at);
        }
        rg = 0.f;
        if (w == X::NW - 1 && lane < valid) rg = a.g[(t + lane) * a.g_row + h];
    };
    auto put = [&](const Stage<X> &s) {
        constexpr int PK = DK / E, PV = DV / E;
#pragma unroll
        for (int i = 0; i < X::NPK; ++i) {
            const int p = tid + i * X::THREADS, row = p / PK, at = p % PK * E;
            *(u32x4 *)(s.q + row * X::SK + at) = rq[i];
            *(u32x4 *)(s.k + row * X::SK + at) = rk[i];
        }
#pragma unroll
        for (int i = 0; i < X::NPV; ++i) {
            const int p = tid + i * X::THREADS, row = p / PV, at = p % PV * E;
            *(u32x4 *)(s.v + row * X::SV + at) = rv[i];
        }
        if (w == X::NW - 1) write_decays<X>(s, rg, a.scale);
    };

    fetch(0);
    put(Stage<X>(lds));
    fetch(C);
    __syncthreads();
    for (int first = 0, buf = 0; first < len; first += C, buf ^= 1) {
        const Stage<X> s(lds + buf * X::STAGE);
        const int valid = min(C, len - first);
        const int nt = (valid + 15) >> 4;

        // P^T tiles (rows j, columns i): lane holds 4 consecutive j of its i
        constexpr int TILES = NT * (NT + 1) / 2;
        for (int t = w; t < TILES + NJ; t += X::NW) {
            if (t >= TILES) {                           // the upper tile of a diagonal 32-block
                const int it = 2 * (t - TILES);
                O::st4(sp + (16 * it + m) * X::SP + 16 * it + 16 + 4 * gq, f32x4{0.f, 0.f, 0.f, 0.f});
                continue;
            }
            const int it = t < 1 ? 0 : t < 3 ? 1 : t < 6 ? 2 : 3, jt = t - it * (it + 1) / 2;
            if (it >= nt) continue;
            const int i = 16 * it + m, j = 16 * jt + 4 * gq;
            f32x4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb)
                p = O::mma32(p, O::ld8(s.k + (16 * jt + m) * X::SK + 32 * kb + 8 * gq),
                             O::ld8(s.q + i * X::SK + 32 * kb + 8 * gq));
            const f32x4 hj = *(const f32x4 *)(s.hi + j), lj = *(const f32x4 *)(s.lo + j);
            const float hi = s.hi[i], li = s.lo[i];
#pragma unroll
            for (int r = 0; r < 4; ++r)
                p[r] = j + r <= i ? a.scale * decay_between<X>(hi, li, hj[r], lj[r]) * p[r] : 0.f;
            O::st4(sp + i * X::SP + j, p);
        }

        // o^T = e^G S^T q^T: lane holds token 16 it + m, columns 16 w + 4 gq + r
        f32x4 acc[NT];
#pragma unroll
        for (int it = 0; it < NT; ++it) acc[it] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kb = 0; kb < NKB; ++kb) {
            const F8 sf = O::cvt44(S[kb][0], S[kb][1]);
#pragma unroll
            for (int it = 0; it < NT; ++it)
                if (it < nt) acc[it] = O::mma32(acc[it], sf, O::ld8(s.q + (16 * it + m) * X::SK + 32 * kb + 8 * gq));
        }
#pragma unroll
        for (int it = 0; it < NT; ++it) acc[it] *= s.out[16 * it + m];

        // v^T of this wave's columns
        F8 vf[NJ];
        bool odd = false;
#pragma unroll
        for (int jb = 0; jb < NJ; ++jb) {
            if constexpr (BF) vf[jb] = ld_t<X>(s.v + (32 * jb + 8 * gq + (m >> 2)) * X::SV + 16 * w + 4 * (m & 3), X::SV);
            else vf[jb] = ld_t<X>(s.v + (32 * jb + 8 * gq) * X::SV + 16 * w + m, X::SV);
            float x[8];
            O::unpack8(vf[jb], x);
#pragma unroll
            for (int e = 0; e < 8; ++e) odd |= not_finite(x[e]);
        }
        __syncthreads();   // P is there

        // infinities and NaN must not meet the zeros of P above its diagonal: they are left out of
        // the products and added token by token
        const bool rare = __any(odd);
        F8 vp[NJ];
#pragma unroll
        for (int jb = 0; jb < NJ; ++jb) vp[jb] = rare ? finite_part<X>(vf[jb]) : vf[jb];
#pragma unroll
        for (int it = 0; it < NT; ++it)
            if (it < nt) {
#pragma unroll
                for (int jb = 0; jb < NJ; ++jb)
                    if (2 * jb <= it) acc[it] = O::mma32(acc[it], vp[jb], O::ld8(sp + (16 * it + m) * X::SP + 32 * jb + 8 * gq));
            }
        if (rare) {
            for (int j = 0; j < valid; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float x = (float)s.v[j * X::SV + 16 * w + 4 * gq + r];
#pragma unroll
                    for (int it = 0; it < NT; ++it)
                        if (not_finite(x) && j <= 16 * it + m) acc[it][r] += (float)sp[(16 * it + m) * X::SP + j] * x;
                }
        }
#pragma unroll
        for (int it = 0; it < NT; ++it) {
            const int i = 16 * it + m;
            if (i < valid)
                O::st4((T *)a.o + ((c0 + first + i) * a.Hv + h) * DV + 16 * w + 4 * gq, acc[it]);
        }

        // S <- e^{G_C} S + k^T (weights v)
        const float all = *s.all;
#pragma unroll
        for (int kb = 0; kb < NKB; ++kb) { S[kb][0] *= all; S[kb][1] *= all; }
#pragma unroll
        for (int jb = 0; jb < NJ; ++jb) {
            float x[8], wt[8];
            O::unpack8(vf[jb], x);
            mf::load8f(s.keep + 32 * jb + 8 * gq, wt);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = 32 * jb + 8 * gq + e < valid ? x[e] * wt[e] : 0.f;
            const Terms<X> wv = terms8<X>(x);
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    F8 kf;
                    if constexpr (BF) kf = ld_t<X>(s.k + (32 * jb + 8 * gq + (m >> 2)) * X::SK + 32 * kb + 8 * (m & 3) + 4 * hf, X::SK);
                    else kf = ld_t<X>(s.k + (32 * jb + 8 * gq) * X::SK + 32 * kb + 8 * (m >> 2) + (m & 3) + 4 * hf, X::SK);
#pragma unroll
                    for (int t = 0; t < X::TERMS; ++t) S[kb][hf] = O::mma32(S[kb][hf], kf, wv.t[t]);
                }
        }

        if (first + C < len) {
            put(Stage<X>(lds + (buf ^ 1) * X::STAGE));
            fetch(first + 2 * C);
        }
        const int end = first + C;
        if (a.interval && end <= len && end % a.interval == 0) {
            float *dst = a.ckpt + (((a.ckpt_off ? a.ckpt_off[n] : 0) + end / a.interval - 1) * a.Hv + h) * state + s_at;
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                    for (int i = 0; i < 4; ++i) dst[(32 * kb + 4 * hf + i) * DV] = S[kb][hf][i];
        }
        __syncthreads();
    }

    float *dst = slot_of(a, a.write_idx, n, state);
    if (dst) {
        dst += h * state + s_at;
#pragma unroll
        for (int kb = 0; kb < NKB; ++kb)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                for (int i = 0; i < 4; ++i) dst[(32 * kb + 4 * hf + i) * DV] = S[kb][hf][i];
    }
}

template <int DK, int DV, bool BF>
hipError_t launch(const LinArgs &a, hipStream_t s) {
    using X = Shape<DK, DV, BF>;
    const hipError_t e = hipFuncSetAttribute((const void *)lin_kernel<DK, DV, BF>,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, X::LDS);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((lin_kernel<DK, DV, BF>), dim3((unsigned)(a.N * a.Hv)), dim3(X::THREADS), X::LDS, s, a);
    return hipGetLastError();
}

}  // namespace

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
