// kda_rotate.hip -- RMS norm of every query and key head with the rotation by
// position in the same pass.
//
// For token t and head x in R^D:
//     y = x * w / sqrt(mean(x^2) + eps)
//     (y_a, y_b) <- (y_a cos - y_b sin, y_b cos + y_a sin)
// for the pairs (a, b) of the first `rot` dims, with the cosine and sine of the
// pair's angle at the token's position read from a table (fp32, filled once by
// the caller: angles of far positions need more than fp32 arithmetic).
//
// One read and one write per element: bound by HBM.  A workgroup takes one
// token; D/8 lanes take a head, 8 dims each (a 16-byte bf16 vector), so a
// lane's dims are the same for all of its heads and the weights, cosines and
// sines are loaded once per lane.  All arithmetic in fp32, one rounding at the
// store.  A head whose mean square leaves fp32's range (elements beyond about 2^63,
// or tiny ones with an eps as small) is scaled by a power of two first, which costs
// the others a comparison (57.2 -> 58.6 us below).  16,384 tokens at 32 / 8 heads of 128
// with bf16 rows: 58.6 us (343 MB, 5.9 TB/s; a large copy 5.15), with fp32 rows 139 (4.9);
// 64 tokens 4.7 us, the launch.

#include "kda_attn.h"
#include "kda_mfma.h"

namespace kda {
namespace {

constexpr int kRotThreads = 256;

// Least mean square (eps in it) that is used as it stands: what its squares lost below
// fp32's smallest normal, 2^-126 each, is less than 2^-24 of it.
constexpr float kLeastMean = 0x1p-100f;

// The head x of L lanes as x / 2^k, and eps as eps / 4^k, with the larger of max |x| and
// sqrt(eps) within [1/2, 1): the mean square is then at least 2^-9.  Returns its
// reciprocal root.  All lanes of the head call it; infinities and NaN are left as they are.
template <int L>
__device__ __forceinline__ float rescale(float (&x)[8], float eps) {
    float top = sqrtf(eps);
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(x[j]));
#pragma unroll
    for (int off = 1; off < L; off <<= 1) top = fmaxf(top, __shfl_xor(top, off));
    const int k = top > 0.f && top < __builtin_inff() ? __builtin_amdgcn_frexp_expf(top) : 0;
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        x[j] = ldexpf(x[j], -k);
        ss += x[j] * x[j];
    }
#pragma unroll
    for (int off = 1; off < L; off <<= 1) ss += __shfl_xor(ss, off);
    return rsqrtf(ss * (1.f / (8 * L)) + ldexpf(eps, -2 * k));
}

template <int D, bool BF, bool PAIRS>
__global__ __launch_bounds__(kRotThreads) void rotate_kernel(const RotateArgs a) {
    constexpr int L = D / 8;                  // lanes per head
    constexpr int G = kRotThreads / L;        // heads per pass
    const int tid = threadIdx.x;
    const int d0 = (tid % L) * 8, grp = tid / L;
    const int64_t t = blockIdx.x;

    float cs[8], sn[8];                       // y_j -> y_j cs_j + partner_j sn_j
#pragma unroll
    for (int j = 0; j < 8; ++j) { cs[j] = 1.f; sn[j] = 0.f; }
    const int half = a.rot >> 1;
    int partner = tid & 63;
    if (a.table) {
        const int64_t p = a.positions[t];
        if (p < 0 || p >= a.n_pos) return;    // a padded token: its rows stay as they are
        const float *row = a.table + p * a.rot;
        if (d0 < a.rot) {
            if (PAIRS) {
                const float4 c = *(const float4 *)(row + (d0 >> 1));
                const float4 s = *(const float4 *)(row + half + (d0 >> 1));
                const float cv[4] = {c.x, c.y, c.z, c.w}, sv[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    cs[2 * j] = cs[2 * j + 1] = cv[j];
                    sn[2 * j] = -sv[j];
                    sn[2 * j + 1] = sv[j];
                }
            } else {
                const bool hi = d0 >= half;
                const int i0 = hi ? d0 - half : d0;
                mf::load8f(row + i0, cs);
                mf::load8f(row + half + i0, sn);
                if (!hi) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) sn[j] = -sn[j];
                }
                partner += hi ? -(half >> 3) : (half >> 3);
            }
        }
    }
    float wq[8], wk[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) { wq[j] = 1.f; wk[j] = 1.f; }
    if (a.q_weight) mf::load8f(a.q_weight + d0, wq);
    if (a.k_weight) mf::load8f(a.k_weight + d0, wk);

    const int H = a.Hq + a.Hk;
    for (int h0 = 0; h0 < H; h0 += G) {       // every lane takes part in the exchanges
        const int h = h0 + grp;
        const bool isq = h < a.Hq, live = h < H;
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = 0.f;
        if (live) {
            if (isq) load8_once<BF>(a.q, t * a.q_row + (int64_t)h * D + d0, x);
            else load8_once<BF>(a.k, t * a.k_row + (int64_t)(h - a.Hq) * D + d0, x);
        }
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss += x[j] * x[j];
#pragma unroll
        for (int off = 1; off < L; off <<= 1) ss += __shfl_xor(ss, off);
        const float mean = ss * (1.f / D) + a.eps;
        float r = rsqrtf(mean);
        if (live && !(mean >= kLeastMean && mean < __builtin_inff()))   // rare; the same in a head's lanes
            r = rescale<L>(x, a.eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] *= r * (isq ? wq[j] : wk[j]);
        if (a.table) {
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                y[j] = PAIRS ? x[j ^ 1] : __shfl(x[j], partner);
                if (d0 >= a.rot) y[j] = 0.f;  // not rotated: an infinity stays (times sn = 0 it is a NaN)
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = x[j] * cs[j] + y[j] * sn[j];
        }
        if (live) {
            if (isq) mf::IO<BF>::store8(a.q_out, t * a.q_out_row + (int64_t)h * D + d0, x);
            else mf::IO<BF>::store8(a.k_out, t * a.k_out_row + (int64_t)(h - a.Hq) * D + d0, x);
        }
    }
}

template <int D, bool BF>
hipError_t launch_rot(bool pairs, const RotateArgs &a, hipStream_t s) {
    const dim3 grid((unsigned)a.T), block(kRotThreads);
    if (pairs) hipLaunchKernelGGL((rotate_kernel<D, BF, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((rotate_kernel<D, BF, false>), grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rotate(bool bf16, int D, bool pairs, const RotateArgs &a, hipStream_t s) {
    if (a.T <= 0) return hipSuccess;
    if (a.T > INT32_MAX) return hipErrorInvalidValue;
    if (D == 128) return bf16 ? launch_rot<128, true>(pairs, a, s) : launch_rot<128, false>(pairs, a, s);
    if (D == 64) return bf16 ? launch_rot<64, true>(pairs, a, s) : launch_rot<64, false>(pairs, a, s);
    return hipErrorInvalidValue;
}

}  // namespace kda
