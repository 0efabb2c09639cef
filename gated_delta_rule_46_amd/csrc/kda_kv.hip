// kda_kv.hip -- the 8-bit key/value cache: quantised as it is written, read back.
//
// A page holds `page` consecutive tokens of one sequence.  For each page and
// head the keys (and, apart from them, the values) are e4m3 codes c with one
// scale s = 2^e, x ~ c s, where e is the smallest exponent with
// amax <= 448 * 2^e over the finite values that the page holds.  A power of two
// costs a floating code no precision (its relative step does not depend on the
// scale) and makes every product with it exact: the codes are the values
// rounded once to e4m3's grid, c s is exact in bf16 and in fp32, and a page
// whose scale grows rounds its older codes again only where they fall below the
// grid's smallest normal.  e stays within [-100, 119], so that c s is a normal
// number; larger values and infinities saturate at 448 s, NaN stays NaN.
//
// Both kernels move each byte once and are bound by HBM for long calls and by
// their launch for a decode step.  kv_write: one workgroup per (page touched,
// head, keys or values) holds all new elements of its page in registers between
// the maximum and the conversion, so they are read once.  It owns the page's
// codes and scale of that head: no two workgroups meet.  Eight prompts of 2,048 to
// 16,384 tokens at 8 heads of 128 with bf16 rows: 95 us written, 94 read back (0.46 GB
// each, 4.9 TB/s), with fp32 rows at 4.7 and 4.5 TB/s; one token on each of 64 sequences
// 5.8 us, the last 65 tokens of each read back 9.3.

#include "kda_attn.h"
#include "kda_mfma.h"

namespace kda {
namespace {

constexpr int kKvThreads = 256;
constexpr int kScaleExpMin = -100, kScaleExpMax = 119;
constexpr float kCodeMax = 448.f;

// x limited to the code range; a NaN stays (both comparisons fail).
__device__ __forceinline__ float limited(float x) {
    x = x > kCodeMax ? kCodeMax : x;
    return x < -kCodeMax ? -kCodeMax : x;
}

// Smallest e (in range) with amax <= 448 * 2^e.  amax = 1.f * 2^x: 448 = 1.75 * 2^8.
__device__ __forceinline__ int scale_exp(float amax) {
    const uint32_t b = f32_bits(amax);
    const int x = (int)(b >> 23) - 127 - 8;
    const int e = x + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    return amax > 0.f ? min(max(e, kScaleExpMin), kScaleExpMax) : kScaleExpMin;
}

// 2^e for e in [-126, 127]
__device__ __forceinline__ float pow2(int e) { return bits_f32((uint32_t)(e + 127) << 23); }

// Workgroup x of the page axis -> a sequence and one of the pages that its new
// tokens touch.  A sequence of len tokens touches at most (len - 1) / page + 2
// pages, which is at most first(n + 1) - first(n) for first(n) = cu[n] / page +
// 2 n: the pages of all sequences are numbered without a pass over them.
template <int D, int PAGE, bool BF>
__global__ __launch_bounds__(kKvThreads) void kv_write_kernel(const KvArgs a) {
    constexpr int CH = D / 8;                                     // 8-element pieces per row
    constexpr int NC = (PAGE * CH + kKvThreads - 1) / kKvThreads;   // pieces per thread
    __shared__ float s_max[kKvThreads / 64];
    const int tid = threadIdx.x;
    // heads, keys and values of the same tokens are neighbours: their rows lie together
    const uint32_t hz = blockIdx.x % (2 * (uint32_t)a.Hk);
    const int64_t x = blockIdx.x / (2 * (uint32_t)a.Hk);
    const bool is_v = hz >= (uint32_t)a.Hk;
    const int h = (int)(is_v ? hz - a.Hk : hz);
    const int n = last_not_above(a.N, x, [&](int i) { return a.cu[i] / PAGE + 2 * (int64_t)i; });
    const int64_t c0 = a.cu[n], c1 = min(a.cu[n + 1], a.T);
    const int64_t kvl = a.kv_len[n], start = kvl - (c1 - c0);     // position of the first new token
    if (c0 < 0 || c1 <= c0) return;
    const int64_t from = max(start, (int64_t)0);
    const int64_t b = from / PAGE + (x - (c0 / PAGE + 2 * (int64_t)n));
    const int64_t lo = max(from, b * PAGE), hi = min(kvl, (b + 1) * PAGE);
    if (lo >= hi || b >= a.width) return;
    const int32_t pid = a.table[(int64_t)n * a.width + b];
    if (pid < 0 || pid >= a.n_pages) return;

    const int first = (int)(lo - b * PAGE), rows = (int)(hi - lo);
    const void *src = is_v ? a.v : a.k;
    const int64_t row = is_v ? a.v_row : a.k_row;
    const int64_t at = (c0 + (lo - start)) * row + (int64_t)h * D;
    uint8_t *codes = (is_v ? a.v_codes : a.k_codes) + ((int64_t)pid * a.Hk + h) * (PAGE * D);
    float *scale = (is_v ? a.v_scale : a.k_scale) + (int64_t)pid * a.Hk + h;
    const float held = first > 0 ? *scale : 0.f;

    float v[NC][8];
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = i * kKvThreads + tid, r = c / CH;
        if (r < rows) {
            load8_once<BF>(src, at + r * row + (c % CH) * 8, v[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float y = fabsf(v[i][j]);
                m = y < __builtin_inff() ? fmaxf(m, y) : m;       // finite values only
            }
        }
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
    if ((tid & 63) == 0) s_max[tid >> 6] = m;
    __syncthreads();                                              // and every thread has read *scale
    m = fmaxf(fmaxf(s_max[0], s_max[1]), fmaxf(s_max[2], s_max[3]));
    const int e = scale_exp(m);
    const float need = pow2(e);
    const float s = fmaxf(held, need), inv = held > need ? 1.f / held : pow2(-e);

#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = i * kKvThreads + tid, r = c / CH;
        if (r < rows) {
            uint2 w;
            w.x = codes4(limited(v[i][0] * inv), limited(v[i][1] * inv), limited(v[i][2] * inv),
                         limited(v[i][3] * inv));
            w.y = codes4(limited(v[i][4] * inv), limited(v[i][5] * inv), limited(v[i][6] * inv),
                         limited(v[i][7] * inv));
            *(uint2 *)(codes + (first + r) * D + (c % CH) * 8) = w;
        }
    }
    if (first > 0 && s > held) {                                  // older rows, to the larger scale
        const float f = held / s;
        for (int c = tid; c < first * CH; c += kKvThreads) {
            uint2 w = *(const uint2 *)(codes + c * 8);
            float y[8];
            uncode4(w.x, y);
            uncode4(w.y, y + 4);
            w.x = codes4(y[0] * f, y[1] * f, y[2] * f, y[3] * f);
            w.y = codes4(y[4] * f, y[5] * f, y[6] * f, y[7] * f);
            *(uint2 *)(codes + c * 8) = w;
        }
    }
    if (tid == 0 && s != held) *scale = s;
}

// One workgroup per ROWS packed tokens, whose places are looked up side by side first;
// then a thread takes the codes of 16 bytes of output at a time, kReadDeep of them in
// flight.  Tokens without a page read as zeros.  ROWS: 16, or 4 while that leaves
// compute units idle.
constexpr int kReadDeep = 8;

template <int D, bool BF, int ROWS>
__global__ __launch_bounds__(kKvThreads) void kv_read_kernel(const KvArgs a) {
    constexpr int PC = BF ? 8 : 4;            // codes per piece
    constexpr int CH = D / PC;                // pieces per row
    __shared__ int64_t s_row[ROWS];           // pid * Hk * page + row of the page, -1: absent, -2: not there
    __shared__ int s_pid[ROWS];
    const int tid = threadIdx.x;
    const int64_t t0 = (int64_t)blockIdx.x * ROWS;
    if (t0 >= a.cu[a.N]) return;              // rows behind the last sequence stay as they are
    int n = last_not_above(a.N, t0, [&](int i) { return a.cu[i]; });
    if (tid < ROWS) {
        const int64_t t = t0 + tid;
        while (n < a.N && t >= a.cu[n + 1]) ++n;
        int64_t place = -2;
        int pid = -1;
        if (t < a.T && n < a.N && t >= a.cu[n]) {
            const int64_t pos = a.kv_len[n] - a.cu[n + 1] + t;
            const int shift = __builtin_ctz(a.page);
            place = -1;
            if (pos >= 0 && (pos >> shift) < a.width) {
                pid = a.table[(int64_t)n * a.width + (pos >> shift)];
                if (pid >= 0 && pid < a.n_pages)
                    place = (int64_t)pid * a.Hk * a.page + (pos & (a.page - 1));
            }
        }
        s_row[tid] = place;
        s_pid[tid] = pid;
    }
    __syncthreads();
    const int per = a.Hk * CH;                // pieces per token of keys, and of values
    const int all = 2 * ROWS * per;
    for (int c0 = tid; c0 < all; c0 += kReadDeep * kKvThreads) {
        uint32_t w[kReadDeep][PC / 4];
        float s[kReadDeep];
        int64_t to[kReadDeep];
        bool is_v[kReadDeep];
#pragma unroll
        for (int u = 0; u < kReadDeep; ++u) {
            const int c = c0 + u * kKvThreads;
#pragma unroll
            for (int j = 0; j < PC / 4; ++j) w[u][j] = 0;
            s[u] = 1.f;
            to[u] = -1;
            is_v[u] = false;
            if (c >= all) continue;
            const int ix = (int)((uint32_t)c / (uint32_t)per), x = c - ix * per, i = ix >> 1;
            const int64_t place = s_row[i];
            if (place == -2) continue;
            is_v[u] = ix & 1;
            const int h = x / CH, d = x % CH * PC;
            to[u] = ((t0 + i) * a.Hk + h) * D + d;
            if (place >= 0) {
                const uint8_t *p = (is_v[u] ? a.v_codes : a.k_codes) + (place + (int64_t)h * a.page) * D + d;
#pragma unroll
                for (int j = 0; j < PC / 4; ++j) w[u][j] = ((const uint32_t *)p)[j];
                s[u] = (is_v[u] ? a.v_scale : a.k_scale)[(int64_t)s_pid[i] * a.Hk + h];
            }
        }
#pragma unroll
        for (int u = 0; u < kReadDeep; ++u) {
            if (to[u] < 0) continue;
            float y[PC];
#pragma unroll
            for (int j = 0; j < PC / 4; ++j) uncode4(w[u][j], y + 4 * j);
#pragma unroll
            for (int j = 0; j < PC; ++j) y[j] *= s[u];
            void *out = is_v[u] ? a.v_out : a.k_out;
            if constexpr (BF) mf::IO<true>::store8(out, to[u], y);
            else *(float4 *)((float *)out + to[u]) = make_float4(y[0], y[1], y[2], y[3]);
        }
    }
}

template <int D, int PAGE>
hipError_t launch_write(bool bf16, const KvArgs &a, hipStream_t s) {
    const int64_t blocks = (a.T / PAGE + 2 * (int64_t)a.N) * 2 * a.Hk;
    if (blocks > INT32_MAX) return hipErrorInvalidValue;
    const dim3 grid((unsigned)blocks), block(kKvThreads);
    if (bf16) hipLaunchKernelGGL((kv_write_kernel<D, PAGE, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((kv_write_kernel<D, PAGE, false>), grid, block, 0, s, a);
    return hipGetLastError();
}

template <int D>
hipError_t launch_write_page(bool bf16, const KvArgs &a, hipStream_t s) {
    switch (a.page) {
        case 16: return launch_write<D, 16>(bf16, a, s);
        case 32: return launch_write<D, 32>(bf16, a, s);
        case 64: return launch_write<D, 64>(bf16, a, s);
        case 128: return launch_write<D, 128>(bf16, a, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_kv_write(bool bf16, int D, const KvArgs &a, hipStream_t s) {
    if (a.T <= 0 || a.N <= 0) return hipSuccess;
    if (D == 128) return launch_write_page<128>(bf16, a, s);
    if (D == 64) return launch_write_page<64>(bf16, a, s);
    return hipErrorInvalidValue;
}

template <int D, bool BF>
static hipError_t launch_read(const KvArgs &a, hipStream_t s) {
    const dim3 block(kKvThreads);
    if (a.T < 16 * 1024) {
        hipLaunchKernelGGL((kv_read_kernel<D, BF, 4>), dim3((unsigned)((a.T + 3) / 4)), block, 0, s, a);
    } else {
        const int64_t g = (a.T + 15) / 16;
        if (g > INT32_MAX) return hipErrorInvalidValue;
        hipLaunchKernelGGL((kv_read_kernel<D, BF, 16>), dim3((unsigned)g), block, 0, s, a);
    }
    return hipGetLastError();
}

hipError_t launch_kv_read(bool bf16, int D, const KvArgs &a, hipStream_t s) {
    if (a.T <= 0 || a.N <= 0) return hipSuccess;
    if (D == 128) return bf16 ? launch_read<128, true>(a, s) : launch_read<128, false>(a, s);
    if (D == 64) return bf16 ? launch_read<64, true>(a, s) : launch_read<64, false>(a, s);
    return hipErrorInvalidValue;
}

}  // namespace kda
