// kernels_norm.hip -- residual addition and root-mean-square norm in one
// pass, y = s / sqrt(mean(s^2) + eps) * weight with s = x + residual.
//
// A row stays in the registers of the lanes that read it (16-byte vectors,
// widened to fp32), so x and the residual are read once and the sum of
// squares costs one reduction.  The 8-bit outputs are made from the same
// fp32 values: static e4m3, or MX codes whose 32-value blocks are the four
// neighbouring lanes of a quad.
//
// The factor of a row errs coherently in all its codes, and each rounding of a
// value moves it across more ties.  So the squares are added up in fp64 (no square
// leaves its range either), the factor is carried in two fp32 numbers, and a value
// goes to its 8-bit code as if it had not been rounded before.  Forty drawn calls had
// no code other than the exact one so; with sums in fp32 6, and 39 by rounding
// every step.  It takes 2-5 % of the time.
//
// Many rows are bound by HBM: 8192 x 7168 with a residual to MX moves 411 MB in
// 80 us, 5.1 TB/s, one call after another (89 us in a kernel trace; a copy on this
// card: 4.7 TB/s).  One row takes 3.9 us: a launch, a load, the reduction's barrier
// and a store, one after another.
#include <algorithm>

#include "device_common.h"
#include "internal.h"
#include "moe_internal.h"
#include "mx_common.h"

namespace skg {

namespace {

struct NormArgs {
    const uint16_t *x, *residual, *weight;
    const float *scale;
    uint8_t *y, *e8;
    uint16_t *residual_out;
    float eps;
    double inv_k;
    int M, K;
};

// A factor as the sum of two fp32 numbers.
struct Factor {
    float hi, lo;
};

template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v) {
    const unsigned long long u = (unsigned long long)__double_as_longlong(v);
    const unsigned lo = dpp_u32<CTRL>((unsigned)u), hi = dpp_u32<CTRL>((unsigned)(u >> 32));
    return __longlong_as_double((long long)((unsigned long long)hi << 32 | lo));
}
// Sum over 16 lanes, the same in each.
__device__ __forceinline__ double row16_sum(double v) {
    v += dpp_f64<kDppQuadSwap1>(v);
    v += dpp_f64<kDppQuadSwap2>(v);
    v += dpp_f64<kDppHalfMirror>(v);
    return v + dpp_f64<kDppMirror>(v);
}

// Sum over the wave's 64 lanes, the same in each.
__device__ __forceinline__ double wave_sum64(double v) {
    v = row16_sum(v);
    v += __shfl_xor(v, 16, 64);
    return v + __shfl_xor(v, 32, 64);
}

// 1 / sqrt(m): the hardware's (1 ulp) and what it leaves, from 1 - m hi^2 with
// exact products.  Where that is no number (m 0, infinite or NaN) hi stands alone.
__device__ __forceinline__ Factor rsqrt_factor(double m) {
    const float mh = (float)m, ml = (float)(m - (double)mh), c = __builtin_amdgcn_rsqf(mh);
    const float t = c * c, te = __builtin_fmaf(c, c, -t);
    const float d = __builtin_fmaf(-mh, te, __builtin_fmaf(-ml, t, __builtin_fmaf(-mh, t, 1.0f)));
    const float lo = 0.5f * c * d;
    return {c, fabsf(lo) <= fabsf(c) * 1e-3f ? lo : 0.0f};
}
// f / v, likewise.
__device__ __forceinline__ Factor divided(Factor f, float v) {
    const float q = 1.0f / v, ql = __builtin_fmaf(-q, v, 1.0f) * q, hi = f.hi * q;
    const float lo = __builtin_fmaf(f.hi, q, -hi) + __builtin_fmaf(f.hi, ql, f.lo * q);
    return {hi, fabsf(lo) <= fabsf(hi) * 1e-3f ? lo : 0.0f};
}

// a / v to 2 ulp for any v: the hardware's reciprocal takes no subnormals and makes none.
__device__ __forceinline__ float quotient(float a, float v) {
    const float m = fabsf(v) < 0x1p-100f ? 0x1p50f : fabsf(v) > 0x1p100f ? 0x1p-50f : 1.0f;
    return a * m * __builtin_amdgcn_rcpf(v * m * m) * m;
}

// y + rest, |rest| up to half a step of y, as the odd one of the two fp32 numbers
// around it: a tie between codes, an even number, is then met only by y itself,
// so that the code is that of the sum.  y infinite, NaN or 0: as it is.
__device__ __forceinline__ float to_odd(float y, float rest) {
    const unsigned b = __float_as_uint(y);
    const int step = ((int)(__float_as_uint(rest) ^ b) >> 31) | 1;  // away from 0, or towards it
    return (b & 1u) == 0 && rest != 0.0f && fabsf(rest) < fabsf(y) ? __uint_as_float(b + (unsigned)step) : y;
}

// The eight fp32 sums of vector i of a row.
__device__ __forceinline__ void norm_load(const NormArgs &a, size_t row0, int i, float (&s)[8]) {
    bf16x8_to_f32(*reinterpret_cast<const u32x4 *>(a.x + row0 + (size_t)i * 8), s);
    if (a.residual) {
        float r[8];
        bf16x8_to_f32(*reinterpret_cast<const u32x4 *>(a.residual + row0 + (size_t)i * 8), r);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] += r[j];
    }
}

// Vector i of a row's output.  c: the row's factor, over the scale for e4m3;
// plain: the factor alone, in one number.
template <int OUT>
__device__ __forceinline__ void norm_store(const NormArgs &a, size_t row0, int i,
                                           const float (&s)[8], Factor c, float plain) {
    float w[8], y[8];
    bf16x8_to_f32(*reinterpret_cast<const u32x4 *>(a.weight + (size_t)i * 8), w);
    // s * (hi + lo) * w, in effect rounded once; what is left of it in `rest`
    auto value = [&](int j, float *rest) {
        const float p = s[j] * c.hi, e = __builtin_fmaf(s[j], c.lo, __builtin_fmaf(s[j], c.hi, -p)) * w[j];
        const float v = __builtin_fmaf(p, w[j], e);
        if (rest) *rest = __builtin_fmaf(p, w[j], -v) + e;
        return v;
    };
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = value(j, nullptr);
    // Past fp32's range (a scale near 0, an infinite weight) what is left over is
    // infinite too, and their sum NaN: such values by the formula as it stands.
    // Ties between codes end in 19 zeros, and so do infinities and that NaN.
    bool again;
    if constexpr (OUT == SKG_NORM_BF16) {
        float finite = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) finite = __builtin_fmaf(y[j], 0.0f, finite);
        again = finite != 0.0f;
    } else {
        unsigned low = ~0u;
#pragma unroll
        for (int j = 0; j < 8; ++j) low = min(low, __float_as_uint(y[j]) << 13);
        again = low == 0;
    }
    if (__builtin_expect(again, 0)) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float rest;
            const float v = value(j, &rest);
            if (!(fabsf(v) < __builtin_inff())) {
                y[j] = s[j] * plain * w[j];
                if constexpr (OUT == SKG_NORM_E4M3) y[j] = quotient(y[j], a.scale[0]);
            } else if constexpr (OUT != SKG_NORM_BF16) {
                y[j] = to_odd(v, rest);
            }
        }
    }
    const size_t at = row0 + (size_t)i * 8;
    if constexpr (OUT == SKG_NORM_BF16) {
        *reinterpret_cast<u32x4 *>(a.y + at * 2) = f32x8_to_bf16(y);
    } else if constexpr (OUT == SKG_NORM_E4M3) {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = quant_clamp(y[j]);
        *reinterpret_cast<uint2 *>(a.y + at) = mx_codes8_e4m3(y, 1.0f);
    } else {
        const int e = mx_store8<kMxE4m3>(y, a.y, at);
        if ((i & 3) == 0) a.e8[at / 32] = (uint8_t)e;
    }
}

}  // namespace

// TPR lanes per row (64: one wave, four rows a workgroup; else a whole
// workgroup), V vectors of 8 values per lane held in registers; V == 0: rows
// longer than the registers hold, read a second time for the output.
template <int OUT, int TPR, int V>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR, 8) rmsnorm_kernel(NormArgs a) {
    constexpr int ROWS = TPR < 256 ? 256 / TPR : 1;
    const int t = threadIdx.x % TPR;
    const int row = blockIdx.x * ROWS + threadIdx.x / TPR;
    if (ROWS > 1 && row >= a.M) return;  // whole waves; no barrier below when ROWS > 1
    const int k8 = a.K / 8;
    const size_t row0 = (size_t)row * a.K;
    constexpr int N = V > 0 ? V : 1;
    float s[N][8];
    double sq = 0.0;
    const int nv = V > 0 ? V : (k8 + TPR - 1) / TPR;
#pragma unroll
    for (int v = 0; v < nv; ++v) {
        const int i = t + v * TPR;
        float(&sv)[8] = s[V > 0 ? v : 0];
#pragma unroll
        for (int j = 0; j < 8; ++j) sv[j] = 0.0f;
        if (i < k8) norm_load(a, row0, i, sv);
#pragma unroll
        for (int j = 0; j < 8; ++j) sq = __builtin_fma((double)sv[j], (double)sv[j], sq);
    }
    sq = wave_sum64(sq);
    if constexpr (TPR > 64) {
        __shared__ double part[TPR / 64];
        if ((threadIdx.x & 63) == 0) part[threadIdx.x / 64] = sq;
        __syncthreads();
        // every lane of a row of 16 adds the same up to 16 partial sums
        sq = row16_sum((threadIdx.x & 15) < TPR / 64 ? part[threadIdx.x & 15] : 0.0);
    }
    double mean = __builtin_fma(sq, a.inv_k, (double)a.eps);
    // Past either end of what the factor's fp32 takes the row is moved by the power
    // of two that leaves its mean square near one; 0, infinite and NaN stay.
    float move = 1.0f;
    if (__builtin_expect(!(mean >= 0x1p-70 && mean <= 0x1p110), 0) && mean > 0.0 && mean <= 0x1p300) {
        const int n = min(max(-(ilogb(mean) / 2), -120), 120);
        move = ldexpf(1.0f, n);
        mean = ldexp(mean, 2 * n);
    }
    Factor c = rsqrt_factor(mean);
    const float plain = c.hi;
    if constexpr (OUT == SKG_NORM_E4M3) c = divided(c, a.scale[0]);
#pragma unroll
    for (int v = 0; v < nv; ++v) {
        const int i = t + v * TPR;
        if (i >= k8) continue;  // K / 8 is a multiple of 4 for MX: whole quads
        float(&sv)[8] = s[V > 0 ? v : 0];
        if constexpr (V == 0) norm_load(a, row0, i, sv);
        if (a.residual_out)
            *reinterpret_cast<u32x4 *>(a.residual_out + row0 + (size_t)i * 8) = f32x8_to_bf16(sv);
        if (__builtin_expect(move != 1.0f, 0))
#pragma unroll
            for (int j = 0; j < 8; ++j) sv[j] *= move;
        norm_store<OUT>(a, row0, i, sv, c, plain);
    }
}

namespace {

template <int OUT, int TPR, int V>
int go(const NormArgs &a, hipStream_t stream) {
    constexpr int ROWS = TPR < 256 ? 256 / TPR : 1;
    hipLaunchKernelGGL((rmsnorm_kernel<OUT, TPR, V>), dim3((unsigned)((a.M + ROWS - 1) / ROWS)),
                       dim3(TPR < 256 ? 256 : TPR), 0, stream, a);
    return (int)hipGetLastError();
}

// One vector of 8 values a lane up to 8192 values (in us, with residual, to MX,
// at 1, 1024 and 8192 rows; beside it half the lanes with two each):
//   2880 values   3.0  7.7 37.9    3.9  8.2 35.3
//   4096          3.2  9.6 44.1    4.2 10.0 43.8
//   7168          3.7 13.8 87.0    4.5 14.3 80.6
// so the shorter chain wins for few rows everywhere, and for many rows two
// vectors only where a row needs more than 512 lanes.
template <int OUT>
int pick(const NormArgs &a, hipStream_t stream) {
    const int k8 = a.K / 8;
    if (k8 <= 64) return go<OUT, 64, 1>(a, stream);
    if (k8 <= 256) return go<OUT, 256, 1>(a, stream);
    if (k8 <= 512) return go<OUT, 512, 1>(a, stream);
    if (k8 <= 1024) return a.M <= 1024 ? go<OUT, 1024, 1>(a, stream) : go<OUT, 512, 2>(a, stream);
    if (k8 <= 2048) return go<OUT, 1024, 2>(a, stream);
    // longer rows are read twice: 16384 values, 4096 rows: 108 us against 90
    return go<OUT, 1024, 0>(a, stream);
}

}  // namespace

int launch_rmsnorm(const void *x, const void *residual, const void *weight, float eps,
                   int out_format, const float *scale, void *y, void *e8, void *residual_out,
                   int M, int K, hipStream_t stream) {
    // a grid has fewer than 2^32 work-items: 2^21 rows of up to 1024 lanes at a time
    constexpr int kMostRows = 1 << 21;
    for (size_t m0 = 0; m0 < (size_t)M; m0 += kMostRows) {
        const size_t at = m0 * K;
        auto rows = [&](const void *p) { return p ? (const uint16_t *)p + at : nullptr; };
        const NormArgs a{rows(x), rows(residual), (const uint16_t *)weight, scale,
                         (uint8_t *)y + (out_format == SKG_NORM_BF16 ? 2 * at : at),
                         e8 ? (uint8_t *)e8 + at / 32 : nullptr, const_cast<uint16_t *>(rows(residual_out)),
                         eps, 1.0 / K, (int)std::min<size_t>(M - m0, kMostRows), K};
        const int e = out_format == SKG_NORM_BF16   ? pick<SKG_NORM_BF16>(a, stream)
                      : out_format == SKG_NORM_E4M3 ? pick<SKG_NORM_E4M3>(a, stream)
                                                    : pick<SKG_NORM_MX>(a, stream);
        if (e != (int)hipSuccess) return e;
    }
    return (int)hipSuccess;
}

}  // namespace skg
