// kernels_latent_append.hip -- new tokens' latents into the paged cache: the norm
// of 512 values, the rotation of 64, one rounding to the cache's type; and the
// rotation of the queries' 64 a head.
//
// A token's row is one wave's, 8 latents a lane and one of the 32 pairs in each of
// the first 32 lanes; everything about it is in fp64, so that a code next to a tie is
// the exact one's.  That costs 2 us of 19 at 8192 tokens of 16 heads to e4m3 (59 MB at
// 3.1 TB/s); one token of 128 heads takes 2.6 us, four trips to memory one after another.
// Rows before queries: both kinds in turn, on every XCD, took 23 us for 19.  Two heads'
// queries a thread: 3.4 us for one token, 19.8 for 18.6 at 8192.
#include <algorithm>

#include "internal.h"
#include "latent_common.h"
#include "latent_internal.h"

namespace skg {

namespace {

constexpr int kStartsLds = 1024;  // sequences whose starts are searched in LDS

// v in fp32 such that its next rounding is that of v: where v lies between two
// fp32 numbers, the odd one of them (a tie of the next rounding is even).  One beyond
// the largest number becomes that number, a NaN stays one.
__device__ __forceinline__ float to_odd(double v) {
    const float f = (float)v;
    const double d = (double)f;
    const unsigned u = __float_as_uint(f);
    const unsigned other = (d < v) != (bool)(u >> 31) ? u + 1 : u - 1;  // the fp32 number on v's other side
    return __uint_as_float((u & 1u) || d == v ? u : other);
}
// The quotient u / s as the division's instructions end, without its scaling: with
// inv = 1 / s rounded, one correction of u inv; exact where the quotient is.  Without it
// where it would meet an infinity.
__device__ __forceinline__ double over(double u, double s, double inv) {
    const double q = u * inv;
    return fabs(q) < __builtin_inf() && inv != 0.0 ? __builtin_fma(__builtin_fma(-q, s, u), inv, q) : q;
}

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
    return v;
}

// The sequence of token t and its row in the cache; false: the token is none's.
struct Where {
    int b, row;
};
__device__ __forceinline__ bool find_token(const LatentAppendArgs &a, const int *starts, int t, int cap, Where &w) {
    int b = t, end = t + 1;
    if (a.q_starts) {
        // the last sequence that starts at or before t
        int lo = 0, hi = a.B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (starts[mid] <= t) lo = mid;
            else hi = mid;
        }
        b = lo;
        const int s = min(max(starts[b], 0), a.T);
        end = min(max(starts[b + 1], 0), a.T);
        if (t < s || t >= end) return false;
    }
    w.b = b;
    w.row = min(max(a.kv_lens[b], 0), cap) - (end - t);
    return true;
}

// (a, b) turned by (c, s)
template <class F>
__device__ __forceinline__ void turn(F &a, F &b, F c, F s) {
    const F x = a * c - b * s;
    b = a * s + b * c;
    a = x;
}

}  // namespace

// Blocks [0, rows): four tokens' rows each; the others: 16 values of a head's
// queries a thread.  HALVES: value i turns with i + 32, else 2i with 2i + 1.
template <bool HALVES, bool E4M3>
__global__ void __launch_bounds__(256) latent_append_kernel(LatentAppendArgs a, int rows) {
    __shared__ int lds_starts[kStartsLds + 1];
    const int *starts = a.q_starts;
    if (a.q_starts && a.B <= kStartsLds) {
        for (int i = threadIdx.x; i <= a.B; i += 256) lds_starts[i] = a.q_starts[i];
        __syncthreads();
        starts = lds_starts;
    }
    const int cap = (int)min((long)a.W << a.page_shift, 0x7FFFFFFFL - 64);
    const int lane = threadIdx.x & 63;
    if ((int)blockIdx.x < rows) {
        const int t = (int)blockIdx.x * 4 + (int)(threadIdx.x >> 6);
        Where w;
        if (t >= a.T || !find_token(a, starts, t, cap, w)) return;
        const uint16_t *x = a.kv + (size_t)t * a.kv_stride;
        const u32x4 raw = *reinterpret_cast<const u32x4 *>(x + lane * 8);
        // pair `lane` of the rotated part
        const int i0 = HALVES ? (lane & 31) : 2 * (lane & 31), i1 = HALVES ? i0 + 32 : i0 + 1;
        double k0 = bf16_to_f32(x[SKG_LATENT + i0]), k1 = bf16_to_f32(x[SKG_LATENT + i1]);
        const float *turnrow = a.rotations + (size_t)max(w.row, 0) * SKG_LATENT_ROPE;
        turn(k0, k1, (double)turnrow[lane & 31], (double)turnrow[32 + (lane & 31)]);
        double y[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            y[2 * j] = bf16_lo(raw[j]);
            y[2 * j + 1] = bf16_hi(raw[j]);
        }
        if (a.weight) {
            const u32x4 g = *reinterpret_cast<const u32x4 *>(a.weight + lane * 8);
            double sq = 0.0;
#pragma unroll
            for (int j = 0; j < 8; ++j) sq = __builtin_fma(y[j], y[j], sq);
            const double f = 1.0 / sqrt(wave_sum64(sq) * (1.0 / SKG_LATENT) + (double)a.eps);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                y[2 * j] *= f * bf16_lo(g[j]);
                y[2 * j + 1] *= f * bf16_hi(g[j]);
            }
        }
        u32x4 o;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            o[j] = f32_to_bf16_rne(to_odd(y[2 * j])) | (unsigned)f32_to_bf16_rne(to_odd(y[2 * j + 1])) << 16;
        const uint16_t r0 = f32_to_bf16_rne(to_odd(k0)), r1 = f32_to_bf16_rne(to_odd(k1));
        auto put = [&](uint16_t *row) {
            *reinterpret_cast<u32x4 *>(row + lane * 8) = o;
            if (lane >= 32) return;
            if (HALVES) {
                row[SKG_LATENT + i0] = r0;
                row[SKG_LATENT + i1] = r1;
            } else {
                *reinterpret_cast<unsigned *>(row + SKG_LATENT + i0) = r0 | (unsigned)r1 << 16;
            }
        };
        if (a.latent_out) put(a.latent_out + (size_t)t * SKG_LATENT_ROW);
        if (w.row < 0) return;
        const int page = a.table[(size_t)w.b * a.W + (w.row >> a.page_shift)];
        if (page < 0 || page >= a.pages) return;
        const size_t at = (((size_t)page << a.page_shift) + (w.row & ((1 << a.page_shift) - 1))) * SKG_LATENT_ROW;
        if constexpr (!E4M3) {
            put(reinterpret_cast<uint16_t *>(a.cache) + at);
        } else {
            const double s = a.scale[0], inv = 1.0 / s;
            auto code2 = [&](double u, double v) {
                return (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(quant_clamp(to_odd(over(u, s, inv))), quant_clamp(to_odd(over(v, s, inv))), 0, false) & 0xFFFFu;
            };
            uint2 c;
            c.x = code2(y[0], y[1]) | code2(y[2], y[3]) << 16;
            c.y = code2(y[4], y[5]) | code2(y[6], y[7]) << 16;
            *reinterpret_cast<uint2 *>(a.cache + at + lane * 8) = c;
            const unsigned r = code2(k0, k1);
            if (lane < 32) {
                uint8_t *row = a.cache + at + SKG_LATENT;
                if (HALVES) {
                    row[i0] = (uint8_t)r;
                    row[i1] = (uint8_t)(r >> 8);
                } else {
                    *reinterpret_cast<uint16_t *>(row + i0) = (uint16_t)r;
                }
            }
        }
        return;
    }
    // four threads a head: pairs 8 c .. 8 c + 7
    const long u = (long)(blockIdx.x - rows) * 256 + threadIdx.x;
    const int per = a.H * 4;
    const int t = (int)(u / per), e = (int)(u - (long)t * per), h = e >> 2, c = e & 3;
    Where w;
    if (t >= a.T || !find_token(a, starts, t, cap, w)) return;
    const uint16_t *q = a.q + (size_t)t * a.q_token + (size_t)h * a.q_head;
    uint16_t *o = a.q_out + (size_t)t * a.o_token + (size_t)h * a.o_head;
    const int p0 = HALVES ? 8 * c : 16 * c, p1 = HALVES ? p0 + 32 : p0 + 8;
    const u32x4 lo = *reinterpret_cast<const u32x4 *>(q + p0), hi = *reinterpret_cast<const u32x4 *>(q + p1);
    const float *r = a.rotations + (size_t)max(w.row, 0) * SKG_LATENT_ROPE + 8 * c;
    float cs[8], sn[8];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        *reinterpret_cast<f32x4 *>(cs + 4 * j) = *reinterpret_cast<const f32x4 *>(r + 4 * j);
        *reinterpret_cast<f32x4 *>(sn + 4 * j) = *reinterpret_cast<const f32x4 *>(r + 32 + 4 * j);
    }
    float x[8], y[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (HALVES) {
            x[2 * j] = bf16_lo(lo[j]);
            x[2 * j + 1] = bf16_hi(lo[j]);
            y[2 * j] = bf16_lo(hi[j]);
            y[2 * j + 1] = bf16_hi(hi[j]);
        } else {
            x[j] = bf16_lo(lo[j]);
            y[j] = bf16_hi(lo[j]);
            x[4 + j] = bf16_lo(hi[j]);
            y[4 + j] = bf16_hi(hi[j]);
        }
    }
    u32x4 ol, oh;
#pragma unroll
    for (int j = 0; j < 8; ++j) turn(x[j], y[j], cs[j], sn[j]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        auto two = [](float v, float z) { return f32_to_bf16_rne(v) | (unsigned)f32_to_bf16_rne(z) << 16; };
        ol[j] = HALVES ? two(x[2 * j], x[2 * j + 1]) : two(x[j], y[j]);
        oh[j] = HALVES ? two(y[2 * j], y[2 * j + 1]) : two(x[4 + j], y[4 + j]);
    }
    *reinterpret_cast<u32x4 *>(o + p0) = ol;
    *reinterpret_cast<u32x4 *>(o + p1) = oh;
}

int launch_latent_append(const LatentAppendArgs &a, int style, bool e4m3, hipStream_t stream) {
    const int rows = (a.T + 3) / 4;
    const long queries = ((long)a.T * a.H * 4 + 255) / 256;
    const dim3 grid((unsigned)(rows + queries));
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, a, rows); };
    if (style == SKG_ROPE_HALVES) e4m3 ? go(latent_append_kernel<true, true>) : go(latent_append_kernel<true, false>);
    else e4m3 ? go(latent_append_kernel<false, true>) : go(latent_append_kernel<false, false>);
    return (int)hipGetLastError();
}

}  // namespace skg
