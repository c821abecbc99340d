// latent_common.h -- device helpers shared by the kernels of latent attention.
#pragma once

#include <type_traits>

#include "device_common.h"

namespace skg {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// f(0), f(1), .. f(N - 1), the numbers as types.
template <int N, class F>
__device__ __forceinline__ void each(F f) {
    if constexpr (N > 0) {
        each<N - 1>(f);
        f(std::integral_constant<int, N - 1>{});
    }
}

// ---------------------------------------------------------------- sequences
// New tokens of sequence b, their number and the first, within [0, T].
struct Tokens {
    int first, n;
};
__device__ __forceinline__ Tokens new_tokens(const int *starts, int b, int T) {
    if (!starts) return {b, 1};
    const int s = min(max(starts[b], 0), T), e = min(max(starts[b + 1], 0), T);
    return {s, max(e - s, 0)};
}

// pre[b] = sum of work(0 .. b - 1) for b = 0 .. B, by a workgroup of WAVES waves;
// `part` holds as many values.  Every thread calls it; ends with a barrier.
template <int WAVES, class Work>
__device__ __forceinline__ void block_prefix(int B, long *pre, long *part, Work work) {
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    long carry = 0;
    if (t == 0) pre[0] = 0;
    for (int b0 = 0; b0 < B; b0 += 64 * WAVES) {
        const int b = b0 + t;
        long v = b < B ? work(b) : 0;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const long u = __shfl_up(v, d, 64);
            if (lane >= d) v += u;
        }
        if (lane == 63) part[wave] = v;
        __syncthreads();
        long before = carry;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            if (w < wave) before += part[w];
            carry += part[w];
        }
        if (b < B) pre[b + 1] = before + v;
        __syncthreads();
    }
}
// The b with pre[b] <= x < pre[b + 1], for 0 <= x < pre[B].
__device__ __forceinline__ int find_sequence(const long *pre, int B, long x) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (pre[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// ---------------------------------------------------------------- tiles in LDS
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
// v, of which nothing is computed before this point: in a rare path, so that no
// register holds its addresses everywhere else.
__device__ __forceinline__ int here(int v) {
    asm volatile("" : "+v"(v));
    return v;
}
__device__ __forceinline__ Tokens uniform(Tokens q) { return {uniform(q.first), uniform(q.n)}; }

// An address in LDS, for the loads below.
__device__ __forceinline__ unsigned lds_address(const unsigned char *p) {
    return (unsigned)(uintptr_t)(__attribute__((address_space(3))) const unsigned char *)p;
}
// 16 bytes a lane from a buffer straight into LDS, at dst + AT + 16 * lane (dst uniform).
// Written as an instruction: beside the builtin, the compiler waits for every such
// load that is under way before a transposed read (vmcnt(0) in each step of the
// ring).  The ring's own waits count it.  It writes no register but m0, which no asm may
// declare, being reserved; that nothing else in these kernels uses m0 is checked in the
// built library.
//
// A buffer instruction may read a scalar register that a vector instruction wrote (the
// descriptors come from v_readlane) five wait states later at the earliest, and one after
// m0 was written; the compiler does not see that this is one.  The addition and s_nop 3
// are five, whatever stands before.  Waiting once for each new descriptor instead gains
// 1 % at most (150 e4m3 tokens of 12 sequences 76.0 us for 76.7, 512 tokens of 128 heads
// over 8192 rows 934 for 939, a prompt of 4096 759 for 759), and would be wrong where the
// compiler brings a spilled word back by v_readlane.
template <int AT>
__device__ __forceinline__ void ring_load16(Rsrc r, unsigned dst, unsigned off) {
    asm volatile("s_add_u32 m0, %0, %3\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(dst), "v"(off), "s"(r), "i"(AT)
                 : "memory", "scc");
}

// Rows lie in LDS with 16-byte pieces permuted: piece c of row r at c ^ swz(r) within
// 4, 8 or 16.  LDS has 64 banks of 4 bytes; a fragment read takes one piece of 16
// rows at once, or neighbouring ones of two times 8 rows (rows 0-3 and 12-15 beside 4-11),
// a transposed read four pieces of four rows, and either comes from 16
// different places of 16 bytes.  By the rows' size: 576 bytes (swz4), 1152 or 128 bytes, an odd
// multiple of 128 (swz8), 512 bytes (swz16).
__device__ __forceinline__ int swz4(int r) { return (r >> 2) & 3; }
// 0, 2, 3, 1: with it rows 0-3 and 12-15 differ from each other in the lowest bit alone.
__device__ __forceinline__ int swz_quarter(int r) {
    const int x = (r >> 2) & 3;
    return (((x ^ (x >> 1)) & 1) << 1) | (x >> 1);
}
__device__ __forceinline__ int swz8(int r) { return ((r & 2) << 1) | swz_quarter(r); }
__device__ __forceinline__ int swz16(int r) { return ((r & 3) << 2) | swz_quarter(r); }

// Four 2-byte values of this lane's column from four rows: lane i of 16 points at
// row i / 4, columns 4 (i % 4) .. + 3, and gets column i of rows 0 .. 3.
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
__device__ __forceinline__ s16x4 lds_transposed4(const unsigned char *p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
}
// Eight 1-byte values of this lane's column from eight rows: lane i of 16 points
// at row i / 2, columns 8 (i % 2) .. + 7.
typedef __attribute__((address_space(3))) i32x2 lds_i32x2;
__device__ __forceinline__ i32x2 lds_transposed8(const unsigned char *p) {
    return __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i32x2 *)p);
}

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

// Eight e4m3 codes -> eight bf16 values (exact).
__device__ __forceinline__ bf16x8 e4m3_to_bf16(i32x2 c) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.x, 1.0f, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.x, 1.0f, true);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.y, 1.0f, false);
    const bf16x2 e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.y, 1.0f, true);
    return bf16x8{a.x, a.y, b.x, b.y, d.x, d.y, e.x, e.y};
}

// A fragment as the matrix instruction takes it.
__device__ __forceinline__ bf16x8 as_bf16(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }
__device__ __forceinline__ bf16x8 as_bf16(s16x8 v) { return __builtin_bit_cast(bf16x8, v); }
__device__ __forceinline__ bf16x8 as_bf16(i32x2 v) { return e4m3_to_bf16(v); }

// Fragments read ahead: what stands before this in the source is read before, and x is
// there after it.  (Left to itself the compiler reads each fragment right before its use.)
template <class T, int N>
__device__ __forceinline__ void arrived(T (&x)[N]) {
#pragma unroll
    for (int i = N - 1; i >= 0; --i) asm volatile("" : "+v"(x[i])::"memory");  // LDS reads return in order: one wait
}

// ---------------------------------------------------------------- softmax
// Eight fp32 values -> bf16, to nearest, ties to even.
__device__ __forceinline__ bf16x8 to_bf16x8(const float *v) {
    bf16x8 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = (__bf16)v[i];
    return r;
}
// sum + the eight values.  Weights go to the second product in bf16, since the matrix
// instruction takes both operands in one type and the values have no more bits (weights of
// 16 bits would take a second product of what the first left).  The sum of the weights is made of the rounded ones, which
// the second product takes: what their roundings have in common then cancels in the
// quotient (errors of 1.0 to 1.4 times the output's own rounding instead of 1.1 to 1.5).
__device__ __forceinline__ float add_bf16x8(bf16x8 v, float sum) {
    const bf16x2 one{(__bf16)1.0f, (__bf16)1.0f};
    sum = __builtin_amdgcn_fdot2_f32_bf16(__builtin_shufflevector(v, v, 0, 1), one, sum, false);
    sum = __builtin_amdgcn_fdot2_f32_bf16(__builtin_shufflevector(v, v, 2, 3), one, sum, false);
    sum = __builtin_amdgcn_fdot2_f32_bf16(__builtin_shufflevector(v, v, 4, 5), one, sum, false);
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_shufflevector(v, v, 6, 7), one, sum, false);
}
__device__ __forceinline__ uint2 to_bf16x4(float a, float b, float c, float d) {
    const bf16x4 r{(__bf16)a, (__bf16)b, (__bf16)c, (__bf16)d};
    return __builtin_bit_cast(uint2, r);
}

// The other half's value: lane l and lane l ^ 32.
__device__ __forceinline__ float other_half_max(float v) {
    const unsigned u = __float_as_uint(v);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float other_half_sum(float v) {
    const unsigned u = __float_as_uint(v);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Sums of weights, and of weighted columns, joined by those of another part; one that
// saw no row has the maximum -inf and sums of 0.
template <int N>
__device__ __forceinline__ void add_part(float &m, float &l, f32x4 (&sum)[N], f32x2 ml, const f32x4 (&y)[N]) {
    const float next = fmaxf(m, ml.x), ref = next == -__builtin_inff() ? 0.0f : next;
    const float w0 = __builtin_amdgcn_exp2f(m - ref), w1 = __builtin_amdgcn_exp2f(ml.x - ref);
    m = next;
    l = __builtin_fmaf(w1, ml.y, l * w0);
#pragma unroll
    for (int v = 0; v < N; ++v)
#pragma unroll
        for (int u = 0; u < 4; ++u) sum[v][u] = __builtin_fmaf(w1, y[v][u], sum[v][u] * w0);
}

__device__ __forceinline__ bool not_finite(float v) {
    return (__float_as_uint(v) & 0x7F800000u) == 0x7F800000u;
}

}  // namespace skg
