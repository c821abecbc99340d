// mx_common.h -- microscaling (MX) on gfx950: 32 consecutive values of a row
// share one power of two, stored as the byte e of 2^(e - 127) (e8m0).
//
// The scale rule is the smallest power of two that keeps the block inside
// the codes' range, amax <= largest * 2^(e - 127), so nothing saturates
// (the rule of floor(log2(amax)) saturates up to a fifth of a binade).  With
// amax = 1.m * 2^(E - 127) and largest = 1.75 * 2^8 (e4m3) or 1.5 * 2^2
// (e2m1) that is e = E - 8 + (1.m > 1.75) or E - 2 + (1.m > 1.5): integer
// work on amax's bits, no rounding.  The product v * 2^(127 - e) is exact
// (or far below the smallest code), so a code is rounded once.
#pragma once

#include "device_common.h"

namespace skg {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// The codes of a format as the matrix instruction names them.
constexpr int kMxE4m3 = 0;
constexpr int kMxE2m1 = 4;
// Bytes of n codes.
template <int FMT>
__host__ __device__ constexpr size_t mx_bytes(size_t n) {
    return FMT == kMxE4m3 ? n : n / 2;
}

// The scale byte of a block with largest magnitude amax (>= 0, or NaN): 127
// for an all-zero block, 255 (NaN) if a value is infinite or NaN, else in
// [0, 253].  fp32-subnormal amax falls under the clamp at 0.
template <int FMT>
__device__ __forceinline__ int mx_exponent(float amax) {
    const unsigned u = __float_as_uint(amax) & 0x7FFFFFFFu;
    const int E = (int)(u >> 23);
    const int over = (u & 0x7FFFFFu) > (FMT == kMxE4m3 ? 0x600000u : 0x400000u) ? 1 : 0;
    const int e = max(E - (FMT == kMxE4m3 ? 8 : 2) + over, 0);
    return u == 0 ? 127 : (E == 255 ? 255 : e);
}

// 2^(127 - e) for e in [0, 253]; for 255 the codes do not matter (the scale
// is NaN) and the factor is 0, which keeps them finite or NaN, never garbage.
__device__ __forceinline__ float mx_factor(int e) {
    return e > 253 ? 0.0f : __uint_as_float((unsigned)(254 - e) << 23);
}

// e4m3 codes, four to a dword, as the sum of two: those of 2 and more, and the
// rest (bit 6 of a code, its exponent's highest, tells).  Code for code one of the
// two is 0; NaN is among the large.
//
// Of eight consecutive products the matrix instruction with an 8-bit operand keeps
// 14 binades: multiples of 2^-13 of the largest sum of exponents among them
// (measured; with two e2m1 operands that is all).  e4m3 times e2m1 has multiples of
// 2^-10 up to exponents of 10, so that sums of whole rows hold fewer bits than fp32,
// and a hidden value next to a tie then gets the other code.  The large codes'
// products are multiples of 2^-3, exponents up to 10, and the others' of 2^-10,
// exponents up to 2: two instructions keep every bit of both, and their sums are
// fp32's.  As bf16 (16 x 16 x 32) the products take the matrix pipes as long, and the
// conversions longer (one token's experts 18.0 us, this way 16.3).
struct MxParts {
    unsigned large, small;
};
__device__ __forceinline__ MxParts mx_parts(unsigned q) {
    // a selector of 13 and more makes a byte of ones; 0 takes byte 0 of the zeros
    const unsigned ones = __builtin_amdgcn_perm(0u, 0u, q & 0x40404040u);
    return {q & ones, q & ~ones};
}
__device__ __forceinline__ void mx_parts8(u32x4 p, u32x4 q, i32x8 &large, i32x8 &small) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const MxParts a = mx_parts(p[i]), b = mx_parts(q[i]);
        large[i] = (int)a.large;
        small[i] = (int)a.small;
        large[4 + i] = (int)b.large;
        small[4 + i] = (int)b.small;
    }
}

// Larger magnitude; NaN wins (as an unsigned number its bits exceed every
// other's), so that a block with a NaN gets the NaN scale.
__device__ __forceinline__ unsigned mx_abs_max(unsigned a, unsigned b) { return max(a, b); }
__device__ __forceinline__ unsigned mx_abs(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Eight scaled values -> eight codes: two dwords (e4m3) or one (e2m1, value
// i in nibble i).  Both conversions round to nearest, ties to even.
__device__ __forceinline__ uint2 mx_codes8_e4m3(const float (&v)[8], float f) {
    uint2 r;
    int a = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * f, v[1] * f, 0, false);
    r.x = (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(v[2] * f, v[3] * f, a, true);
    a = __builtin_amdgcn_cvt_pk_fp8_f32(v[4] * f, v[5] * f, 0, false);
    r.y = (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(v[6] * f, v[7] * f, a, true);
    return r;
}
__device__ __forceinline__ unsigned mx_codes8_e2m1(const float (&v)[8], float f) {
    unsigned r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0] * f, v[1] * f, 1.0f, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2] * f, v[3] * f, 1.0f, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4] * f, v[5] * f, 1.0f, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6] * f, v[7] * f, 1.0f, 3);
    return r;
}

// Four bf16 pairs -> eight fp32 values.
__device__ __forceinline__ void bf16x8_to_f32(u32x4 w, float (&v)[8]) {
    v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x);
    v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
    v[4] = bf16_lo(w.z); v[5] = bf16_hi(w.z);
    v[6] = bf16_lo(w.w); v[7] = bf16_hi(w.w);
}

__device__ __forceinline__ u32x4 f32x8_to_bf16(const float (&v)[8]) {
    u32x4 r;
    r.x = f32_to_bf16_rne(v[0]) | (unsigned)f32_to_bf16_rne(v[1]) << 16;
    r.y = f32_to_bf16_rne(v[2]) | (unsigned)f32_to_bf16_rne(v[3]) << 16;
    r.z = f32_to_bf16_rne(v[4]) | (unsigned)f32_to_bf16_rne(v[5]) << 16;
    r.w = f32_to_bf16_rne(v[6]) | (unsigned)f32_to_bf16_rne(v[7]) << 16;
    return r;
}

template <int CTRL>
__device__ __forceinline__ unsigned dpp_u32(unsigned v) {
    return (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
// Largest over the four lanes of a quad, in each of them.
__device__ __forceinline__ unsigned quad_max(unsigned v) {
    v = mx_abs_max(v, dpp_u32<kDppQuadSwap1>(v));
    return mx_abs_max(v, dpp_u32<kDppQuadSwap2>(v));
}

// silu(g) * u = g * u / (1 + exp(-g)) by the hardware's exp2 and reciprocal
// (1 ulp each): within (8 + 2 |g|) 2^-23 of the value, the |g| for the exponent's
// rounding, far inside the half step of the codes it becomes.  exp(-g) = inf gives
// -0 * u = 0.
__device__ __forceinline__ float swiglu(float g, float u) {
    return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504088896341f)) * u;
}

// A lane's eight values of a 32-block that its quad holds -> their codes at
// q + bytes of index i0, and the block's scale byte (returned in each lane).
template <int FMT>
__device__ __forceinline__ int mx_store8(const float (&v)[8], uint8_t *q, size_t i0) {
    unsigned m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = mx_abs_max(m, mx_abs(v[i]));
    const int e = mx_exponent<FMT>(__uint_as_float(quad_max(m)));
    const float f = mx_factor(e);
    if constexpr (FMT == kMxE4m3)
        *reinterpret_cast<uint2 *>(q + i0) = mx_codes8_e4m3(v, f);
    else
        *reinterpret_cast<unsigned *>(q + i0 / 2) = mx_codes8_e2m1(v, f);
    return e;
}

// Values [8i, 8i + 8) of bf16 rows of 8 * k8 values, quantised into rows of
// codes and scales q_stride and e_stride bytes apart; the scale bytes past the
// row's blocks become 0.  i runs over whole quads of lanes.
template <int FMT>
__device__ __forceinline__ void quant_padded8(const uint16_t *x, uint8_t *q, uint8_t *e8, unsigned i,
                                              unsigned k8, unsigned q_stride, unsigned e_stride) {
    float v[8];
    bf16x8_to_f32(*reinterpret_cast<const u32x4 *>(x + (size_t)i * 8), v);
    const unsigned row = i / k8, c = i - row * k8;
    const int e = mx_store8<FMT>(v, q + (size_t)row * q_stride, (size_t)c * 8);
    if ((i & 3u) != 0) return;
    uint8_t *er = e8 + (size_t)row * e_stride;
    er[c / 4] = (uint8_t)e;
    if (c / 4 == k8 / 4 - 1)
        for (unsigned z = k8 / 4; z < e_stride; ++z) er[z] = 0;
}

}  // namespace skg
