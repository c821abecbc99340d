// kernels_mx.hip -- MX quantisation of bf16 rows to e4m3 or e2m1 codes with
// one e8m0 byte per 32 values, the way back, and the layout the MXFP4
// products read their weights in.
//
// All three are single passes bound by HBM: 4096 x 7168 to e2m1 takes 15 us
// (74 MB, 4.9 TB/s) and back 14 us (5.4), where a copy on this card moves 4.7;
// 64 x 2880 takes 2.2 us, a launch and one trip to memory; the layout of 128 x 2880 x
// 2880 226 us (1.13 GB, 5.0).  The pieces are 16
// bytes a thread and independent, so there is nothing to share or stage.
#include "device_common.h"
#include "internal.h"
#include "moe_internal.h"
#include "mx_common.h"

namespace skg {

// Thread i quantises values [8i, 8i + 8): one 16-byte load, one store of 8
// (e4m3) or 4 (e2m1) bytes, and the block's byte from one lane of the quad
// that holds the block.  PAD: rows of codes and scales are q_stride and
// e_stride bytes apart (the products' workspace) and the scale bytes past
// K / 32 are written as 0.
template <int FMT, bool PAD>
__global__ void __launch_bounds__(256)
    quant_mx_kernel(const uint16_t *__restrict__ x, uint8_t *__restrict__ q,
                    uint8_t *__restrict__ e8, unsigned n8, unsigned k8, unsigned q_stride,
                    unsigned e_stride) {
    const unsigned i = blockIdx.x * 256u + threadIdx.x;
    if (i >= n8) return;  // n8 is a multiple of 4: whole quads leave
    if constexpr (PAD) {
        quant_padded8<FMT>(x, q, e8, i, k8, q_stride, e_stride);
    } else {
        float v[8];
        bf16x8_to_f32(*reinterpret_cast<const u32x4 *>(x + (size_t)i * 8), v);
        const int e = mx_store8<FMT>(v, q, (size_t)i * 8);
        if ((i & 3u) == 0) e8[i / 4] = (uint8_t)e;
    }
}

// Thread i turns codes [8i, 8i + 8) into bf16 values.  Every code times its
// scale is a bf16 number unless the scale takes it out of bf16's range.
template <int FMT>
__global__ void __launch_bounds__(256)
    dequant_mx_kernel(const uint8_t *__restrict__ q, const uint8_t *__restrict__ e8,
                      uint16_t *__restrict__ out, unsigned n8) {
    const unsigned i = blockIdx.x * 256u + threadIdx.x;
    if (i >= n8) return;
    const int e = e8[i / 4];
    float v[8];
    if constexpr (FMT == kMxE4m3) {
        const uint2 w = *reinterpret_cast<const uint2 *>(q + (size_t)i * 8);
        const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w.x, false);
        const auto b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w.x, true);
        const auto c = __builtin_amdgcn_cvt_pk_f32_fp8((int)w.y, false);
        const auto d = __builtin_amdgcn_cvt_pk_f32_fp8((int)w.y, true);
        v[0] = a[0]; v[1] = a[1]; v[2] = b[0]; v[3] = b[1];
        v[4] = c[0]; v[5] = c[1]; v[6] = d[0]; v[7] = d[1];
    } else {
        const unsigned w = *reinterpret_cast<const unsigned *>(q + (size_t)i * 4);
        const auto a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
        const auto b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
        const auto c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
        const auto d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
        v[0] = a[0]; v[1] = a[1]; v[2] = b[0]; v[3] = b[1];
        v[4] = c[0]; v[5] = c[1]; v[6] = d[0]; v[7] = d[1];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = e == 255 ? __uint_as_float(0x7FC00000u) : ldexpf(v[j], e - 127);
    *reinterpret_cast<u32x4 *>(out + (size_t)i * 8) = f32x8_to_bf16(v);
}

// Caller's scale rows [M][kb] -> the products' padded rows [M][e_stride].
__global__ void __launch_bounds__(256)
    pad_scales_kernel(const uint8_t *__restrict__ e8, uint8_t *__restrict__ out, unsigned n,
                      unsigned kb, unsigned e_stride) {
    const unsigned i = blockIdx.x * 256u + threadIdx.x;
    if (i >= n) return;
    const unsigned row = i / e_stride, b = i - row * e_stride;
    out[i] = b < kb ? e8[(size_t)row * kb + b] : (uint8_t)0;
}

// Row-major MXFP4 weights -> column groups of 16 rows of W in the order the
// matrix instruction takes them, so that a wave reads a group as one
// contiguous stream: KS steps of 1 KB (lane l = 16g + r: the 32 codes of row
// r, K block g of the step), then KC dwords per lane, byte s of dword c the
// scale of block g of step 4c + s.  Rows past N and blocks past K take codes
// 0 (and scale 127), so they add exactly 0.
// One workgroup: one group of one expert (blockIdx.y).
__global__ void __launch_bounds__(256)
    mxfp4_pack_kernel(const uint8_t *__restrict__ q, const uint8_t *__restrict__ e8,
                      uint8_t *__restrict__ out, int N, int K) {
    const int KS = mxfp4_steps(K), KC = mxfp4_chunks(K), KB = K / 32;
    const int j = blockIdx.x;
    const size_t ex = blockIdx.y;
    uint8_t *dst = out + (ex * gridDim.x + j) * mxfp4_group_bytes(K);
    for (int i = threadIdx.x; i < KS * 64; i += 256) {
        const int l = i & 63, row = j * 16 + (l & 15), blk = (i >> 6) * 4 + (l >> 4);
        u32x4 v{0, 0, 0, 0};
        if (row < N && blk < KB)
            v = *reinterpret_cast<const u32x4 *>(q + ((ex * N + row) * (size_t)KB + blk) * 16);
        *reinterpret_cast<u32x4 *>(dst + (size_t)i * 16) = v;
    }
    for (int i = threadIdx.x; i < KC * 64; i += 256) {
        const int l = i & 63, row = j * 16 + (l & 15);
        unsigned v = 0;
        for (int s = 0; s < 4; ++s) {
            const int blk = ((i >> 6) * 4 + s) * 4 + (l >> 4);
            const unsigned b = row < N && blk < KB ? e8[(ex * N + row) * (size_t)KB + blk] : 127u;
            v |= b << (8 * s);
        }
        *reinterpret_cast<unsigned *>(dst + (size_t)KS * 1024 + (size_t)i * 4) = v;
    }
}

namespace {
unsigned blocks_of(size_t n) { return (unsigned)((n + 255) / 256); }
}  // namespace

int launch_quant_mx(const void *x, void *q, void *e8, int fmt, int M, int K, bool padded,
                    hipStream_t stream) {
    const unsigned n8 = (unsigned)((size_t)M * K / 8), k8 = (unsigned)K / 8;
    const unsigned qs = (unsigned)mx_code_stride(fmt, K), es = (unsigned)mx_scale_stride(K);
    auto *const f = fmt == kMxE4m3 ? (padded ? quant_mx_kernel<kMxE4m3, true> : quant_mx_kernel<kMxE4m3, false>)
                                   : (padded ? quant_mx_kernel<kMxE2m1, true> : quant_mx_kernel<kMxE2m1, false>);
    hipLaunchKernelGGL(f, dim3(blocks_of(n8)), dim3(256), 0, stream, (const uint16_t *)x,
                       (uint8_t *)q, (uint8_t *)e8, n8, k8, qs, es);
    return (int)hipGetLastError();
}

int launch_dequant_mx(const void *q, const void *e8, int fmt, void *out, int M, int K,
                      hipStream_t stream) {
    const unsigned n8 = (unsigned)((size_t)M * K / 8);
    const dim3 grid(blocks_of(n8)), block(256);
    if (fmt == kMxE4m3)
        hipLaunchKernelGGL((dequant_mx_kernel<kMxE4m3>), grid, block, 0, stream, (const uint8_t *)q,
                           (const uint8_t *)e8, (uint16_t *)out, n8);
    else
        hipLaunchKernelGGL((dequant_mx_kernel<kMxE2m1>), grid, block, 0, stream, (const uint8_t *)q,
                           (const uint8_t *)e8, (uint16_t *)out, n8);
    return (int)hipGetLastError();
}

int launch_pad_scales(const void *e8, void *out, int M, int K, hipStream_t stream) {
    const unsigned stride = (unsigned)mx_scale_stride(K);
    const unsigned n = (unsigned)M * stride;
    hipLaunchKernelGGL(pad_scales_kernel, dim3(blocks_of(n)), dim3(256), 0, stream,
                       (const uint8_t *)e8, (uint8_t *)out, n, (unsigned)K / 32, stride);
    return (int)hipGetLastError();
}

int launch_mxfp4_pack(const void *q, const void *e8, void *out, int E, int N, int K,
                      hipStream_t stream) {
    hipLaunchKernelGGL(mxfp4_pack_kernel, dim3((unsigned)mxfp4_groups(N), (unsigned)E), dim3(256),
                       0, stream, (const uint8_t *)q, (const uint8_t *)e8, (uint8_t *)out, N, K);
    return (int)hipGetLastError();
}

}  // namespace skg
