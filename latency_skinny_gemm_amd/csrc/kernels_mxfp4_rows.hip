// kernels_mxfp4_rows.hip -- MXFP4 products of few rows: the waves of a
// workgroup share a few column groups and split K.
//
// At few rows a product is the weight's stream and the latency around it.
// So a workgroup owns R groups of 16 columns over the whole K, its NW waves
// take the 128-wide steps w, w + NW, ..., each wave has the loads of U steps in
// flight at once, and the only exchange is one sum over the waves through LDS
// at the end, in wave order: no second launch, no partials in memory, the same
// bits every time.  The rows are brought to LDS by the workgroup, bf16 ones
// quantised on the way, while the weights are in flight: that saves the launch
// that would do it.  More rows go in blocks to more workgroups, while there are
// CUs without one: what a workgroup waits for grows with its rows.
//
// Measured, weights from memory, bf16 rows to e4m3 (e2m1): one row of 7168 by 2112
// columns 5.1 us (4.4; 8.0 MB of weights, 1.6 TB/s: a launch and one load after
// another make most of it, and in e4m3 the rows' two parts), 16 rows 9.8 (7.6; the
// rows' quantising), 16 rows by 576 columns 5.3 (4.5), in four blocks.  Experts of
// 2880 x 2880, one token's four, in e4m3: 10.2 us gate and up (35 MB, 3.4 TB/s) and
// 7.2 down (18 MB, 2.5).  Fragments loaded straight to registers, without LDS, took
// 1.7 times as long for the one row; the parts of several steps taken before the
// weights arrive 7 % longer for the token, for the registers.
#include "device_common.h"
#include "internal.h"
#include "lds_limit.h"
#include "moe_internal.h"
#include "mx_common.h"

namespace skg {

namespace {

typedef short i16x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ unsigned pk_max(unsigned a, unsigned b) {
    return __builtin_bit_cast(unsigned, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                  __builtin_bit_cast(u16x2, b)));
}
// Magnitude bits of the largest of 8 bf16 values (two 16-bit candidates).
__device__ __forceinline__ unsigned amax8(u32x4 v) {
    constexpr unsigned A = 0x7FFF7FFFu;
    return pk_max(pk_max(v.x & A, v.y & A), pk_max(v.z & A, v.w & A));
}
__device__ __forceinline__ unsigned fold16(unsigned v) { return max(v & 0xFFFFu, v >> 16); }

// mx_exponent of a bf16 magnitude's 16 bits: the carry of the addition is the
// comparison with 1.75 (e4m3) or 1.5 (e2m1).
template <int FMT>
__device__ __forceinline__ int mx_exponent16(unsigned a) {
    const int e = FMT == kMxE4m3 ? (int)((a + 31u) >> 7) - 8 : (int)((a + 63u) >> 7) - 2;
    return a == 0 ? 127 : (a >= 0x7F80u ? 255 : max(e, 0));
}
// The conversions below divide by the scale's exponent field alone: the bits
// e << 23 mean 2^(e - 127) for every e, 0 included (checked code by code).
__device__ __forceinline__ float scale_of(int e) { return __uint_as_float((unsigned)e << 23); }

// 8 bf16 values -> 8 e4m3 codes (two dwords) or 8 e2m1 codes (one).  Pairs
// are taken from the 8-element view with shufflevector: bit-casting the 32-bit
// lanes one by one is folded onto the first by this compiler.
__device__ __forceinline__ uint2 codes8_e4m3(u32x4 v, float s) {
    const bf16x8 b = __builtin_bit_cast(bf16x8, v);
    i16x2 lo{0, 0}, hi{0, 0};
    lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(lo, __builtin_shufflevector(b, b, 0, 1), s, false);
    lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(lo, __builtin_shufflevector(b, b, 2, 3), s, true);
    hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(hi, __builtin_shufflevector(b, b, 4, 5), s, false);
    hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(hi, __builtin_shufflevector(b, b, 6, 7), s, true);
    return uint2{__builtin_bit_cast(unsigned, lo), __builtin_bit_cast(unsigned, hi)};
}
__device__ __forceinline__ unsigned codes8_e2m1(u32x4 v, float s) {
    const bf16x8 b = __builtin_bit_cast(bf16x8, v);
    unsigned r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_shufflevector(b, b, 0, 1), s, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_shufflevector(b, b, 2, 3), s, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_shufflevector(b, b, 4, 5), s, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_shufflevector(b, b, 6, 7), s, 3);
    return r;
}

enum { kRowsDense = 0, kRowsGateUp = 1, kRowsDown = 2 };

// A value that is the same in the whole wave and that nothing here writes.  By
// the scalar unit: a vector load in front of the weights' would be waited for
// with everything older, loads return in order.
template <typename T>
__device__ __forceinline__ T scalar_load(const T *p) {
    return *(const __attribute__((address_space(4))) T *)(uintptr_t)p;
}

struct RowArgs {
    const uint8_t *x;        // bf16 rows, or codes
    unsigned xs;             // bytes from row to row
    const uint8_t *xe;       // codes: scale bytes, es a row
    unsigned es;
    const uint8_t *W;
    const uint16_t *bias;
    uint8_t *out, *out_e;
    int out_f32;
    int M, N, K;             // gate-up: N = I, W holds 2I rows
    const int *ids;          // experts
    const float *weights;
    int top, E;
    int blocks, block_rows;  // dense: blocks of rows, and rows of all but the last
    // set by go(): waves' loads per row of codes (or bf16) and of scale bytes,
    // and what divides by them and by the steps of K
    int row_loads, scale_loads;
    unsigned by_row_loads, by_scale_loads, by_steps;
};

// n / d by a multiplication, for n * d < 2^31: a division takes some 20 vector
// instructions, and what a wave does before its first load is latency.
constexpr unsigned divider(unsigned d) { return (0x80000000u + d - 1) / d; }
__device__ __forceinline__ int divide(int n, unsigned by) {
    return (int)(((unsigned long long)(unsigned)n * by) >> 31);
}

}  // namespace

// Dense: workgroup j owns column groups j * R ..; MT blocks of 16 rows.
// Gate-up (R = 4, one row): workgroup (pair, 32 columns of h).
// Down (one row a unit): workgroup (token, R groups); the units are the steps
// of all the token's choices.
// XB: 16-byte pieces of the rows that a thread has in flight.
template <int MODE, int MT, int R, int FX, bool BF16, int NW, int U, int XB>
__global__ void __launch_bounds__(NW * 64) mxfp4_rows_kernel(RowArgs a) {
    constexpr bool ONE = MODE != kRowsDense;  // one row: only lanes of row 0 hold data
    constexpr int ROWS = ONE ? 1 : MT * 16;
    __shared__ float part[NW][ROWS][R * 16];
    extern __shared__ __attribute__((aligned(16))) uint8_t row_lds[];  // the rows' codes, then their scales
    const int t = threadIdx.x, lane = t & 63, fr = lane & 15, fg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int KS = mxfp4_steps(a.K);
    const size_t gb = mxfp4_group_bytes(a.K);
    const int ng = mxfp4_groups(MODE == kRowsGateUp ? 2 * a.N : a.N);

    int j0, row = 0, units = KS;  // first group, (pair or token), steps to share
    if constexpr (MODE == kRowsDense) {
        // the blocks of a column group side by side on one XCD (workgroup b runs on
        // XCD b % 8): they read the same weights
        const int i = blockIdx.x >> 3, g = i / a.blocks;
        j0 = (g * 8 + (int)(blockIdx.x & 7)) * R;
        row = (i - g * a.blocks) * a.block_rows;
        if (j0 >= ng || row >= a.M) return;
    } else if constexpr (MODE == kRowsGateUp) {
        const int cols = a.N / 32;
        row = blockIdx.x / cols;
        j0 = (blockIdx.x - row * cols) * 2;
    } else {
        const int cols = (ng + R - 1) / R;
        row = blockIdx.x / cols;
        j0 = (blockIdx.x - row * cols) * R;
        units = KS * a.top;
    }
    auto group_of = [&](int b) -> int {
        if constexpr (MODE == kRowsGateUp) return j0 + (b & 1) + (b < 2 ? 0 : a.N / 16);
        else return min(j0 + b, ng - 1);  // a group past the end is computed twice, stored once
    };
    const uint8_t *We = a.W;
    if constexpr (MODE == kRowsGateUp) {
        const int e = a.ids[row];
        if ((unsigned)e >= (unsigned)a.E) return;
        We += (size_t)e * ng * gb;
    }

    const unsigned rowb = BF16 ? (unsigned)a.K * 2u : FX == kMxE4m3 ? (unsigned)a.K : (unsigned)a.K / 2;
    const unsigned kb = (unsigned)a.K / 32;
    f32x4 acc[MT][R];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int b = 0; b < R; ++b) acc[m][b] = f32x4{0.f, 0.f, 0.f, 0.f};

    // the rows: a view that ends with the last one
    const size_t x0 = MODE == kRowsGateUp ? (size_t)(row / a.top) : MODE == kRowsDown ? (size_t)row * a.top : (size_t)row;
    const unsigned xrows = MODE == kRowsGateUp ? 1u : MODE == kRowsDown ? (unsigned)a.top : (unsigned)min(a.block_rows, a.M - row);
    const Rsrc xr = make_rsrc(a.x + x0 * a.xs, (xrows - 1) * a.xs + rowb);
    const Rsrc er = make_rsrc(BF16 ? nullptr : a.xe + x0 * a.es, BF16 ? 0u : xrows * a.es);
    constexpr unsigned CB = FX == kMxE4m3 ? 128u : 64u;  // bytes of a row's codes in a step

    // The rows go to LDS once, as codes in whole steps (zeros past K) and their
    // scale bytes: straight to registers they would be fragments of 16 rows,
    // and a lane that is out of range costs what one with data does.  A wave's
    // load is 64 pieces of one row: 8 bf16 values (a block is a quad of lanes)
    // or 16 bytes of codes each; or 64 scale bytes.
    const int xp = KS * (BF16 ? 16 : (int)CB / 16);  // pieces of a row
    const int rs = KS * (int)CB + kRowLdsPad;
    const int xn = (int)xrows * a.row_loads, sn = BF16 ? 0 : (int)xrows * a.scale_loads;
    uint8_t *const row_sc = row_lds + (size_t)xrows * rs;
    u32x4 xv[XB];
    uint8_t sv[XB];
    auto load_rows = [&](int v0) {
#pragma unroll
        for (int v = 0; v < XB; ++v) {
            const int q = wave + (v0 + v) * NW;
            if (q < xn) {
                const int r = divide(q, a.by_row_loads), c = (q - r * a.row_loads) * 64 + lane;
                xv[v] = load16<kCacheDefault>(xr, (unsigned)c * 16u < rowb ? (unsigned)r * a.xs + (unsigned)c * 16u : kOOB);
            }
            if (q < sn) {
                const int r = divide(q, a.by_scale_loads), c = (q - r * a.scale_loads) * 64 + lane;
                sv[v] = __builtin_amdgcn_raw_buffer_load_b8(
                    er, (unsigned)c < kb ? (unsigned)r * a.es + (unsigned)c : kOOB, 0, kCacheDefault);
            }
        }
    };
    auto store_rows = [&](int v0) {
#pragma unroll
        for (int v = 0; v < XB; ++v) {
            const int q = wave + (v0 + v) * NW;
            if (q < xn) {
                const int r = divide(q, a.by_row_loads), c = (q - r * a.row_loads) * 64 + lane;
                if constexpr (BF16) {
                    const int e = mx_exponent16<FX>(quad_max(fold16(amax8(xv[v]))));
                    if (c < xp) {
                        if constexpr (FX == kMxE4m3)
                            *reinterpret_cast<uint2 *>(row_lds + r * rs + c * 8) = codes8_e4m3(xv[v], scale_of(e));
                        else
                            *reinterpret_cast<unsigned *>(row_lds + r * rs + c * 4) = codes8_e2m1(xv[v], scale_of(e));
                        if ((c & 3) == 0) row_sc[r * (KS * 4) + c / 4] = (uint8_t)e;
                    }
                } else {
                    if (c < xp) *reinterpret_cast<u32x4 *>(row_lds + r * rs + c * 16) = xv[v];
                }
            }
            if (q < sn) {
                const int r = divide(q, a.by_scale_loads), c = (q - r * a.scale_loads) * 64 + lane;
                if (c < KS * 4) row_sc[r * (KS * 4) + c] = sv[v];
            }
        }
    };
    load_rows(0);  // before the weights: loads return in order

    const int batches = (units + NW * U - 1) / (NW * U);  // the same for every wave
    for (int it = 0; it < batches; ++it) {
        const int u0 = it * NW * U + wave;
        u32x4 w[U][R];
        unsigned ws[U][R];
        float wt[U];
        int expert[U];  // down: of the unit's choice; -1: none that is held here
        if constexpr (MODE == kRowsDown) {
            int id[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const size_t p = (size_t)row * a.top + divide(min(u0 + i * NW, units - 1), a.by_steps);
                id[i] = scalar_load(a.ids + p);
                wt[i] = scalar_load(a.weights + p);
            }
            // all together: one by one each would be waited for
            static_assert(MODE != kRowsDown || U == 6, "the operands below");
            asm volatile("" : "+s"(id[0]), "+s"(id[1]), "+s"(id[2]), "+s"(id[3]), "+s"(id[4]), "+s"(id[5]),
                              "+s"(wt[0]), "+s"(wt[1]), "+s"(wt[2]), "+s"(wt[3]), "+s"(wt[4]), "+s"(wt[5]));
#pragma unroll
            for (int i = 0; i < U; ++i) {
                expert[i] = u0 + i * NW < units && (unsigned)id[i] < (unsigned)a.E ? id[i] : -1;
                if (expert[i] < 0) wt[i] = 0.0f;  // whatever stands there, infinite or NaN too
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int u = u0 + i * NW;
            int s = u < units ? u : -1;
            const uint8_t *Wu = We;
            if constexpr (MODE == kRowsDown) {
                s = expert[i] >= 0 ? u - divide(u, a.by_steps) * KS : -1;
                Wu += (size_t)max(expert[i], 0) * ng * gb;
            }
            // s < 0: nothing (loads past the views' ends return 0)
            const unsigned so = s < 0 ? kOOB : (unsigned)s;
            // A dense product reads its weights once (2112 x 7168 from memory:
            // 7.3 -> 6.9 us); pairs may share an expert's (16 pairs, 64 experts:
            // 33 us, 35 past the caches).
            constexpr int CACHE = MODE == kRowsDense ? kCacheStream : kCacheDefault;
#pragma unroll
            for (int b = 0; b < R; ++b) {
                const uint8_t *g = Wu + (size_t)group_of(b) * gb;
                const Rsrc wr = make_rsrc(g, (unsigned)gb);
                w[i][b] = load16<CACHE>(wr, s < 0 ? kOOB : so * 1024u + lane * 16u);
                ws[i][b] = __builtin_amdgcn_raw_buffer_load_b32(
                    wr, s < 0 ? kOOB : (unsigned)KS * 1024u + so / 4u * 256u + lane * 4u, 0, kCacheDefault);
            }
        }
        // every load of the batch goes out before the first product; steps past
        // the end hold zeros, which add nothing
        __builtin_amdgcn_sched_barrier(0);
        if (it == 0) {  // while the weights are on their way
            store_rows(0);
            for (int v0 = XB; v0 * NW < max(xn, sn); v0 += XB) {
                load_rows(v0);
                store_rows(v0);
            }
            wait_vmcnt_lds<63>();  // the writes to LDS alone
            barrier_nofence();
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int u = u0 + i * NW;
            const int j = MODE == kRowsDown ? divide(min(u, units - 1), a.by_steps) : 0;
            const int s = u - j * KS, sl = min(s, KS - 1);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                // lanes past the last row hold it again; their columns of the
                // result are not used
                const int rl = MODE == kRowsDown ? j : min(m * 16 + fr, (int)xrows - 1);
                const uint8_t *rp = row_lds + rl * rs + sl * CB + fg * 16;
                const u32x4 p = *reinterpret_cast<const u32x4 *>(rp);
                const u32x4 x1 = *reinterpret_cast<const u32x4 *>(rp + (FX == kMxE4m3 ? 64 : 0));
                i32x8 xq{(int)p.x, (int)p.y, (int)p.z, (int)p.w, 0, 0, 0, 0}, xs;
                if constexpr (FX == kMxE4m3) mx_parts8(p, x1, xq, xs);
                const int xe = row_sc[rl * (KS * 4) + sl * 4 + fg];
                // fp32 sums of e4m3 in two instructions (mx_parts)
                auto multiply = [&](const i32x8 &wf, int sc, f32x4 d) {
                    if constexpr (FX == kMxE4m3)
                        d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf, xs, d, kMxE2m1, FX, 0, sc, 0, xe);
                    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf, xq, d, kMxE2m1, FX, 0, sc, 0, xe);
                };
#pragma unroll
                for (int b = 0; b < R; ++b) {
                    const u32x4 q = w[i][b];
                    const i32x8 wf{(int)q.x, (int)q.y, (int)q.z, (int)q.w, 0, 0, 0, 0};
                    const int sc = (int)(ws[i][b] >> (8 * (s & 3)));
                    if constexpr (MODE == kRowsDown) {
                        const f32x4 d = multiply(wf, sc, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                        for (int c = 0; c < 4; ++c) acc[m][b][c] = __builtin_fmaf(wt[i], expert[i] >= 0 ? d[c] : 0.0f, acc[m][b][c]);
                    } else {
                        acc[m][b] = multiply(wf, sc, acc[m][b]);
                    }
                }
            }
        }
    }

    // lane (fr, fg): row m * 16 + fr, columns 4 fg + 0..3 of each group
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int b = 0; b < R; ++b)
            if (!ONE || fr == 0)
                *reinterpret_cast<f32x4 *>(&part[wave][ONE ? 0 : m * 16 + fr][b * 16 + fg * 4]) = acc[m][b];
    __syncthreads();
    auto sum = [&](int r, int c) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w) v += part[w][r][c];
        return v;
    };

    if constexpr (MODE == kRowsGateUp) {
        if (t >= 64) return;
        // lane c < 32: column c of the 32-block (both halves of the wave alike)
        const int c = t & 31;
        const float h = swiglu(sum(0, c), sum(0, 32 + c));
        unsigned m = mx_abs(h);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) m = mx_abs_max(m, (unsigned)__shfl_xor((int)m, d, 64));
        const int e = mx_exponent<FX>(__uint_as_float(m));
        const float hf = h * mx_factor(e);
        if (FX == kMxE4m3) {
            if (t < 32)
                a.out[(size_t)row * mx_code_stride(FX, a.N) + j0 * 16 + c] = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(hf, hf, 0, false);
        } else {
            const float next = __shfl_xor(hf, 1, 64);
            if (t < 32 && (c & 1) == 0)
                a.out[(size_t)row * mx_code_stride(FX, a.N) + (j0 * 16 + c) / 2] =
                    (uint8_t)__builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, hf, next, 1.0f, 0);
        }
        if (t == 0) a.out_e[(size_t)row * mx_scale_stride(a.N) + j0 / 2] = (uint8_t)e;
    } else {
        for (int i = t; i < ROWS * R * 16; i += NW * 64) {
            const int r = i / (R * 16), c = i % (R * 16), n = j0 * 16 + c;
            if (n >= a.N || (!ONE && r >= (int)xrows)) continue;
            float v = sum(r, c);
            if (MODE == kRowsDense && a.bias) v += bf16_to_f32(a.bias[n]);
            store_out(a.out, (size_t)(ONE ? row : row + r) * a.N + n, v, a.out_f32);
        }
    }
}

namespace {

template <int MODE, int MT, int R, int FX, bool BF16, int NW, int U, int XB>
int go(RowArgs a, size_t grid, hipStream_t stream) {
    const int rows = MODE == kRowsGateUp ? 1 : MODE == kRowsDown ? a.top : a.block_rows;
    const size_t lds = rows * mxfp4_row_lds_bytes(FX, a.K);
    const int KS = mxfp4_steps(a.K);
    a.row_loads = (KS * (BF16 ? 16 : FX == kMxE4m3 ? 8 : 4) + 63) / 64;
    a.scale_loads = (KS * 4 + 63) / 64;
    a.by_row_loads = divider((unsigned)a.row_loads);
    a.by_scale_loads = divider((unsigned)a.scale_loads);
    a.by_steps = divider((unsigned)KS);
    static std::atomic<unsigned long long> lds_set{0};
    const hipError_t e = allow_dynamic_lds(
        reinterpret_cast<const void *>(&mxfp4_rows_kernel<MODE, MT, R, FX, BF16, NW, U, XB>),
        kMxRowMaxLds, lds_set);
    if (e != hipSuccess) return (int)e;
    hipLaunchKernelGGL((mxfp4_rows_kernel<MODE, MT, R, FX, BF16, NW, U, XB>), dim3((unsigned)grid),
                       dim3(NW * 64), lds, stream, a);
    return (int)hipGetLastError();
}

// Waves that share the steps: enough that a wave has at most U of them, up to 16.
inline int waves_of(int units, int U) { return units <= 4 * U ? 4 : units <= 8 * U ? 8 : 16; }

template <int MODE, int MT, int R, int FX, bool BF16, int U, int XB>
int waves(const RowArgs &a, int nw, size_t grid, hipStream_t stream) {
    if (nw == 4) return go<MODE, MT, R, FX, BF16, 4, U, XB>(a, grid, stream);
    if (nw == 8) return go<MODE, MT, R, FX, BF16, 8, U, XB>(a, grid, stream);
    return go<MODE, MT, R, FX, BF16, 16, U, XB>(a, grid, stream);
}

// XB as many as a wave has loads of rows, up to 4: what is not needed costs its
// instructions before the weights' loads (one row of 7168: 4.1 us with one,
// 4.3 with four, 4.8 with eight), and a second round waits for the weights (four
// rows: 5.5, 4.8).
template <int FX, bool BF16>
int dense16(const RowArgs &a, int KS, size_t grid, hipStream_t stream) {
    const int nw = waves_of(KS, 4), pieces = KS * (BF16 ? 16 : FX == kMxE4m3 ? 8 : 4);
    const int loads = a.block_rows * ((max(pieces, BF16 ? 0 : KS * 4) + 63) / 64);
    if (loads <= nw) return waves<kRowsDense, 1, 1, FX, BF16, 4, 1>(a, nw, grid, stream);
    if (loads <= 2 * nw) return waves<kRowsDense, 1, 1, FX, BF16, 4, 2>(a, nw, grid, stream);
    return waves<kRowsDense, 1, 1, FX, BF16, 4, 4>(a, nw, grid, stream);
}

template <int FX>
int dense(const RowArgs &a, bool bf16, hipStream_t stream) {
    const size_t grid = (size_t)((mxfp4_groups(a.N) + 7) / 8 * 8) * a.blocks;
    const int KS = mxfp4_steps(a.K);
    if (bf16) return dense16<FX, true>(a, KS, grid, stream);
    if (a.block_rows <= 16) return dense16<FX, false>(a, KS, grid, stream);
    return waves<kRowsDense, 2, 1, FX, false, 4, 4>(a, waves_of(KS, 4), grid, stream);
}

}  // namespace

int launch_mxfp4_rows(const Mxfp4Args &p, int blocks, hipStream_t stream) {
    RowArgs a{};
    a.x = p.x;
    a.xs = (unsigned)(p.xe ? p.xs : p.K * 2);
    a.xe = p.xe;
    a.es = (unsigned)p.es;
    a.W = p.W;
    a.bias = p.bias;
    a.out = (uint8_t *)p.out;
    a.out_f32 = p.out_f32;
    a.M = p.M;
    a.N = p.N;
    a.K = p.K;
    a.blocks = blocks;
    a.block_rows = (p.M + blocks - 1) / blocks;
    return p.fmt == kMxE4m3 ? dense<kMxE4m3>(a, p.xe == nullptr, stream)
                            : dense<kMxE2m1>(a, p.xe == nullptr, stream);
}

namespace {
template <int FX>
int moe_rows(const MoeArgs &m, uint8_t *h, uint8_t *he, hipStream_t stream) {
    RowArgs a{};
    a.x = (const uint8_t *)m.x;
    a.xs = (unsigned)m.H * 2;
    a.W = m.W13;
    a.out = h;
    a.out_e = he;
    a.N = m.I;
    a.K = m.H;
    a.ids = m.ids;
    a.weights = m.weights;
    a.top = m.k;
    a.E = m.E;
    int e = go<kRowsGateUp, 1, 4, FX, true, 8, 3, 1>(a, (size_t)m.T * m.k * (m.I / 32), stream);
    if (e != (int)hipSuccess) return e;
    a.x = h;
    a.xs = (unsigned)mx_code_stride(m.fmt, m.I);
    a.xe = he;
    a.es = (unsigned)mx_scale_stride(m.I);
    a.W = m.W2;
    a.out = (uint8_t *)m.out;
    a.out_f32 = 0;
    a.N = m.H;
    a.K = m.I;
    return waves<kRowsDown, 1, 1, FX, false, 6, 1>(a, waves_of(m.k * mxfp4_steps(m.I), 6),
                                                   (size_t)m.T * mxfp4_groups(m.H), stream);
}
}  // namespace

int launch_moe_rows(const MoeArgs &m, uint8_t *h, uint8_t *he, hipStream_t stream) {
    return m.fmt == kMxE4m3 ? moe_rows<kMxE4m3>(m, h, he, stream)
                            : moe_rows<kMxE2m1>(m, h, he, stream);
}

}  // namespace skg
