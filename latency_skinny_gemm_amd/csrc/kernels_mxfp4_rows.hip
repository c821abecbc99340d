// kernels_mxfp4_rows.hip -- MXFP4 products of few rows: the waves of a
// workgroup share a few column groups and split K.
//
// At few rows a product is the weight's stream and the latency around it.
// So a workgroup owns R groups of 16 columns over the whole K, its NW waves
// take the 128-wide steps w, w + NW, ..., each wave has the loads of U steps in
// flight at once, and the only exchange is one sum over the waves through LDS
// at the end, in wave order: no second launch, no partials in memory, the same
// bits every time.  bf16 rows are quantised in the registers that feed the
// matrix instruction (mx_quant_*: about 60 instructions a step, hidden under
// the weights' latency), which saves the launch that would do it.
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

// One step of one row block as the matrix instruction takes it: the codes a
// lane holds and the scale byte of its 32-block.
struct Frag {
    i32x8 q;
    int e;
};

// What a lane loads of bf16 rows for one step: 32 values.
//   e2m1: K 32g .. 32g + 31, block g itself;
//   e4m3: K 16g .. 16g + 15 and 64 + 16g .., halves of blocks g / 2 and
//         2 + g / 2 (v[0..1] and v[2..3]).
template <int FX>
__device__ __forceinline__ Frag quantise_frag(const u32x4 (&v)[4], int fg) {
    Frag f;
    if constexpr (FX == kMxE2m1) {
        const unsigned a = fold16(pk_max(pk_max(amax8(v[0]), amax8(v[1])), pk_max(amax8(v[2]), amax8(v[3]))));
        f.e = mx_exponent16<FX>(a);
        const float s = scale_of(f.e);
        f.q = i32x8{(int)codes8_e2m1(v[0], s), (int)codes8_e2m1(v[1], s), (int)codes8_e2m1(v[2], s),
                    (int)codes8_e2m1(v[3], s), 0, 0, 0, 0};
    } else {
        // both halves' candidates in one register, then the other half of
        // each block from lane l ^ 16
        const unsigned lo = fold16(pk_max(amax8(v[0]), amax8(v[1])));
        const unsigned hi = fold16(pk_max(amax8(v[2]), amax8(v[3])));
        unsigned a = lo | hi << 16;
        const auto x = __builtin_amdgcn_permlane16_swap(a, a, false, false);
        a = pk_max(x[0], x[1]);
        const int e0 = mx_exponent16<FX>(a & 0xFFFFu), e1 = mx_exponent16<FX>(a >> 16);
        const float s0 = scale_of(e0), s1 = scale_of(e1);
        const uint2 c0 = codes8_e4m3(v[0], s0), c1 = codes8_e4m3(v[1], s0);
        const uint2 c2 = codes8_e4m3(v[2], s1), c3 = codes8_e4m3(v[3], s1);
        f.q = i32x8{(int)c0.x, (int)c0.y, (int)c1.x, (int)c1.y, (int)c2.x, (int)c2.y, (int)c3.x, (int)c3.y};
        // lane group g supplies block g's byte: 0 and 3 have it, 1 and 2 take
        // it from lane l ^ 32 (groups 3 and 0)
        const unsigned both = (unsigned)e0 | (unsigned)e1 << 16;
        const auto y = __builtin_amdgcn_permlane32_swap(both, both, false, false);
        const unsigned other = fg < 2 ? y[1] : y[0];
        f.e = fg == 0 ? e0 : fg == 3 ? e1 : fg == 1 ? (int)(other & 0xFFFFu) : (int)(other >> 16);
    }
    return f;
}

// Byte offset of the i-th 16-byte piece of a lane's 32 bf16 values in a step.
template <int FX>
__device__ __forceinline__ unsigned bf16_piece(int fg, int i) {
    return FX == kMxE2m1 ? (unsigned)(fg * 64 + i * 16)
                         : (unsigned)((i >> 1) * 128 + fg * 32 + (i & 1) * 16);
}

enum { kRowsDense = 0, kRowsGateUp = 1, kRowsDown = 2 };

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
};

}  // namespace

// Dense: workgroup j owns column groups j * R ..; MT blocks of 16 rows.
// Gate-up (R = 4, one row): workgroup (pair, 32 columns of h).
// Down (one row a unit): workgroup (token, R groups); the units are the steps
// of all the token's choices.
template <int MODE, int MT, int R, int FX, bool BF16, int NW, int U>
__global__ void __launch_bounds__(NW * 64) mxfp4_rows_kernel(RowArgs a) {
    constexpr bool ONE = MODE != kRowsDense;  // one row: only lanes of row 0 hold data
    constexpr int ROWS = ONE ? 1 : MT * 16;
    __shared__ float part[NW][ROWS][R * 16];
    extern __shared__ __attribute__((aligned(16))) uint8_t row_lds[];  // gate-up: the row's codes and scales
    const int t = threadIdx.x, lane = t & 63, fr = lane & 15, fg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int KS = mxfp4_steps(a.K);
    const size_t gb = mxfp4_group_bytes(a.K);
    const int ng = mxfp4_groups(MODE == kRowsGateUp ? 2 * a.N : a.N);

    int j0, row = 0, units = KS;  // first group, (pair or token), steps to share
    if constexpr (MODE == kRowsDense) {
        j0 = blockIdx.x * R;
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
    const size_t x0 = MODE == kRowsGateUp ? (size_t)(row / a.top) : MODE == kRowsDown ? (size_t)row * a.top : 0;
    const unsigned xrows = MODE == kRowsGateUp ? 1u : MODE == kRowsDown ? (unsigned)a.top : (unsigned)a.M;
    const Rsrc xr = make_rsrc(a.x + x0 * a.xs, (xrows - 1) * a.xs + rowb);
    const Rsrc er = make_rsrc(BF16 ? nullptr : a.xe + x0 * a.es, BF16 ? 0u : xrows * a.es);
    constexpr bool LDS_ROW = MODE == kRowsGateUp;
    constexpr int XV = BF16 ? 4 : FX == kMxE4m3 ? 2 : 1;  // 16-byte pieces of a lane and step
    constexpr int XM = LDS_ROW ? 0 : MT;                  // blocks whose rows come straight to registers
    constexpr unsigned CB = FX == kMxE4m3 ? 128u : 64u;   // bytes of a row's codes in a step

    const int batches = (units + NW * U - 1) / (NW * U);  // the same for every wave
    for (int it = 0; it < batches; ++it) {
        const int u0 = it * NW * U + wave;
        u32x4 w[U][R], x[U][XM > 0 ? XM : 1][XV];
        unsigned ws[U][R], xs[U][XM > 0 ? XM : 1];
        float wt[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int u = u0 + i * NW;
            const bool live = u < units;
            int s = u, j = 0;
            const uint8_t *Wu = We;
            if constexpr (MODE == kRowsDown) {
                j = u / KS;
                s = u - j * KS;
                const size_t p = (size_t)row * a.top + (live ? j : 0);
                const int e = a.ids[p];
                const bool in = live && (unsigned)e < (unsigned)a.E;
                wt[i] = in ? a.weights[p] : 0.0f;
                Wu += in ? (size_t)e * ng * gb : 0;
                if (!in) s = -1;
            } else {
                if (!live) s = -1;
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
#pragma unroll
            for (int m = 0; m < XM; ++m) {
                const int r = ONE ? j : m * 16 + fr;
                const bool has = s >= 0 && (ONE ? fr == 0 : r < a.M);
                const unsigned stepb = BF16 ? 256u : CB;
#pragma unroll
                for (int v = 0; v < XV; ++v) {
                    const unsigned in = so * stepb + (BF16 ? bf16_piece<FX>(fg, v)
                                                           : (unsigned)(v * 64 + fg * 16));
                    x[i][m][v] = load16<kCacheDefault>(xr, has && in < rowb ? (unsigned)r * a.xs + in : kOOB);
                }
                if constexpr (!BF16) {
                    const unsigned blk = so * 4u + fg;
                    xs[i][m] = __builtin_amdgcn_raw_buffer_load_b8(
                        er, has && blk < kb ? (unsigned)r * a.es + blk : kOOB, 0, kCacheDefault);
                }
            }
        }
        // every load of the batch goes out before the first product; steps past
        // the end hold zeros, which add nothing
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (LDS_ROW) {
            // The one row, quantised once by the workgroup while the weights
            // are on their way: 8 values a thread, a block per quad; codes to
            // the end of the last step (zeros past K), then the scale bytes.
            if (it == 0) {
                uint8_t *const rs = row_lds + (size_t)KS * CB;
                for (int i = t; i < KS * 16; i += NW * 64) {
                    const u32x4 v = load16<kCacheDefault>(xr, (unsigned)i * 16u < rowb ? (unsigned)i * 16u : kOOB);
                    const unsigned am = quad_max(fold16(amax8(v)));
                    const int e = mx_exponent16<FX>(am);
                    if constexpr (FX == kMxE4m3)
                        *reinterpret_cast<uint2 *>(row_lds + i * 8) = codes8_e4m3(v, scale_of(e));
                    else
                        *reinterpret_cast<unsigned *>(row_lds + i * 4) = codes8_e2m1(v, scale_of(e));
                    if ((i & 3) == 0) rs[i / 4] = (uint8_t)e;
                }
                __syncthreads();
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int u = u0 + i * NW;
            const int s = MODE == kRowsDown ? u % KS : u;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                Frag f;
                if constexpr (LDS_ROW) {
                    // every lane row holds the one row; only column 0 of the
                    // result is used
                    const int sl = min(s, KS - 1);
                    const uint8_t *rp = row_lds + sl * CB + fg * 16;
                    const u32x4 p = *reinterpret_cast<const u32x4 *>(rp);
                    const u32x4 q = *reinterpret_cast<const u32x4 *>(rp + (FX == kMxE4m3 ? 64 : 0));
                    f.q = FX == kMxE4m3 ? i32x8{(int)p.x, (int)p.y, (int)p.z, (int)p.w, (int)q.x, (int)q.y, (int)q.z, (int)q.w}
                                        : i32x8{(int)p.x, (int)p.y, (int)p.z, (int)p.w, 0, 0, 0, 0};
                    f.e = row_lds[(size_t)KS * CB + sl * 4 + fg];
                } else if constexpr (BF16) {
                    f = quantise_frag<FX>(x[i][m], fg);
                } else {
                    const u32x4 p = x[i][m][0], q = x[i][m][XV - 1];
                    f.q = XV == 2 ? i32x8{(int)p.x, (int)p.y, (int)p.z, (int)p.w, (int)q.x, (int)q.y, (int)q.z, (int)q.w}
                                  : i32x8{(int)p.x, (int)p.y, (int)p.z, (int)p.w, 0, 0, 0, 0};
                    f.e = (int)xs[i][m];
                }
#pragma unroll
                for (int b = 0; b < R; ++b) {
                    const u32x4 q = w[i][b];
                    const i32x8 wf{(int)q.x, (int)q.y, (int)q.z, (int)q.w, 0, 0, 0, 0};
                    const int sc = (int)(ws[i][b] >> (8 * (s & 3)));
                    if constexpr (MODE == kRowsDown) {
                        const f32x4 d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            wf, f.q, f32x4{0.f, 0.f, 0.f, 0.f}, kMxE2m1, FX, 0, sc, 0, f.e);
#pragma unroll
                        for (int c = 0; c < 4; ++c) acc[m][b][c] = __builtin_fmaf(wt[i], d[c], acc[m][b][c]);
                    } else {
                        acc[m][b] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            wf, f.q, acc[m][b], kMxE2m1, FX, 0, sc, 0, f.e);
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
            if (n >= a.N || (!ONE && r >= a.M)) continue;
            float v = sum(r, c);
            if (MODE == kRowsDense && a.bias) v += bf16_to_f32(a.bias[n]);
            store_out(a.out, (size_t)(ONE ? row : r) * a.N + n, v, a.out_f32);
        }
    }
}

namespace {

template <int MODE, int MT, int R, int FX, bool BF16, int NW, int U>
int go(const RowArgs &a, size_t grid, hipStream_t stream) {
    size_t lds = 0;
    if (MODE == kRowsGateUp) {
        lds = mxfp4_row_lds_bytes(FX, a.K);
        static std::atomic<unsigned long long> lds_set{0};
        const hipError_t e = allow_dynamic_lds(
            reinterpret_cast<const void *>(&mxfp4_rows_kernel<MODE, MT, R, FX, BF16, NW, U>),
            kMxRowMaxLds, lds_set);
        if (e != hipSuccess) return (int)e;
    }
    hipLaunchKernelGGL((mxfp4_rows_kernel<MODE, MT, R, FX, BF16, NW, U>), dim3((unsigned)grid),
                       dim3(NW * 64), lds, stream, a);
    return (int)hipGetLastError();
}

// Waves that share the steps: enough that a wave has at most U of them, up to 16.
template <int MODE, int MT, int R, int FX, bool BF16, int U>
int waves(const RowArgs &a, int units, size_t grid, hipStream_t stream) {
    if (units <= 4 * U) return go<MODE, MT, R, FX, BF16, 4, U>(a, grid, stream);
    if (units <= 8 * U) return go<MODE, MT, R, FX, BF16, 8, U>(a, grid, stream);
    return go<MODE, MT, R, FX, BF16, 16, U>(a, grid, stream);
}

template <int FX>
int dense(const RowArgs &a, bool bf16, hipStream_t stream) {
    const size_t grid = (size_t)mxfp4_groups(a.N);
    const int KS = mxfp4_steps(a.K);
    if (bf16) return waves<kRowsDense, 1, 1, FX, true, 4>(a, KS, grid, stream);
    if (a.M <= 16) return waves<kRowsDense, 1, 1, FX, false, 4>(a, KS, grid, stream);
    return waves<kRowsDense, 2, 1, FX, false, 4>(a, KS, grid, stream);
}

}  // namespace

int launch_mxfp4_rows(const Mxfp4Args &p, hipStream_t stream) {
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
    int e = go<kRowsGateUp, 1, 4, FX, true, 8, 3>(a, (size_t)m.T * m.k * (m.I / 32), stream);
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
    return waves<kRowsDown, 1, 1, FX, false, 6>(a, m.k * mxfp4_steps(m.I),
                                                (size_t)m.T * mxfp4_groups(m.H), stream);
}
}  // namespace

int launch_moe_rows(const MoeArgs &m, uint8_t *h, uint8_t *he, hipStream_t stream) {
    return m.fmt == kMxE4m3 ? moe_rows<kMxE4m3>(m, h, he, stream)
                            : moe_rows<kMxE2m1>(m, h, he, stream);
}

}  // namespace skg
