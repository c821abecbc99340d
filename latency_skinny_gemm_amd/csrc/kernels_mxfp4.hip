// kernels_mxfp4.hip -- products with MXFP4 weights on the scaled matrix
// instruction (v_mfma_scale_f32_16x16x128_f8f6f4): one weight for all rows, or
// the routed experts' weights for the rows sorted by expert.
#include "device_common.h"
#include "internal.h"
#include "lds_limit.h"
#include "moe_internal.h"
#include "mx_common.h"

namespace skg {

namespace {

enum { kDense = 0, kGateUp = 1, kDown = 2 };

struct TileArgs {
    const uint8_t *x;       // codes, K (or K / 2) bytes a row
    const uint8_t *xe;      // scale bytes, mx_scale_stride(K) a row
    unsigned x_rows;        // rows of x
    const uint8_t *W;       // packed
    const uint16_t *bias;   // dense
    uint8_t *out;           // dense: out; gate-up: h codes; down: y fp32 [pair][N]
    uint8_t *out_e;         // gate-up: h's scale rows
    int out_f32;
    int M, N, K;            // N: output columns (gate-up: I; W holds 2I)
    const MoeTile *tiles;   // grouped
    const int *count;       // grouped: tiles in use
    const int *pairs;       // grouped: sorted row -> pair
    int top;                // grouped: pairs per token
    int col_tiles;          // workgroups side by side in a row tile
    int row_tiles;          // dense
};

__device__ __forceinline__ float silu(float g) { return g / (1.0f + expf(-g)); }

// Larger of two over lanes l, l ^ 16, l ^ 32, l ^ 48 (the four lanes that
// hold one output row).
__device__ __forceinline__ unsigned row_max(unsigned v) {
    const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max(a[0], a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return max(b[0], b[1]);
}

// Workgroup b's place in the work list of n: the workgroups of one XCD (b % 8)
// take one contiguous run of it, so that neighbours in the list, which share
// weights, share that XCD's L2.  -1: nothing left.
__device__ __forceinline__ int xcd_order(int b, int n) {
    const int per = (n + 7) / 8, at = (b & 7) * per + (b >> 3);
    return (b >> 3) < per && at < n ? at : -1;
}

}  // namespace

// Scale bytes of a stage: 16 a row, in whole KB (a load fills one).
constexpr int tile_scale_bytes(int MT) { return MT * 256 < 1024 ? 1024 : MT * 256; }

// The key that piece c of row r is stored under: the rows that share a
// 256-byte window of the banks get different ones.
template <int CPR>
__device__ __forceinline__ int piece_key(int r) {
    return (r / (16 / CPR)) & (CPR - 1);
}

// A workgroup of four waves computes MT * 16 rows x (4 waves * NBW * 16)
// columns over the whole K.  Stages of 256 K: the rows' codes and scale bytes
// go to LDS by direct loads (two stages), each wave's weights to registers,
// both one stage ahead of the products.  A 16-byte piece c of row r sits at
// c ^ piece_key(r), so that the 16 rows of a fragment read hit all banks once.
template <int MT, int NBW, int FX, int MODE>
__global__ void __launch_bounds__(256) mxfp4_tile_kernel(TileArgs a) {
    constexpr int RB = FX == kMxE4m3 ? 256 : 128;  // bytes of a row and stage
    constexpr int CPR = RB / 16;                   // pieces of a row and stage
    constexpr int ROWS = MT * 16;
    constexpr int XS = ROWS * RB;                  // codes of a stage
    constexpr int STAGE = XS + tile_scale_bytes(MT);  // and 16 scale bytes a row
    constexpr int XI = XS / 1024 / 4 > 0 ? XS / 1024 / 4 : 1;  // loads per wave
    constexpr int XW = XS / 1024 < 4 ? XS / 1024 : 4;          // waves that load codes
    extern __shared__ __attribute__((aligned(16))) unsigned char lds_raw[];

    const int t = threadIdx.x, lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int row_tiles = MODE == kDense ? a.row_tiles : a.count[0];
    const int at = xcd_order(blockIdx.x, a.col_tiles * row_tiles);
    if (at < 0) return;
    const int ct = at / row_tiles, rt = at - ct * row_tiles;  // column tile, row tile
    int row0 = rt * ROWS, rows = min(ROWS, a.M - row0), expert = 0;
    if constexpr (MODE != kDense) {
        const MoeTile tile = a.tiles[rt];
        row0 = tile.row;
        rows = tile.rows;
        expert = tile.expert;
    }
    const int live = (rows + 15) / 16;  // row blocks that hold rows
    const int KS = mxfp4_steps(a.K), nst = (KS + 1) / 2;
    const size_t gb = mxfp4_group_bytes(a.K);
    const unsigned rowb = FX == kMxE4m3 ? (unsigned)a.K : (unsigned)a.K / 2;
    const unsigned es = (unsigned)mx_scale_stride(a.K);

    // this wave's column groups
    const int ng = mxfp4_groups(MODE == kGateUp ? 2 * a.N : a.N);
    const uint8_t *We = a.W + (size_t)expert * ng * gb;
    Rsrc wr[NBW], sr[NBW];
#pragma unroll
    for (int b = 0; b < NBW; ++b) {
        int j;
        bool in;
        if constexpr (MODE == kGateUp) {
            const int c = (ct * 4 + wave) * (NBW / 2) + b % (NBW / 2);
            in = c * 16 < a.N;
            j = c + (b < NBW / 2 ? 0 : a.N / 16);
        } else {
            j = (ct * 4 + wave) * NBW + b;
            in = j < ng;
        }
        wr[b] = make_rsrc(We + (in ? j * gb : 0), in ? (unsigned)KS * 1024u : 0u);
        sr[b] = make_rsrc(We + (in ? j * gb : 0) + (size_t)KS * 1024,
                          in ? (unsigned)mxfp4_chunks(a.K) * 256u : 0u);
    }

    // this lane's pieces of the rows
    const Rsrc xr = make_rsrc(a.x, a.x_rows * rowb);
    const Rsrc er = make_rsrc(a.xe, a.x_rows * es);
    auto row_of = [&](int r) -> int {  // x row of tile row r < rows
        if constexpr (MODE == kGateUp) return a.pairs[row0 + r] / a.top;
        else return row0 + r;
    };
    unsigned xoff[XI];
    unsigned xcol[XI];
#pragma unroll
    for (int i = 0; i < XI; ++i) {
        const int lin = ((wave * XI + i) * 64 + lane);
        const int r = lin / CPR, c = (lin % CPR) ^ piece_key<CPR>(r);
        xcol[i] = (unsigned)c * 16u;
        xoff[i] = r < rows && wave < XW ? (unsigned)row_of(r) * rowb + xcol[i] : kOOB;
    }
    const int erow = wave * 64 + lane;
    const unsigned eoff = erow < rows ? (unsigned)row_of(erow) * es : kOOB;

    auto issue_x = [&](int slot, int st) {
        unsigned char *base = lds_raw + slot * STAGE;
        if (wave < XW)
#pragma unroll
            for (int i = 0; i < XI; ++i) {
                const unsigned k = (unsigned)st * RB;
                lds_load16<kCacheDefault>(xr, base + (wave * XI + i) * 1024,
                                          k + xcol[i] < rowb ? xoff[i] + k : kOOB);
            }
        if (wave * 64 < ROWS)
            lds_load16<kCacheDefault>(er, base + XS + wave * 1024,
                                      eoff == kOOB ? kOOB : eoff + (unsigned)(st / 2) * 16u);
    };
    u32x4 w[2][2][NBW];  // [buffer][step][group]
    unsigned ws[2][NBW];
    auto issue_w = [&](int buf, int st) {
#pragma unroll
        for (int b = 0; b < NBW; ++b) {
#pragma unroll
            for (int s = 0; s < 2; ++s)
                w[buf][s][b] = load16<kCacheDefault>(wr[b], (unsigned)(2 * st + s) * 1024u + lane * 16u);
            ws[buf][b] = __builtin_amdgcn_raw_buffer_load_b32(
                sr[b], (unsigned)(st / 2) * 256u + lane * 4u, 0, kCacheDefault);
        }
    };

    f32x4 acc[MT][NBW];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int b = 0; b < NBW; ++b) acc[m][b] = f32x4{0.f, 0.f, 0.f, 0.f};

    const int fr = lane & 15, fg = lane >> 4;
    auto compute = [&](int slot, int buf, int st) {
        const unsigned char *base = lds_raw + slot * STAGE;
        int wsc[NBW];
#pragma unroll
        for (int b = 0; b < NBW; ++b) wsc[b] = (int)(ws[buf][b] >> (16 * (st & 1)));
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            if (m >= live) break;
            const unsigned char *rp = base + (m * 16 + fr) * RB;
            const uint2 ev = *reinterpret_cast<const uint2 *>(base + XS + (m * 16 + fr) * 16 +
                                                              8 * (st & 1));
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                i32x8 xf{0, 0, 0, 0, 0, 0, 0, 0};
                if constexpr (FX == kMxE4m3) {
                    const u32x4 p0 = *reinterpret_cast<const u32x4 *>(rp + (((8 * s + fg) ^ piece_key<CPR>(fr)) * 16));
                    const u32x4 p1 = *reinterpret_cast<const u32x4 *>(rp + (((8 * s + 4 + fg) ^ piece_key<CPR>(fr)) * 16));
                    xf = i32x8{(int)p0.x, (int)p0.y, (int)p0.z, (int)p0.w,
                               (int)p1.x, (int)p1.y, (int)p1.z, (int)p1.w};
                } else {
                    const u32x4 p0 = *reinterpret_cast<const u32x4 *>(rp + (((4 * s + fg) ^ piece_key<CPR>(fr)) * 16));
                    xf = i32x8{(int)p0.x, (int)p0.y, (int)p0.z, (int)p0.w, 0, 0, 0, 0};
                }
                const int xsc = (int)((s ? ev.y : ev.x) >> (8 * fg));
#pragma unroll
                for (int b = 0; b < NBW; ++b) {
                    const u32x4 q = w[buf][s][b];
                    const i32x8 wf{(int)q.x, (int)q.y, (int)q.z, (int)q.w, 0, 0, 0, 0};
                    if (s == 0)
                        acc[m][b] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            wf, xf, acc[m][b], kMxE2m1, FX, 0, wsc[b], 0, xsc);
                    else
                        acc[m][b] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            wf, xf, acc[m][b], kMxE2m1, FX, 1, wsc[b], 0, xsc);
                }
            }
        }
    };

    issue_x(0, 0);
    issue_w(0, 0);
    for (int st = 0; st < nst; st += 2) {
        // nst is the same for every wave: every wave reaches every barrier
        wait_vmcnt_lds<0>();
        barrier_nofence();
        if (st + 1 < nst) {
            issue_x(1, st + 1);
            issue_w(1, st + 1);
        }
        compute(0, 0, st);
        if (st + 1 >= nst) break;
        wait_vmcnt_lds<0>();
        barrier_nofence();
        if (st + 2 < nst) {
            issue_x(0, st + 2);
            issue_w(0, st + 2);
        }
        compute(1, 1, st + 1);
    }

    // lane (fr, fg) holds, of row m * 16 + fr, columns 4 fg + 0..3 of each group
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int r = m * 16 + fr;
        if constexpr (MODE == kGateUp) {
            static_assert(MODE != kGateUp || NBW == 4, "a wave holds one 32-block of h");
            if (m >= live) break;  // uniform: the exchange below needs the whole wave
            const int c0 = (ct * 4 + wave) * 32;
            float h[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                h[i] = silu(acc[m][i / 4][i % 4]) * acc[m][2 + i / 4][i % 4];
            unsigned big = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) big = mx_abs_max(big, mx_abs(h[i]));
            const int e = mx_exponent<FX>(__uint_as_float(row_max(big)));
            if (r >= rows || c0 >= a.N) continue;
            const size_t o = (size_t)(row0 + r) * a.N + c0 + 4 * fg;
            if constexpr (FX == kMxE4m3) {
                const uint2 q = mx_codes8_e4m3(h, mx_factor(e));
                *reinterpret_cast<unsigned *>(a.out + o) = q.x;
                *reinterpret_cast<unsigned *>(a.out + o + 16) = q.y;
            } else {
                const unsigned q = mx_codes8_e2m1(h, mx_factor(e));
                *reinterpret_cast<uint16_t *>(a.out + o / 2) = (uint16_t)q;
                *reinterpret_cast<uint16_t *>(a.out + o / 2 + 8) = (uint16_t)(q >> 16);
            }
            if (fg == 0) {
                const unsigned hs = (unsigned)mx_scale_stride(a.N);
                uint8_t *er_ = a.out_e + (size_t)(row0 + r) * hs;
                er_[c0 / 32] = (uint8_t)e;
                if (c0 + 32 == a.N)  // the last block also clears the row's padding
                    for (unsigned z = a.N / 32; z < hs; ++z) er_[z] = 0;
            }
        } else {
            if (r >= rows) continue;
            size_t orow = (size_t)(row0 + r);
            if constexpr (MODE == kDown) orow = (size_t)a.pairs[row0 + r];
#pragma unroll
            for (int b = 0; b < NBW; ++b) {
                const int n0 = ((ct * 4 + wave) * NBW + b) * 16 + 4 * fg;
                f32x4 v = acc[m][b];
                if constexpr (MODE == kDense) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (n0 + i >= a.N) break;
                        if (a.bias) v[i] += bf16_to_f32(a.bias[n0 + i]);
                        store_out(a.out, orow * a.N + n0 + i, v[i], a.out_f32);
                    }
                } else {
                    if (n0 < a.N)  // N % 32 == 0
                        *reinterpret_cast<f32x4 *>(a.out + (orow * a.N + n0) * 4) = v;
                }
            }
        }
    }
}

namespace {

template <int MT, int NBW, int FX, int MODE>
int go(TileArgs a, int tiles, hipStream_t stream) {
    constexpr size_t bytes = 2 * (MT * 16 * (FX == kMxE4m3 ? 256 : 128) + tile_scale_bytes(MT));
    static std::atomic<unsigned long long> lds_set{0};
    const hipError_t e = allow_dynamic_lds(
        reinterpret_cast<const void *>(&mxfp4_tile_kernel<MT, NBW, FX, MODE>), bytes, lds_set);
    if (e != hipSuccess) return (int)e;
    const int cols = MODE == kGateUp ? 128 : 64 * NBW;
    a.col_tiles = (a.N + cols - 1) / cols;
    a.row_tiles = tiles;
    hipLaunchKernelGGL((mxfp4_tile_kernel<MT, NBW, FX, MODE>),
                       dim3(((unsigned)a.col_tiles * (unsigned)tiles + 7) / 8 * 8), dim3(256), bytes, stream, a);
    return (int)hipGetLastError();
}

template <int NBW, int MODE>
int pick(const TileArgs &a, int fmt, int rows, int tiles, hipStream_t stream) {
    if (fmt == kMxE4m3) {
        if (rows <= 16) return go<1, NBW, kMxE4m3, MODE>(a, tiles, stream);
        if (rows <= 32) return go<2, NBW, kMxE4m3, MODE>(a, tiles, stream);
        if (rows <= 64) return go<4, NBW, kMxE4m3, MODE>(a, tiles, stream);
        return go<8, NBW, kMxE4m3, MODE>(a, tiles, stream);
    }
    if (rows <= 16) return go<1, NBW, kMxE2m1, MODE>(a, tiles, stream);
    if (rows <= 32) return go<2, NBW, kMxE2m1, MODE>(a, tiles, stream);
    if (rows <= 64) return go<4, NBW, kMxE2m1, MODE>(a, tiles, stream);
    return go<8, NBW, kMxE2m1, MODE>(a, tiles, stream);
}

}  // namespace

int launch_mxfp4(const Mxfp4Args &p, hipStream_t stream) {
    TileArgs a{};
    a.x = p.x;
    a.xe = p.xe;
    a.x_rows = (unsigned)p.M;
    a.W = p.W;
    a.bias = p.bias;
    a.out = (uint8_t *)p.out;
    a.out_f32 = p.out_f32;
    a.M = p.M;
    a.N = p.N;
    a.K = p.K;
    const int rows = p.M <= 16 ? 16 : p.M <= 32 ? 32 : p.M <= 64 ? 64 : 128;
    return pick<1, kDense>(a, p.fmt, rows, (p.M + rows - 1) / rows, stream);
}

// The two products of the routed experts (kernels_moe.hip sorts and combines).
int launch_moe_gate_up(const MoeArgs &m, const MoeLists &s, const uint8_t *xq, const uint8_t *xe,
                       uint8_t *h, uint8_t *he, int rows, int tiles, hipStream_t stream) {
    TileArgs a{};
    a.x = xq;
    a.xe = xe;
    a.x_rows = (unsigned)m.T;
    a.W = m.W13;
    a.out = h;
    a.out_e = he;
    a.N = m.I;
    a.K = m.H;
    a.tiles = s.tiles;
    a.count = s.count;
    a.pairs = s.pairs;
    a.top = m.k;
    return pick<4, kGateUp>(a, m.fmt, rows, tiles, stream);
}

int launch_moe_down(const MoeArgs &m, const MoeLists &s, const uint8_t *h, const uint8_t *he,
                    float *y, int rows, int tiles, hipStream_t stream) {
    TileArgs a{};
    a.x = h;
    a.xe = he;
    a.x_rows = (unsigned)(m.T * m.k);
    a.W = m.W2;
    a.out = (uint8_t *)y;
    a.N = m.H;
    a.K = m.I;
    a.tiles = s.tiles;
    a.count = s.count;
    a.pairs = s.pairs;
    a.top = m.k;
    return pick<2, kDown>(a, m.fmt, rows, tiles, stream);
}

}  // namespace skg
