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
    const uint8_t *x;       // codes, x_stride bytes from row to row
    unsigned x_stride;
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
    int tall;               // grouped: as MoeLists
    int col_tiles;          // workgroups side by side in a row tile
    int row_tiles;          // dense
};

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
// operands, share that XCD's L2.  -1: nothing left.
__device__ __forceinline__ int xcd_order(int b, int n) {
    const int per = (n + 7) / 8, at = (b & 7) * per + (b >> 3);
    return (b >> 3) < per && at < n ? at : -1;
}

}  // namespace

// The key that piece c of row r is stored under.  Measured on fragment reads of
// 64- and 128-byte rows: r / 2 leaves no bank conflict in either, r / 4 or none
// costs 4 clocks a read in the shorter, none 12 in the longer.
template <int CPR>
__device__ __forceinline__ int piece_key(int r) {
    return (r / 2) & (CPR - 1);
}

// Chunks of K (512 each) whose row scales a tile keeps in LDS at a time: whole
// rounds of a ring of SL steps, up to 16.
__host__ __device__ constexpr int tile_scale_most(int SL) { return 16 / (SL / 4) * (SL / 4); }
// ... when n remain.
__host__ __device__ constexpr int tile_scale_chunks(int n, int SL) {
    return n >= tile_scale_most(SL) ? tile_scale_most(SL) : (n + SL / 4 - 1) / (SL / 4) * (SL / 4);
}
// Pieces of 16 bytes from row to row there: an odd number, or the 16 rows of a
// read meet in the banks (4 clocks a read at 14 pieces, 28 at 16).
__host__ __device__ constexpr int tile_scale_pieces(int chunks) { return chunks | 1; }
constexpr int tile_slot_bytes(int MT, int FX) { return MT * (FX == kMxE4m3 ? 2048 : 1024); }
// Chunks of weight scales in LDS: those of the steps in flight and one more,
// as a power of two.
constexpr int tile_wchunks(int SL) { return SL == 4 ? 2 : 4; }
constexpr int tile_wscale_bytes(int NBW, int SL) { return tile_wchunks(SL) * 4 * NBW * 256; }
// chunks: as tile_scale_chunks.  Scale loads fill whole KB.
constexpr size_t tile_lds_bytes(int MT, int NBW, int FX, int SL, int chunks) {
    return (size_t)SL * tile_slot_bytes(MT, FX) + 1024 + tile_wscale_bytes(NBW, SL) +
           ((size_t)MT * 256 * tile_scale_pieces(chunks) + 1023) / 1024 * 1024;
}

// A workgroup of four waves computes MT * 16 rows x (4 waves * NBW * 16)
// columns over the whole K, in steps of 128: the rows' codes go to a ring of SL
// LDS slots by direct loads, each wave's weights to registers (they are used by
// that wave alone, and packed so that a load is 1 KB in a row), both about SL
// steps ahead of the products.  One wait and one barrier a step; the wait
// leaves all younger steps' loads in flight.  The rows' scale bytes are loaded
// once for 8192 K.  A 16-byte piece c of row r sits at c ^ piece_key(r), so that
// the 16 rows of a fragment read hit all banks once.
//
// What bounds it.  Experts, 40 tokens (64 of 4096 x 1408, 8 a token, half of them
// held, e2m1): HBM; 54 us for the 332 MB of gate and up, 6.1 TB/s, 27 us for the
// 172 MB of down.  2048 tokens (128 of 2880 x 2880, 4 a token, e4m3): 346 us and
// 192 us; 3.3 and 2.8 TB/s of weights, the matrix pipes half busy with two
// instructions a product, and the vector instructions that take the rows apart
// issued between them.  Dense, 512 x 4096 x 7168: in e2m1 19 us, 17 bytes a clock
// into each CU; in e4m3 36 us, with the parts.
//
// AHEAD > 0 takes that many steps a barrier and reads their fragments from LDS
// under the products of the steps before.  That pays where a SIMD holds one
// wave (e2m1, 512 x 4096 x 7168: 24.9 -> 21.3 us) and loses, for the registers
// it takes, where it holds two or more (experts: by 15 %).
//
// CACHE: what the weights' loads ask of the caches.
template <int MT, int NBW, int FX, int MODE, int SL, int AHEAD, int CACHE>
__device__ __forceinline__ void mxfp4_tile(const TileArgs &a, const MoeTile &own, const int ct,
                                           const int rt) {
    constexpr int RB = FX == kMxE4m3 ? 128 : 64;   // bytes of a row and step
    constexpr int CPR = RB / 16;                   // pieces of a row and step
    constexpr int ROWS = MT * 16;
    constexpr int SLOT = tile_slot_bytes(MT, FX);
    constexpr int XI = SLOT / 1024;                // loads of a step
    constexpr int XPW = (XI + 3) / 4;              // of a wave; the spare ones fill a KB of their own
    constexpr int LOADS = XPW + NBW;               // a step's loads of a wave, at least
    constexpr int WC = tile_wchunks(SL), SC = tile_scale_most(SL);
    extern __shared__ __attribute__((aligned(16))) unsigned char lds_raw[];
    unsigned char *const pad = lds_raw + SL * SLOT;
    unsigned char *const scales = pad + 1024 + tile_wscale_bytes(NBW, SL);

    const int t = threadIdx.x, lane = t & 63, fr = lane & 15, fg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int row0 = own.row + rt * ROWS, rows = min(ROWS, own.rows - rt * ROWS);
    const int KS = mxfp4_steps(a.K), KC = mxfp4_chunks(a.K);
    const int KP = (KS + SL - 1) / SL * SL;              // steps gone through, whole rounds of the ring
    const size_t gb = mxfp4_group_bytes(a.K);
    const unsigned rowb = FX == kMxE4m3 ? (unsigned)a.K : (unsigned)a.K / 2, xs = a.x_stride;
    const unsigned es = (unsigned)mx_scale_stride(a.K);

    // this wave's column groups; past the last, a view of nothing: its loads
    // return 0
    const int ng = mxfp4_groups(MODE == kGateUp ? 2 * a.N : a.N);
    const uint8_t *const We = a.W + (size_t)own.expert * ng * gb;
    Rsrc wr[NBW];
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
        wr[b] = make_rsrc(We + (in ? j * gb : 0), in ? (unsigned)gb : 0u);
    }

    u32x4 w[SL][NBW];
    // A chunk's dwords of scale bytes go to LDS with its first step: loaded
    // with every step they would be asked of the L1 again while on their way.
    unsigned char *const wscales = pad + 1024 + wave * (NBW * 256);  // chunks 4 waves apart
    auto issue_w = [&](int slot, int st, int chunk, int b) {
        if (slot % 4 == 0)
            lds_load4(wr[b], wscales + (chunk & (WC - 1)) * (4 * NBW * 256) + b * 256,
                      st < KS ? (unsigned)KS * 1024u + (unsigned)(st / 4) * 256u + lane * 4u : kOOB);
        w[slot][b] = load16<CACHE>(wr[b], st < KS ? (unsigned)st * 1024u + lane * 16u : kOOB);
    };
    // the weights' first round goes out before the rows are known
#pragma unroll
    for (int s = 0; s < SL; ++s)
#pragma unroll
        for (int b = 0; b < NBW; ++b) issue_w(s, s, s / 4, b);

    // this lane's pieces of the rows
    const Rsrc xr = make_rsrc(a.x, (a.x_rows - 1) * xs + rowb);
    const Rsrc er = make_rsrc(a.xe, a.x_rows * es);
    auto row_of = [&](int r) -> unsigned {  // x row of tile row r < rows
        if constexpr (MODE == kGateUp) return (unsigned)(a.pairs[row0 + r] / a.top);
        else return (unsigned)(row0 + r);
    };
    unsigned xoff[XPW], xcol[XPW];
#pragma unroll
    for (int i = 0; i < XPW; ++i) {
        const int q = wave + 4 * i, lin = q * 64 + lane;
        const int r = lin / CPR, c = (lin % CPR) ^ piece_key<CPR>(r);
        xcol[i] = (unsigned)c * 16u;
        xoff[i] = q < XI && r < rows ? row_of(r) * xs + xcol[i] : kOOB;
    }
    auto issue_x = [&](int slot, int st) {
        const unsigned k = (unsigned)st * RB;
#pragma unroll
        for (int i = 0; i < XPW; ++i) {
            const int q = wave + 4 * i;
            lds_load16<kCacheDefault>(xr, q < XI ? lds_raw + slot * SLOT + q * 1024 : pad,
                                      xoff[i] != kOOB && k + xcol[i] < rowb ? xoff[i] + k : kOOB);
        }
    };
    // the scale bytes of chunks c0 ..: piece q of row r is slot r * nc + q; the
    // chunks that only fill the ring's last round are zeros (the next row's
    // bytes in their place might be NaN scales)
    int sstride = 0;
    auto load_scales = [&](int c0) {
        const int nc = tile_scale_pieces(tile_scale_chunks(KC - c0, SL));
        sstride = nc * 16;
        for (int b = wave * 64; b < ROWS * nc; b += 256) {
            const int r = (b + lane) / nc, q = (b + lane) - r * nc;
            lds_load16<kCacheDefault>(er, scales + b * 16,
                                      r < rows && c0 + q < KC ? row_of(r) * es + (unsigned)(c0 + q) * 16u : kOOB);
        }
    };
    load_scales(0);
#pragma unroll
    for (int s = 0; s < (AHEAD ? SL : SL - 1); ++s) issue_x(s, s);
    int out_row[MT];  // down: the pair of each row that this lane stores
    if constexpr (MODE == kDown) {
#pragma unroll
        for (int m = 0; m < MT; ++m) out_row[m] = m * 16 + fr < rows ? a.pairs[row0 + m * 16 + fr] : 0;
    }

    f32x4 acc[MT][NBW];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int b = 0; b < NBW; ++b) acc[m][b] = f32x4{0.f, 0.f, 0.f, 0.f};
    // A step's fragments of x and the scale bytes.  AHEAD: read AHEAD steps
    // before their products, in two sets.
    constexpr int U = AHEAD ? AHEAD : 1;  // steps a barrier
    constexpr int FS = AHEAD ? 2 * U : 1;
    u32x4 xf[FS][MT][FX == kMxE4m3 ? 2 : 1];
    unsigned xsc[FS][MT], wsc[FS][NBW];
    // slot s; chunk: of the scale bytes in LDS; wchunk: of all chunks so far
    auto read_frags = [&](int f, int s, int chunk, int wchunk) {
        const unsigned char *base = lds_raw + s * SLOT;
#pragma unroll
        for (int b = 0; b < NBW; ++b)
            wsc[f][b] = *reinterpret_cast<const unsigned *>(wscales + (wchunk & (WC - 1)) * (4 * NBW * 256) + b * 256 + lane * 4);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int r = m * 16 + fr;
            const unsigned char *rp = base + r * RB;
            xsc[f][m] = *reinterpret_cast<const unsigned *>(scales + r * sstride + chunk * 16 + (s % 4) * 4);
            xf[f][m][0] = *reinterpret_cast<const u32x4 *>(rp + ((fg ^ piece_key<CPR>(fr)) * 16));
            if constexpr (FX == kMxE4m3)
                xf[f][m][1] = *reinterpret_cast<const u32x4 *>(rp + (((4 + fg) ^ piece_key<CPR>(fr)) * 16));
        }
    };
    auto multiply = [&](const i32x8 &x8, int f, int s, int m, int b) {
        const u32x4 v = w[s][b];
        const i32x8 w8{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
        const int sx = (int)(xsc[f][m] >> (8 * fg)), sw = (int)wsc[f][b];
        f32x4 &d = acc[m][b];
        if (s % 4 == 0) d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w8, x8, d, kMxE2m1, FX, 0, sw, 0, sx);
        if (s % 4 == 1) d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w8, x8, d, kMxE2m1, FX, 1, sw, 0, sx);
        if (s % 4 == 2) d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w8, x8, d, kMxE2m1, FX, 2, sw, 0, sx);
        if (s % 4 == 3) d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w8, x8, d, kMxE2m1, FX, 3, sw, 0, sx);
    };
    wait_vmcnt_lds<0>();  // the first steps were asked for together
    if constexpr (AHEAD) {
        barrier_nofence();
#pragma unroll
        for (int u = 0; u < U; ++u) read_frags(u, u, 0, 0);
    }
    for (int cb = 0;;) {
        const int nb = cb + SL;  // the loads of a round are the next one's
        // One round, straight: left early, it would carry loads that the
        // compiler then waits for at its head.  Steps past K are gone through
        // as zeros.
#pragma unroll
        for (int s0 = 0; s0 < SL; s0 += U) {
            // AHEAD: the next U steps' loads have landed, all but those of the
            // SL - 2U steps after them.  Else this step's: all but the weights
            // of SL - 1 steps and the rows of SL - 2.  The counts are the same
            // for every wave, so every wave reaches every barrier; behind it
            // every wave has read the slots that are loaded into here.
            wait_vmcnt_lds<AHEAD ? (SL - 2 * U) * LOADS : (SL - 1) * NBW + (SL - 2) * XPW>();
            barrier_nofence();
            if constexpr (AHEAD) {
#pragma unroll
                for (int s = s0; s < s0 + U; ++s) {
                    issue_x(s, nb + s);
                    const int n = cb + s + U;  // the step whose fragments are read
                    read_frags((s + U) % FS, (s + U) % SL, n / 4 % SC, n / 4);
                }
            } else {
                if (s0 == 0) issue_x(SL - 1, cb + SL - 1);
                else issue_x(s0 - 1, nb + s0 - 1);
            }
            // A group's products, then the loads into the registers they leave:
            // free to move, the loads would go first, into as many more.
#pragma unroll
            for (int s = s0; s < s0 + U; ++s) {
                if constexpr (!AHEAD) read_frags(0, s, (cb + s) / 4 % SC, (cb + s) / 4);
                if constexpr (FX == kMxE4m3) {
                    // a row block's parts at a time: those of all are too many registers
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        __builtin_amdgcn_sched_barrier(0);
                        i32x8 large, small;
                        mx_parts8(xf[s % FS][m][0], xf[s % FS][m][1], large, small);
#pragma unroll
                        for (int b = 0; b < NBW; ++b) multiply(small, s % FS, s, m, b);
#pragma unroll
                        for (int b = 0; b < NBW; ++b) {
                            multiply(large, s % FS, s, m, b);
                            if (m == MT - 1) {
                                __builtin_amdgcn_sched_barrier(0);
                                issue_w(s, nb + s, (nb + s) / 4, b);
                            }
                        }
                    }
                } else {
#pragma unroll
                    for (int b = 0; b < NBW; ++b) {
                        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            const u32x4 p = xf[s % FS][m][0];
                            multiply(i32x8{(int)p.x, (int)p.y, (int)p.z, (int)p.w, 0, 0, 0, 0}, s % FS, s, m, b);
                        }
                        __builtin_amdgcn_sched_barrier(0);
                        issue_w(s, nb + s, (nb + s) / 4, b);
                    }
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        // The sums are "used" here: with their next use behind a branch, the
        // compiler moves the whole round's products behind it.
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int b = 0; b < NBW; ++b) asm volatile("" : "+v"(acc[m][b]));
        if (nb >= KP) break;
        cb = nb;
        if (KC > SC && nb / 4 % SC == 0) {
            // other scale bytes, once every wave has read the old ones
            wait_vmcnt_lds<0>();
            barrier_nofence();
            load_scales(nb / 4);
            wait_vmcnt_lds<0>();
            if constexpr (AHEAD) {
                barrier_nofence();
#pragma unroll
                for (int u = 0; u < U; ++u) read_frags(u, u, 0, nb / 4);
            }
        }
    }
    wait_vmcnt_lds<0>();  // no load to LDS outlives the loop

    // lane (fr, fg) holds, of row m * 16 + fr, columns 4 fg + 0..3 of each group
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int r = m * 16 + fr;
        if constexpr (MODE == kGateUp) {
            static_assert(MODE != kGateUp || NBW == 4, "a wave holds one 32-block of h");
            if (m * 16 >= rows) break;  // uniform: the exchange below needs the whole wave
            const int c0 = (ct * 4 + wave) * 32;
            float h[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                h[i] = swiglu(acc[m][i / 4][i % 4], acc[m][2 + i / 4][i % 4]);
            unsigned big = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) big = mx_abs_max(big, mx_abs(h[i]));
            const int e = mx_exponent<FX>(__uint_as_float(row_max(big)));
            if (r >= rows || c0 >= a.N) continue;
            uint8_t *const hr = a.out + (size_t)(row0 + r) * mx_code_stride(FX, a.N);
            if constexpr (FX == kMxE4m3) {
                const uint2 q = mx_codes8_e4m3(h, mx_factor(e));
                *reinterpret_cast<unsigned *>(hr + c0 + 4 * fg) = q.x;
                *reinterpret_cast<unsigned *>(hr + c0 + 4 * fg + 16) = q.y;
            } else {
                const unsigned q = mx_codes8_e2m1(h, mx_factor(e));
                *reinterpret_cast<uint16_t *>(hr + c0 / 2 + 2 * fg) = (uint16_t)q;
                *reinterpret_cast<uint16_t *>(hr + c0 / 2 + 2 * fg + 8) = (uint16_t)(q >> 16);
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
            if constexpr (MODE == kDown) orow = (size_t)out_row[m];
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

// Weights that one row tile alone reads pass the caches by: 12 % of the time of
// 40 tokens (64 experts of 4096 x 1408, 8 a token) and 10 % of 512 tokens' (128 of
// 2880 x 2880, 4 a token).  For those that tiles share the same loads cost 12 %:
// chosen tile by tile.
//
// Grouped tiles of 64 e2m1 rows are 96 high for the experts of which that makes
// fewer (moe_tile_height).
template <int MT, int NBW, int FX, int MODE, int SL, int AHEAD>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2)))
    mxfp4_tile_kernel(TileArgs a) {
    // The work list goes expert by expert (dense: one), in it column tile by
    // column tile, the row tiles of a column tile side by side: those share
    // their weights, and all of an expert's share its rows of x.
    const int tiles = MODE == kDense ? a.row_tiles : a.count[0];
    const int at = xcd_order(blockIdx.x, a.col_tiles * tiles);
    if (at < 0) return;
    MoeTile own{0, 0, a.M, 0};
    if constexpr (MODE != kDense) own = a.tiles[at / a.col_tiles];
    const int height = MODE == kDense ? MT * 16 : moe_tile_height(own.rows, MT * 16, a.tall);
    const int nt = (own.rows + height - 1) / height, local = at - own.first * a.col_tiles;
    const int ct = local / nt, rt = local - ct * nt;
    if constexpr (MODE != kDense && MT == 4 && FX == kMxE2m1) {
        if (height > MT * 16) {
            if (nt == 1)
                mxfp4_tile<6, NBW, FX, MODE, SL, AHEAD, kCacheStream>(a, own, ct, rt);
            else
                mxfp4_tile<6, NBW, FX, MODE, SL, AHEAD, kCacheDefault>(a, own, ct, rt);
            return;
        }
    }
    if (nt == 1)
        mxfp4_tile<MT, NBW, FX, MODE, SL, AHEAD, kCacheStream>(a, own, ct, rt);
    else
        mxfp4_tile<MT, NBW, FX, MODE, SL, AHEAD, kCacheDefault>(a, own, ct, rt);
}

namespace {

// tiles: row tiles (grouped products: a bound on them).
template <int MT, int NBW, int FX, int MODE, int SL, int AHEAD>
int go(TileArgs a, int tiles, hipStream_t stream) {
    constexpr int TALL = MODE != kDense && MT == 4 && FX == kMxE2m1 ? 6 : MT;
    const size_t bytes = tile_lds_bytes(TALL, NBW, FX, SL, tile_scale_chunks(mxfp4_chunks(a.K), SL));
    constexpr size_t most = tile_lds_bytes(TALL, NBW, FX, SL, tile_scale_most(SL));
    static_assert(most <= 160 * 1024 - 256, "LDS of a workgroup");
    static std::atomic<unsigned long long> lds_set{0};
    const hipError_t e = allow_dynamic_lds(
        reinterpret_cast<const void *>(&mxfp4_tile_kernel<MT, NBW, FX, MODE, SL, AHEAD>), most, lds_set);
    if (e != hipSuccess) return (int)e;
    const int cols = MODE == kGateUp ? 128 : 64 * NBW;
    a.col_tiles = (a.N + cols - 1) / cols;
    a.row_tiles = tiles;
    const unsigned grid = (unsigned)a.col_tiles * (unsigned)tiles;
    hipLaunchKernelGGL((mxfp4_tile_kernel<MT, NBW, FX, MODE, SL, AHEAD>), dim3((grid + 7) / 8 * 8),
                       dim3(256),
                       bytes, stream, a);
    return (int)hipGetLastError();
}

// rows: 16, 32 or 64 a tile.  NB16, NB32, NB64: column groups a wave for each.
template <int MODE, int FX, int NB16, int NB32, int NB64>
int pick(const TileArgs &a, int rows, int tiles, hipStream_t stream) {
    if (rows <= 16) return go<1, NB16, FX, MODE, 4, 0>(a, tiles, stream);
    if (rows <= 32) return go<2, NB32, FX, MODE, 4, 0>(a, tiles, stream);
    return go<4, NB64, FX, MODE, 4, 0>(a, tiles, stream);
}

// Rows of e2m1: the smallest tile whose workgroups are at most one a CU.  A CU
// takes in 14-17 bytes a clock of these operands however many workgroups it holds
// and however deep their rings are, so a workgroup's time follows its bytes a step.
//
// Rows of e4m3: taking the rows' parts costs a wave as much as its products, and
// fewer rows by more columns a wave have fewer of them.  Below one workgroup a CU
// steps ahead pay; above it workgroups that alternate on a CU do, up to three.
// Measured (us, quantising included; 16 x 64, 16 x 128 ahead, 16 x 128, 32 x 128,
// 32 x 256; K = 7168, below 2880):
//   64 x 4096    18.4  19.3  20.9  27.9  37.4     128 x 4096   23.7  20.6  21.6  28.7  37.7
//   256 x 4096   36.3  28.9  28.0  30.2  39.1     512 x 4096   65.7  50.4  45.9  40.2  41.2
//   128 x 2880   12.6  11.9  12.1  16.0  21.4     512 x 2880   27.0  20.9  19.7  21.8  23.1
// 512 x 8192 x 4096: 75.7, 53.5, 49.9, 43.0 and 39.6.  Tiles of 64 rows: 49.5 at
// 512 x 4096.
enum DenseTile { kTile16x64, kTile16x128, kTile16x128Ring, kTile32x128Ring, kTile32x256Ring, kTile32x64, kTile32x128, kTile64x128 };

}  // namespace

int dense_tile(int M, int N, int fmt) {
    const long c64 = (N + 63) / 64, c128 = (N + 127) / 128;
    const long r16 = (M + 15) / 16, r32 = (M + 31) / 32;
    constexpr long cus = kNumCusMI355X;
    if (r16 * c64 <= cus) return kTile16x64;
    if (fmt == kMxE4m3)
        return r16 * c128 <= cus       ? kTile16x128
               : r16 * c128 <= 3 * cus ? kTile16x128Ring
               : r32 * c128 <= 3 * cus ? kTile32x128Ring
                                       : kTile32x256Ring;
    return r32 * c64 <= cus ? kTile32x64 : r32 * c128 <= cus ? kTile32x128 : kTile64x128;
}

namespace {

template <int FX>
int dense(const TileArgs &a, hipStream_t stream) {
    const int r16 = (a.M + 15) / 16, r32 = (a.M + 31) / 32, tile = dense_tile(a.M, a.N, FX);
    if (tile == kTile16x64) return go<1, 1, FX, kDense, 8, 2>(a, r16, stream);
    if constexpr (FX == kMxE4m3) {
        if (tile == kTile16x128) return go<1, 2, FX, kDense, 8, 2>(a, r16, stream);
        if (tile == kTile16x128Ring) return go<1, 2, FX, kDense, 4, 0>(a, r16, stream);
        if (tile == kTile32x128Ring) return go<2, 2, FX, kDense, 4, 0>(a, r32, stream);
        return go<2, 4, FX, kDense, 4, 0>(a, r32, stream);
    } else {
        if (tile == kTile32x64) return go<2, 1, FX, kDense, 8, 2>(a, r32, stream);
        if (tile == kTile32x128) return go<2, 2, FX, kDense, 8, 2>(a, r32, stream);
        return go<4, 2, FX, kDense, 8, 2>(a, (a.M + 63) / 64, stream);
    }
}

}  // namespace

// Of the tile that dense() picks: straight lines in K through 392 points a format.
double mxfp4_tile_time(int M, int N, int K, int fmt) {
    const long c128 = (N + 127) / 128;
    switch (dense_tile(M, N, fmt)) {
    case kTile16x64: return fmt == kMxE4m3 ? 5.2 + 1.65e-3 * K : 5.2 + 1.03e-3 * K;
    case kTile16x128: return 6.3 + 1.97e-3 * K;
    case kTile16x128Ring: return (M + 15) / 16 * c128 <= 2 * kNumCusMI355X ? 6.1 + 3.0e-3 * K : 7.6 + 4.1e-3 * K;
    case kTile32x128Ring: return 8.2 + 4.9e-3 * K;
    case kTile32x256Ring: return 14 + 6.6e-3 * K;
    case kTile32x64: return 6.6 + 1.2e-3 * K;
    case kTile32x128: return 7.0 + 1.64e-3 * K;
    default: {
        const double rounds = (double)(((M + 63) / 64 * c128 + kNumCusMI355X - 1) / kNumCusMI355X);
        return 5.0 + 5e-4 * K + rounds * (4.6 + 1.41e-3 * K);
    }
    }
}

int launch_mxfp4(const Mxfp4Args &p, hipStream_t stream) {
    TileArgs a{};
    a.x = p.x;
    a.x_stride = (unsigned)p.xs;
    a.xe = p.xe;
    a.x_rows = (unsigned)p.M;
    a.W = p.W;
    a.bias = p.bias;
    a.out = (uint8_t *)p.out;
    a.out_f32 = p.out_f32;
    a.M = p.M;
    a.N = p.N;
    a.K = p.K;
    return p.fmt == kMxE4m3 ? dense<kMxE4m3>(a, stream) : dense<kMxE2m1>(a, stream);
}

// The two products of the routed experts (kernels_moe.hip sorts and combines).
int launch_moe_gate_up(const MoeArgs &m, const MoeLists &s, const uint8_t *xq, const uint8_t *xe,
                       uint8_t *h, uint8_t *he, int rows, int tiles, hipStream_t stream) {
    TileArgs a{};
    a.x = xq;
    a.x_stride = (unsigned)mx_code_stride(m.fmt, m.H);
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
    a.tall = s.tall;
    return m.fmt == kMxE4m3 ? pick<kGateUp, kMxE4m3, 4, 4, 4>(a, rows, tiles, stream)
                            : pick<kGateUp, kMxE2m1, 4, 4, 4>(a, rows, tiles, stream);
}

int launch_moe_down(const MoeArgs &m, const MoeLists &s, const uint8_t *h, const uint8_t *he,
                    float *y, int rows, int tiles, hipStream_t stream) {
    TileArgs a{};
    a.x = h;
    a.x_stride = (unsigned)mx_code_stride(m.fmt, m.I);
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
    a.tall = s.tall;
    // Wide column tiles halve what the rows cost (e2m1, 2048 tokens: 170 -> 161 us;
    // e4m3, both products of 1024 tokens of 32 experts of 2880 x 1440: 133 -> 128);
    // with few rows more, narrower workgroups stream better (40: 32 -> 30).
    return m.fmt == kMxE4m3 ? pick<kDown, kMxE4m3, 2, 4, 4>(a, rows, tiles, stream)
                            : pick<kDown, kMxE2m1, 2, 2, 4>(a, rows, tiles, stream);
}

}  // namespace skg
