// kernels_latent_attention.hip -- attention over a paged cache of latent rows,
// absorbed form: all heads of a token share keys (576 values) and values (the
// first 512 of them), so (token, head) pairs are the rows of two products with
// the same tile of the cache.
#include <algorithm>

#include "internal.h"
#include "latent_common.h"
#include "latent_internal.h"
#include "lds_limit.h"

namespace skg {

namespace {

constexpr int kTile = 32;  // cache rows a step
constexpr int kRing = 4;   // steps in LDS

struct Shape {
    LatentArgs a;
    int tp;         // tokens a row tile
    int hg;         // head groups (row tiles a token, if it has more heads than a tile rows)
    int min_share;  // least number of steps a workgroup takes
};

// A sequence that ends in other workgroups' shares: parts of one row tile.
struct Shared {
    int b, i, g, parts;
};

template <int RG>
constexpr size_t part_floats() {
    return (size_t)RG * 32 * (SKG_LATENT + 2);
}
__host__ __device__ constexpr int row_bytes(bool e4m3) { return SKG_LATENT_ROW * (e4m3 ? 1 : 2); }
constexpr int kExchangeRow = 36;  // floats: 32 scores and a pad
template <int RG, bool E4M3>
constexpr size_t lds_bytes() {
    const size_t ring = (size_t)kRing * kTile * row_bytes(E4M3);
    return ring + (RG < 4 ? RG * 32 * kExchangeRow * 4 : 0) + 64;
}
static_assert(lds_bytes<2, false>() <= 160 * 1024 - 256, "a workgroup's LDS");
static_assert((SKG_LATENT_MAX_B + 1) * 8 <= kRing * kTile * row_bytes(true), "prefix sums fit the ring");

// Order of N fragments' reads from LDS (READS instructions each) and their MMAS
// matrix instructions: AHEAD fragments before their use, no more of them in registers.
template <int N, int AHEAD, int READS, int MMAS>
__device__ __forceinline__ void read_ahead() {
    __builtin_amdgcn_sched_group_barrier(0x100, AHEAD * READS, 0);
#pragma unroll
    for (int i = 0; i < N - AHEAD; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x8, MMAS, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x8, AHEAD * MMAS, 0);
}

// Steps of one row tile, at least one so that empty rows are written too.
__device__ __forceinline__ int tile_steps(int before, int n, int tp, int i) {
    return max(1, (before + min((i + 1) * tp, n) + kTile - 1) / kTile);
}
// Their sum over the row tiles before `upto` of a sequence with `n` new tokens
// behind `before` rows.  Tile i but the last sees before + (i + 1) tp rows; of 32
// successive tiles each residue's counts grow by tp.
__device__ __forceinline__ long steps_before(int before, int n, int tp, int upto) {
    const int tiles = (n + tp - 1) / tp;
    const int m = min(upto, tiles - 1);
    long sum = upto >= tiles && tiles > 0 ? tile_steps(before, n, tp, tiles - 1) : 0;
    if (m <= 0) return sum;
    const int ones = min(max((kTile - before) / tp, 0), m);  // tiles of one step
    sum += ones;
    const int left = m - ones, c0 = before + (ones + 1) * tp;
    for (int r = 0; r < min(left, kTile); ++r) {
        const long k = (left - r + kTile - 1) / kTile;
        sum += k * ((c0 + r * tp + kTile - 1) / kTile) + tp * (k * (k - 1) / 2);
    }
    return sum;
}

}  // namespace

// A workgroup of 4 waves takes 32 RG rows; CS = 4 / RG waves share 32 of them:
// each makes scores of its part of a step, all hold the weights, and each sums its
// part of the 512 columns.
template <int RG, bool E4M3>
__global__ void __launch_bounds__(256, 1) latent_attention_kernel(Shape s) {
    constexpr int CS = 4 / RG, R = 32 * RG, ROWB = row_bytes(E4M3), TILE = kTile * ROWB;
    constexpr int PIECES = ROWB / 16, LOADS = (8 * PIECES + 63) / 64;  // a wave brings 8 rows
    constexpr int DB = 16 / CS;                                       // blocks of 32 columns a wave
    extern __shared__ __attribute__((aligned(16))) unsigned char lds_raw[];
    const LatentArgs &a = s.a;
    float *exchange = reinterpret_cast<float *>(lds_raw + kRing * TILE);
    unsigned char *flags = lds_raw + kRing * TILE + (CS > 1 ? RG * 32 * kExchangeRow * 4 : 0);
    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int rg = wave / CS, cs = wave % CS;
    // neighbouring shares on one XCD: they read the same sequence
    const int G = gridDim.x, group = (G & 7) == 0 ? (int)(blockIdx.x & 7) * (G / 8) + (int)(blockIdx.x >> 3) : (int)blockIdx.x;
    const int cap = (int)min((long)a.W << a.page_shift, 0x7FFFFFFFL - 64);

    float *const ws = a.ws;
    Shared *const shared = reinterpret_cast<Shared *>(ws + 2 * (size_t)G * part_floats<RG>());

    // ---- this workgroup's share of all steps
    long *pre = reinterpret_cast<long *>(lds_raw);
    auto length = [&](int b) { return min(max(a.kv_lens[b], 0), cap); };
    block_prefix(a.B, pre, reinterpret_cast<long *>(flags), [&](int b) {
        const Tokens q = new_tokens(a.q_starts, b, a.T);
        return s.hg * steps_before(length(b) - q.n, q.n, s.tp, (q.n + s.tp - 1) / s.tp);
    });
    const long total = pre[a.B], share = max((long)s.min_share, (total + G - 1) / G);
    const long from = group * share;
    long left = min(total, from + share) - from;
    int b = 0, i = 0, g = 0;
    Tokens q{0, 0};
    int before = 0;
    int at = 0;  // first step in the row tile
    if (left > 0) {
        b = __builtin_amdgcn_readfirstlane(find_sequence(pre, a.B, from));
        q = new_tokens(a.q_starts, b, a.T);
        before = length(b) - q.n;
        const long off = from - pre[b];
        int lo = 0, hi = (q.n + s.tp - 1) / s.tp;
        while (hi - lo > 1) {
            const int step = (hi - lo + 63) / 64, cand = lo + lane * step;
            const bool in = cand < hi && s.hg * steps_before(before, q.n, s.tp, cand) <= off;
            const int idx = __popcll(__ballot(in)) - 1;
            lo += idx * step;
            hi = min(hi, lo + step);
        }
        i = __builtin_amdgcn_readfirstlane(lo);
        const int rest = (int)(off - s.hg * steps_before(before, q.n, s.tp, i));
        const int steps = tile_steps(before, q.n, s.tp, i);
        g = __builtin_amdgcn_readfirstlane(rest / steps);
        at = __builtin_amdgcn_readfirstlane(rest - g * steps);
    }
    __syncthreads();
    Shared mine{0, 0, 0, 0};

    // ---- constants of the lane
    const int half = lane >> 5, l15 = lane & 15, l31 = lane & 31, g4 = lane >> 4;
    unsigned src[LOADS];
#pragma unroll
    for (int k = 0; k < LOADS; ++k) {
        const int p = k * 64 + lane, row = p / PIECES, c = p % PIECES;
        const int from_c = E4M3 ? (c & ~3) | ((c & 3) ^ ((row >> 1) & 3)) : (c & ~7) | ((c & 7) ^ swz8(row & 7));
        src[k] = (unsigned)(row * ROWB + from_c * 16);
    }
    // fragments of keys: 32 rows by 16 values (CS == 1), or 16 rows by 32
    constexpr int KO = E4M3 ? (CS == 1 ? 4 : 2) : (CS == 1 ? 4 : 2);
    unsigned koff[KO];
#pragma unroll
    for (int j = 0; j < KO; ++j) {
        const int row = CS == 1 ? l31 : (cs & 1) * 16 + l15;
        if constexpr (E4M3) {
            const int sw = (row >> 1) & 3;
            koff[j] = (unsigned)(row * ROWB + (CS == 1 ? (j ^ sw) * 16 + half * 8
                                                       : ((j * 2 + (g4 >> 1)) ^ sw) * 16 + (g4 & 1) * 8));
        } else {
            koff[j] = (unsigned)(row * ROWB + (((CS == 1 ? j * 2 + half : j * 4 + g4) ^ swz8(row & 7)) * 16));
        }
    }
    // and of values, 32 columns by 16 rows: this lane's column from rows 4 half + 0 .. 3
    // and 8 + 4 half + 0 .. 3, as the scores' registers have them
    unsigned voff[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int dg = g4 & 1;
        if constexpr (E4M3) {
            const int k = l15 >> 1, row = (k >> 2) * 8 + 4 * half + (k & 3);
            voff[j] = (unsigned)(row * ROWB + (((j * 2 + dg) ^ ((row >> 1) & 3)) * 16) + (l15 & 1) * 8);
        } else {
            const int row = 4 * half + (l15 >> 2);
            voff[j] = (unsigned)(row * ROWB + (((j * 4 + dg * 2 + ((l15 & 3) >> 1)) ^ swz8(row)) * 16) + (l15 & 1) * 8);
        }
    }
    const float kv_scale = E4M3 ? a.scale[0] : 1.0f;
    const float factor = a.factor * kv_scale;

    // ---- row tiles of the share, one after another
    while (left > 0) {
        const int steps = tile_steps(before, q.n, s.tp, i);
        const int n = (int)min((long)(steps - at), left);  // this workgroup's steps of it
        const int j0 = i * s.tp;                           // first token
        const int lim0 = max(before + j0 + 1, 0);          // rows that it sees
        const int most = max(before + min(j0 + s.tp, q.n), 0);  // and the last one
        // this wave's rows: (token, head) of lane's row, and how many cache rows it sees
        auto place = [&](int r, int &tok, int &head) {
            if (a.H > R) {
                tok = j0;
                head = g * R + r;
                return head < a.H;
            }
            tok = r / a.H;
            head = r - tok * a.H;
            const bool ok = tok < s.tp && j0 + tok < q.n;
            tok += j0;
            return ok;
        };
        int tok, head;
        const bool live = place(rg * 32 + l31, tok, head);
        const int lim = live ? max(before + tok + 1, 0) : 0;

        // queries: fragments as the products take them
        constexpr int QR = CS == 2 ? 2 : 1, QK = CS == 1 ? 36 : 18;
        bf16x8 qf[QR][QK];
#pragma unroll
        for (int x = 0; x < QR; ++x) {
            int qt, qh;
            const int r = CS == 1 ? rg * 32 + l31 : rg * 32 + (CS == 2 ? x : cs >> 1) * 16 + l15;
            const bool ok = place(r, qt, qh);
            const uint16_t *p = a.q + ((size_t)(q.first + (ok ? qt : 0)) * a.H + (ok ? qh : 0)) * SKG_LATENT_ROW +
                                (CS == 1 ? half : g4) * 8;
#pragma unroll
            for (int k = 0; k < QK; ++k) {
                u32x4 v{0, 0, 0, 0};
                if (ok) v = *reinterpret_cast<const u32x4 *>(p + k * (CS == 1 ? 16 : 32));
                qf[x][k] = __builtin_bit_cast(bf16x8, v);
            }
        }

        f32x16 acc[DB];
        float m, l;
        bool careful = false;
        for (;;) {
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[d][r] = 0.0f;
            m = -__builtin_inff();
            l = 0.0f;

            // table entries of 64 pages, one a lane
            int first_page = -64, entry = -1;
            unsigned long seen = 0;  // four bits a step, the newest lowest: groups of 8 rows whose page is one
            auto issue = [&](int step, int slot) {
                const int row0 = step * kTile;
                const int last = (row0 + kTile - 1) >> a.page_shift, one = row0 >> a.page_shift;
                if (last >= first_page + 64) {
                    first_page = one;
                    const int e = first_page + lane;
                    entry = e < a.W ? a.table[(size_t)b * a.W + e] : -1;
                }
                unsigned bits = 0;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int p = __builtin_amdgcn_readlane(entry, ((row0 + 8 * w) >> a.page_shift) - first_page);
                    bits |= (p >= 0 && p < a.pages ? 1u : 0u) << w;
                }
                seen = seen << 4 | bits;
                const int row = row0 + 8 * wave;
                const int page = __builtin_amdgcn_readlane(entry, (row >> a.page_shift) - first_page);
                const int rows = (bits >> wave & 1u) ? min(max(most - row, 0), 8) : 0;
                const size_t off = ((size_t)(rows ? page : 0) << a.page_shift) + (row & ((1 << a.page_shift) - 1));
                const Rsrc rs = make_rsrc(a.cache + off * ROWB, (unsigned)(rows * ROWB));
                unsigned char *dst = lds_raw + slot * TILE + wave * 8 * ROWB;
#pragma unroll
                for (int k = 0; k < LOADS; ++k)
                    if ((k + 1) * 64 <= 8 * PIECES || lane < 8 * PIECES - k * 64)
                        lds_load16<kCacheDefault>(rs, dst + k * 1024, src[k]);
            };

            for (int k = 0; k < kRing - 1; ++k)
                if (k < n) issue(at + k, k);
            int slot = 0, fill = kRing - 1;
            for (int k = 0; k < n; ++k) {
                // loads of up to kRing - 2 later steps may be under way
                const int newer = min(kRing - 2, n - 1 - k);
                if (newer == 2) wait_vmcnt_lds<2 * LOADS>();
                else if (newer == 1) wait_vmcnt_lds<LOADS>();
                else wait_vmcnt_lds<0>();
                barrier_nofence();
                const unsigned bits = (unsigned)(seen >> (4 * newer)) & 15u;
                if (k + kRing - 1 < n) issue(at + k + kRing - 1, fill);
                const unsigned char *tile = lds_raw + slot * TILE;
                const int row0 = (at + k) * kTile;

                // scores, transposed: register r of a lane is row 8 (r / 4) + 4 half + r % 4
                // of the cache, its column the lane's (token, head)
                f32x16 z;
                if constexpr (CS == 1) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) z[r] = 0.0f;
#pragma unroll
                    for (int c = 0; c < 36; ++c) {
                        bf16x8 kf;
                        if constexpr (E4M3)
                            kf = e4m3_to_bf16(*reinterpret_cast<const i32x2 *>(tile + koff[c & 3] + (c >> 2) * 64));
                        else
                            kf = *reinterpret_cast<const bf16x8 *>(tile + koff[c & 3] + (c >> 2) * 128);
                        z = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[0][c], z, 0, 0, 0);
                    }
                } else {
                    f32x4 y[QR][2];
#pragma unroll
                    for (int x = 0; x < QR; ++x) y[x][0] = y[x][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int c = 0; c < 18; ++c) {
                        bf16x8 kf;
                        if constexpr (E4M3)
                            kf = e4m3_to_bf16(*reinterpret_cast<const i32x2 *>(tile + koff[c & 1] + (c >> 1) * 64));
                        else
                            kf = *reinterpret_cast<const bf16x8 *>(tile + koff[c & 1] + (c >> 1) * 128);
#pragma unroll
                        for (int x = 0; x < QR; ++x)
                            y[x][c & 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[x][c], y[x][c & 1], 0, 0, 0);
                    }
                    read_ahead<18, 6, 1, QR>();
                    float *ex = exchange + rg * 32 * kExchangeRow;
#pragma unroll
                    for (int x = 0; x < QR; ++x)
                        *reinterpret_cast<f32x4 *>(ex + ((CS == 2 ? x : cs >> 1) * 16 + l15) * kExchangeRow +
                                                   (cs & 1) * 16 + g4 * 4) = y[x][0] + y[x][1];
                    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
                    barrier_nofence();
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        const f32x4 w = *reinterpret_cast<const f32x4 *>(ex + l31 * kExchangeRow + 8 * v + 4 * half);
#pragma unroll
                        for (int r = 0; r < 4; ++r) z[4 * v + r] = w[r];
                    }
                }
#pragma unroll
                for (int r = 0; r < 16; ++r) z[r] *= factor;
                const bool masked = row0 + kTile > lim0 || bits != 15u;
                if (masked) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const int row = row0 + 8 * (r >> 2) + 4 * half + (r & 3);
                        z[r] = row < lim && (bits >> (r >> 2) & 1u) ? z[r] : -__builtin_inff();
                    }
                }
                float top = z[0];
#pragma unroll
                for (int r = 1; r < 16; ++r) top = fmaxf(top, z[r]);
                top = other_half_max(top);
                // The running maximum follows only where a score is over 2^8 times it: sums and
                // weights then stay below 2^8 times their number, and the columns' sums are
                // multiplied in few steps only.
                if (__any(top > m + 8.0f)) {
                    const float next = fmaxf(m, top);
                    const float down = next == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(m - next);
                    m = next;
                    l *= down;
#pragma unroll
                    for (int d = 0; d < DB; ++d)
#pragma unroll
                        for (int r = 0; r < 16; ++r) acc[d][r] *= down;
                }
                const float ref = m == -__builtin_inff() ? 0.0f : m;
                float p[16];
#pragma unroll
                for (int r = 0; r < 16; ++r) p[r] = __builtin_amdgcn_exp2f(z[r] - ref);
                // the registers of eight scores are what the second product takes, as they lie
                const bf16x8 pf[2] = {to_bf16x8(p), to_bf16x8(p + 8)};
                l = add_bf16x8(pf[1], add_bf16x8(pf[0], l));
                if (__builtin_expect(careful && masked, 0)) {
                    // Rows with infinities or NaN that some of the tile's tokens see and some do
                    // not: their products by vector instructions for those that do, and zeros
                    // in their place for the matrix instruction.
                    bool bad = false;
                    for (int e = 0; e < ROWB * 512 / 576 / 8 / 4; ++e) {
                        const unsigned w = *reinterpret_cast<const unsigned *>(
                            tile + (wave * 8 + (lane >> 3)) * ROWB + (lane & 7) * (ROWB * 512 / 576 / 8) + e * 4);
                        if constexpr (E4M3) {
                            const unsigned u = w & 0x7F7F7F7Fu;
                            bad |= ((u + 0x01010101u) & 0x80808080u) != 0;
                        } else {
                            bad |= (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
                        }
                    }
                    unsigned long long any = __ballot(bad);
                    unsigned rows8 = 0;
#pragma unroll
                    for (int r = 0; r < 8; ++r) rows8 |= ((any >> (8 * r)) & 0xFFull ? 1u : 0u) << r;
                    if (lane == 0) flags[wave] = (unsigned char)rows8;
                    __syncthreads();
                    const unsigned flagged = __builtin_amdgcn_readfirstlane(*reinterpret_cast<const unsigned *>(flags));
                    for (unsigned f = flagged; f; f &= f - 1) {
                        const int k = __builtin_ctz(f), r = (k >> 3) * 4 + (k & 3), kh = (k >> 2) & 1;
                        float mine_p = 0.0f;
#pragma unroll
                        for (int u = 0; u < 16; ++u) mine_p = u == r ? p[u] : mine_p;
                        const float pk = __shfl(mine_p, l31 + 32 * kh, 64);
                        const bool sees = row0 + k < lim && (bits >> (k >> 3) & 1u);
#pragma unroll
                        for (int d = 0; d < DB; ++d)
#pragma unroll
                            for (int v = 0; v < 4; ++v) {
                                const int col = (cs * DB + d) * 32 + 8 * v + 4 * half;
                                float y[4];
                                if constexpr (E4M3) {
                                    const int c = col >> 4;
                                    const unsigned w = *reinterpret_cast<const unsigned *>(
                                        tile + k * ROWB + ((c & ~3) | ((c & 3) ^ ((k >> 1) & 3))) * 16 + (col & 15));
                                    const bf16x8 c8 = e4m3_to_bf16(i32x2{(int)w, 0});
#pragma unroll
                                    for (int u = 0; u < 4; ++u) y[u] = (float)c8[u];
                                } else {
                                    const int c = col >> 3;
                                    const uint2 w = *reinterpret_cast<const uint2 *>(
                                        tile + k * ROWB + ((c & ~7) | ((c & 7) ^ swz8(k & 7))) * 16 + (col & 7) * 2);
                                    y[0] = bf16_lo(w.x);
                                    y[1] = bf16_hi(w.x);
                                    y[2] = bf16_lo(w.y);
                                    y[3] = bf16_hi(w.y);
                                }
#pragma unroll
                                for (int u = 0; u < 4; ++u)
                                    if (sees) acc[d][4 * v + u] = __builtin_fmaf(pk, y[u], acc[d][4 * v + u]);
                            }
                    }
                    __syncthreads();
                    for (unsigned f = flagged; f; f &= f - 1)
                        for (int e = t; e < ROWB * 512 / 576 / 4; e += 256)
                            *reinterpret_cast<unsigned *>(const_cast<unsigned char *>(tile) + __builtin_ctz(f) * ROWB + e * 4) = 0;
                    __syncthreads();
                }
#pragma unroll
                for (int d = 0; d < DB; ++d) {
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk) {
                        const unsigned char *v = tile + voff[d & 1] + kk * 16 * ROWB;
                        bf16x8 vf;
                        if constexpr (E4M3) {
                            vf = e4m3_to_bf16(lds_transposed8(v + ((cs * DB + d) >> 1) * 64));
                        } else {
                            const s16x4 x = lds_transposed4(v + ((cs * DB + d) >> 1) * 128);
                            const s16x4 y = lds_transposed4(v + ((cs * DB + d) >> 1) * 128 + 8 * ROWB);
                            vf = __builtin_bit_cast(bf16x8, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
                        }
                        acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf, pf[kk], acc[d], 0, 0, 0);
                    }
                }
                read_ahead<DB * 2, 4, E4M3 ? 1 : 2, 1>();
                slot = slot + 1 == kRing ? 0 : slot + 1;
                fill = fill + 1 == kRing ? 0 : fill + 1;
            }
            wait_vmcnt_lds<0>();
            __syncthreads();  // the ring is free
            // An infinity or NaN in a cache row reaches, by 0 times itself, tokens that do
            // not see the row.  If there is any in the sums of a row tile whose tokens see
            // different rows, its masked steps are taken apart.
            if (careful || (at + n) * kTile <= lim0 || lim0 >= most) break;
            bool bad = false;
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r) bad |= not_finite(acc[d][r]);
            const unsigned long long found = __ballot(bad && live);
            if (lane == 0) flags[wave] = found != 0;
            __syncthreads();
            const unsigned some = __builtin_amdgcn_readfirstlane(*reinterpret_cast<const unsigned *>(flags));
            __syncthreads();
            if (!some) break;
            careful = true;
        }
        l = other_half_sum(l);

        if (at == 0 && n == steps) {
            const float inv = l == 0.0f ? 0.0f : kv_scale / l;
            if (live) {
                uint16_t *o = a.out + ((size_t)(q.first + tok) * a.H + head) * SKG_LATENT + cs * DB * 32 + 4 * half;
#pragma unroll
                for (int d = 0; d < DB; ++d)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        *reinterpret_cast<uint2 *>(o + d * 32 + 8 * v) =
                            to_bf16x4(acc[d][4 * v] * inv, acc[d][4 * v + 1] * inv, acc[d][4 * v + 2] * inv, acc[d][4 * v + 3] * inv);
            }
        } else {
            // a part: the sums in the registers' order, then maxima and sums of weights
            float *part = ws + (2 * (size_t)group + (at == 0 ? 1 : 0)) * part_floats<RG>();
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    *reinterpret_cast<f32x4 *>(part + (((rg * 16 + cs * DB + d) * 4 + v) * 64 + lane) * 4) =
                        f32x4{acc[d][4 * v], acc[d][4 * v + 1], acc[d][4 * v + 2], acc[d][4 * v + 3]};
            if (cs == 0 && half == 0) {
                float *ml = part + R * SKG_LATENT + (rg * 32 + l31) * 2;
                ml[0] = m;
                ml[1] = l;
            }
            if (at == 0) mine = Shared{b, i, g, 1 + (int)((steps - n + share - 1) / share)};
        }

        left -= n;
        at = 0;
        if (left > 0 && ++g == s.hg) {
            g = 0;
            if (++i * s.tp >= q.n) {
                i = 0;
                do {
                    ++b;
                    q = new_tokens(a.q_starts, b, a.T);
                } while (q.n == 0);  // steps are left, so there is one
                before = length(b) - q.n;
            }
        }
    }
    if (t == 0) shared[group] = mine;
}

// Row tiles that several workgroups shared: parts in the order of the steps.  One
// workgroup for a group and 32 columns.
template <int RG>
__global__ void __launch_bounds__(256) latent_combine_kernel(Shape s, const float *scale) {
    constexpr int R = 32 * RG;
    const LatentArgs &a = s.a;
    const int group = blockIdx.x, G = gridDim.x, d = blockIdx.y;
    const Shared e = reinterpret_cast<const Shared *>(a.ws + 2 * (size_t)G * part_floats<RG>())[group];
    if (e.parts < 2) return;
    const Tokens q = new_tokens(a.q_starts, e.b, a.T);
    const int t = threadIdx.x, v = t >> 6, lane = t & 63, half = lane >> 5;
    const float kv_scale = scale ? scale[0] : 1.0f;
    for (int rg = 0; rg < RG; ++rg) {
        const int r = rg * 32 + (lane & 31);
        int tok = e.i * s.tp, head = e.g * R + r;
        bool live = head < a.H;
        if (a.H <= R) {
            const int x = r / a.H;
            head = r - x * a.H;
            live = x < s.tp && tok + x < q.n;
            tok += x;
        }
        auto part = [&](int p) { return a.ws + (2 * (size_t)(group + p) + (p == 0 ? 1 : 0)) * part_floats<RG>(); };
        float m = -__builtin_inff();
        for (int p = 0; p < e.parts; ++p) m = fmaxf(m, part(p)[R * SKG_LATENT + 2 * r]);
        const float ref = m == -__builtin_inff() ? 0.0f : m;
        float l = 0.0f;
        f32x4 sum{0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
        for (int p = 0; p < e.parts; ++p) {
            const float *x = part(p);
            const float w = __builtin_amdgcn_exp2f(x[R * SKG_LATENT + 2 * r] - ref);
            const f32x4 y = *reinterpret_cast<const f32x4 *>(x + (((rg * 16 + d) * 4 + v) * 64 + lane) * 4);
            // a part that saw no row has sums of 0
            l = __builtin_fmaf(w, x[R * SKG_LATENT + 2 * r + 1], l);
#pragma unroll
            for (int u = 0; u < 4; ++u) sum[u] = __builtin_fmaf(w, y[u], sum[u]);
        }
        if (!live) continue;
        const float inv = l == 0.0f ? 0.0f : kv_scale / l;
        *reinterpret_cast<uint2 *>(a.out + ((size_t)(q.first + tok) * a.H + head) * SKG_LATENT + d * 32 + 8 * v + 4 * half) =
            to_bf16x4(sum[0] * inv, sum[1] * inv, sum[2] * inv, sum[3] * inv);
    }
}

namespace {

template <int RG, bool E4M3>
int go(const LatentArgs &a, hipStream_t stream) {
    constexpr int R = 32 * RG;
    Shape s{a, a.H > R ? 1 : R / a.H, a.H > R ? (a.H + R - 1) / R : 1, 4};
    static std::atomic<unsigned long long> done{0};
    constexpr size_t lds = lds_bytes<RG, E4M3>();
    const hipError_t e = allow_dynamic_lds((const void *)latent_attention_kernel<RG, E4M3>, lds, done);
    if (e != hipSuccess) return (int)e;
    hipLaunchKernelGGL((latent_attention_kernel<RG, E4M3>), dim3(kLatentGroups), dim3(256), lds, stream, s);
    const hipError_t f = hipGetLastError();
    if (f != hipSuccess) return (int)f;
    hipLaunchKernelGGL((latent_combine_kernel<RG>), dim3(kLatentGroups, 16), dim3(256), 0, stream, s, a.scale);
    return (int)hipGetLastError();
}

template <bool E4M3>
int by_rows(const LatentArgs &a, int rows, hipStream_t stream) {
    return rows == 32 ? go<1, E4M3>(a, stream) : go<2, E4M3>(a, stream);
}

}  // namespace

int latent_rows(int B, int T, int H) {
    // row tiles of the call if its tokens are spread evenly
    for (int rows = 64; rows > 32; rows /= 2) {
        const long tp = H > rows ? 1 : rows / H, hg = H > rows ? (H + rows - 1) / rows : 1;
        const long each = ((long)T + B - 1) / B;
        if (rows / 2 < H * each && B * ((each + tp - 1) / tp) * hg >= kLatentGroups) return rows;
    }
    return 32;
}

size_t latent_workspace_bytes(int rows) {
    return 2 * (size_t)kLatentGroups * rows * (SKG_LATENT + 2) * 4 + kLatentGroups * sizeof(Shared);
}

int launch_latent_attention(const LatentArgs &a, bool e4m3, int rows, hipStream_t stream) {
    return e4m3 ? by_rows<true>(a, rows, stream) : by_rows<false>(a, rows, stream);
}

}  // namespace skg
