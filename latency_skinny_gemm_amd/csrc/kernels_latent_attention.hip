// kernels_latent_attention.hip -- attention over a paged cache of latent rows,
// absorbed form: all heads of a token share keys (576 values) and values (the
// first 512 of them), so (token, head) pairs are the rows of two products with
// the same tile of the cache.
#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "latent_common.h"
#include "latent_internal.h"
#include "lds_limit.h"

namespace skg {

namespace {

constexpr int kTile = 32;  // cache rows a step
constexpr int kRing = 4;   // steps in LDS

// Workgroups: two a CU where two rings fit its LDS.
constexpr int groups_of(int rg, bool e4m3) { return rg == 1 && e4m3 ? 512 : 256; }

struct Shape {
    LatentArgs a;
    int tp;         // tokens a row tile
    int hg;         // head groups (row tiles a token, if it has more heads than a tile rows)
    int teams;      // groups that hold all head groups of some tokens
    int min_share;  // least number of steps a workgroup takes.  With 2, 4, 6 and 8: one token of 128 heads over 4000 bf16
                    // rows 24.4, 21.3, 20.5 and 21.3 us; 10 sequences of 16 heads over 3000 e4m3 rows 22.9, 22.4, 23.4 and 25.6
    int anew;       // steps that beginning a row tile costs: with 5, 8, 12, 16 600 tokens over their own rows, 20 heads,
                    // take 51, 48, 47, 49 us, 512 tokens over 8192 rows, 128 heads, 885, 870, 860, 868; without 153, 929
    int by_tile;    // records of row tiles, all of which are known on the host; else of workgroups
};

// A row tile that begins in `group`'s share: how many groups' shares it reaches over.
struct Shared {
    int b, i, group, parts;
};

template <int RG>
constexpr size_t part_floats() {
    return (size_t)RG * 32 * (SKG_LATENT + 2);
}
__host__ __device__ constexpr int row_bytes(bool e4m3) { return SKG_LATENT_ROW * (e4m3 ? 1 : 2); }
// The ring; two steps' weights of 32 cache rows by 32 rows in bf16 for each four
// waves, or one step's scores in fp32; flags.
constexpr int kWeights = 32 * 32;
template <int RG, bool E4M3>
constexpr size_t lds_bytes() {
    return (size_t)kRing * kTile * row_bytes(E4M3) + 2 * RG * kWeights * 2 + 64;
}
static_assert(lds_bytes<2, false>() <= 160 * 1024 && 2 * lds_bytes<1, true>() <= 160 * 1024, "a CU's LDS");
static_assert((SKG_LATENT_MAX_B + 1) * 8 <= kRing * kTile * row_bytes(true), "prefix sums fit the ring");

// Sums of weighted codes to values: times the cache's scale, over the sum of weights l; 0
// where there is none.  The quotient of a small scale may fall below fp32's normal
// numbers, where it has few bits; then 2^64 is taken out of it.
struct Quotient {
    float inv, rest;
    __device__ __forceinline__ Quotient(float scale, float l) {
        const float up = __builtin_fabsf(scale) < 0x1p-64f ? 0x1p64f : 1.0f;
        inv = l == 0.0f ? 0.0f : scale * up / l;
        rest = up == 1.0f ? 1.0f : 0x1p-64f;
    }
    __device__ __forceinline__ float of(float sum) const { return sum * inv * rest; }
};

// Steps of one row tile, at least one so that empty rows are written too.
__device__ __forceinline__ int tile_steps(int before, int n, int tp, int i) {
    return max(1, (before + min((i + 1) * tp, n) + kTile - 1) / kTile);
}
// Their sum over the row tiles before `upto` of a sequence with `n` new tokens behind
// `before` rows.  Tile i but the last sees x = before + (i + 1) tp rows and has
// (x + (-x mod 32)) / 32 steps; -x mod 32 has the period 32 / g, g the largest power of
// two that divides tp and 32, over which it takes every value of its remainder mod g.
__device__ __forceinline__ long steps_before(int before, int n, int tp, int upto) {
    static_assert(kTile == 32, "");
    const int tiles = (n + tp - 1) / tp;
    const int m = min(upto, tiles - 1);
    long sum = upto >= tiles && tiles > 0 ? tile_steps(before, n, tp, tiles - 1) : 0;
    if (m <= 0) return sum;
    const int ones = min(max((kTile - before) / tp, 0), m);  // tiles of one step
    const int left = m - ones, c0 = before + (ones + 1) * tp;
    const int log_g = min(__builtin_ctz(tp), 5), g = 1 << log_g, period = 32 >> log_g;
    long over = (long)(left >> (5 - log_g)) * (period * (-c0 & (g - 1)) + 16 * (period - 1));
    for (int r = 0; r < (left & (period - 1)); ++r) over += -(c0 + r * tp) & 31;
    return sum + ones + (((long)left * c0 + (long)tp * ((long)left * (left - 1) / 2) + over) >> 5);
}

}  // namespace

// A workgroup of four waves takes 32 RG rows, 4 / RG waves 32 of them: each makes the
// weights of half of a step's cache rows and of half of its own (all, if they are two
// waves), which all of them then read from LDS, and sums its
// part of the 512 columns.  The weights are made a step ahead: one barrier a
// step, behind which its weights and the next step's cache rows are there.  A barrier
// starts all waves at the same point, so that each has to fill its own waits: scores
// run while the weights come from LDS, sums beside the next weights' vector
// instructions, and the loads of a later step (36 KB at 64 bytes a clock) between both.
//
// Weights are 2^(score - m), m a row's maximum as of the last step in which a score was
// over m + 8: sums and weights then stay below 2^8 times their number, no wave needs
// the others' scores, and the sums are multiplied in few steps only.  In those steps
// (the first of a row tile, rarely a later one) all scores go through LDS.
//
// Workgroups that hold different heads of the same tokens form a team, which takes
// its share of all steps together, so that a cache row is read from memory once.  Shares
// are equal numbers of steps, the beginning of a tile counted as some, whatever row tile
// they begin or end in, or of one tile each where that makes them little longer; parts of
// a tile are joined by the kernel below.
//
// 512 tokens of 128 heads over 8192 rows: 857 to 940 us by the card, 1020 to 930 TFLOP/s, at
// 2.0 GHz of 2.4.  The matrix pipes are busy 43 % of the cycles; a wave, the only one of its
// SIMD, issues instructions in 47 % of them, waits for counters and barriers in 25 % and for
// a unit to take its next instruction in 28 %.  Decode of 128 sequences, 128 heads, 588 MB:
// 176 us, of which its loads alone take 150 (3.9 TB/s: a team's workgroups have the same
// rows under way); 32 sequences, 16 heads, e4m3, 272 MB: 59 us, loads alone 57.  One token
// of 128 heads over 4000 rows: 16 us; one workgroup's share alone takes 9.0 with one step
// and 12.4 with its six (0.7 a step).
//
// A share brings its ring's rows up to the sequence's end, not its own: three steps more
// than it uses (the 32 sequences read 299 MB for 272).
template <int RG, int CS, bool E4M3>
__global__ void __launch_bounds__(64 * RG * CS)
    __attribute__((amdgpu_waves_per_eu(groups_of(RG, E4M3) / 256 * RG * CS / 4, groups_of(RG, E4M3) / 256 * RG * CS / 4)))
latent_attention_kernel(Shape s) {
    constexpr int NW = RG * CS, R = 32 * RG, ROWB = row_bytes(E4M3), TILE = kTile * ROWB;
    constexpr int QR = 3 - CS / 2;                                                       // halves of the 32 rows that a wave scores
    constexpr int WR = kTile / NW, PIECES = ROWB / 16, LOADS = (WR * PIECES + 63) / 64;  // rows that a wave brings
    constexpr int DB = 16 / CS;                                                         // blocks of 32 columns a wave
    constexpr int KD = 4, VD = 3, YN = 2;  // fragments of keys and of values under way, sums of a score
    using Key = std::conditional_t<E4M3, i32x2, u32x4>;  // fragments as they lie in LDS
    using Value = std::conditional_t<E4M3, i32x2, s16x8>;
    extern __shared__ __attribute__((aligned(16))) unsigned char lds_raw[];
    const LatentArgs &a = s.a;
    const int t = threadIdx.x, lane = t & 63, wave = uniform(t >> 6);
    const int rg = wave / CS, cs = wave % CS;
    const int step_half = cs & 1;
    unsigned char *const exchange = lds_raw + kRing * TILE;
    unsigned *const flags = reinterpret_cast<unsigned *>(exchange + 2 * RG * kWeights * 2);
    // neighbouring groups on one XCD
    const int G = gridDim.x, group = (int)(blockIdx.x & 7) * (G / 8) + (int)(blockIdx.x >> 3);
    const int team = group / s.hg, g = group - team * s.hg;
    const int cap = (int)min((long)a.W << a.page_shift, 0x7FFFFFFFL - 64);
    auto length = [&](int b) { return min(max(a.kv_lens[b], 0), cap); };

    Shared *const records = reinterpret_cast<Shared *>(a.ws + 2 * (size_t)G * part_floats<RG>());

    // ---- this team's share of all steps
    // A row tile counts as `anew` steps more than it has, in front of them; a share that
    // ends among those does not begin the tile.
    int b = 0, i = 0, before = 0, unit = 0;  // sequence, row tile and its first counted step; rows before the sequence's new ones
    Tokens q{0, 0};
    long share, left = 0;
    auto uniform_long = [](long v) { return (long)((unsigned long)(unsigned)uniform((int)(v >> 32)) << 32 | (unsigned)uniform((int)v)); };
    auto share_of = [&](long total) {
        return max((long)s.min_share, total <= 0x7FFFFFFFL - 512 ? (long)((unsigned)(total + s.teams - 1) / (unsigned)s.teams) : (total + s.teams - 1) / s.teams);
    };
    auto of_lane = [](long v, int l) {
        return (long)((unsigned long)(unsigned)__builtin_amdgcn_readlane((int)(v >> 32), l) << 32 | (unsigned)__builtin_amdgcn_readlane((int)v, l));
    };
    // steps `off` .. of sequence b
    auto seek = [&](long off) {
        int lo = 0, hi = (q.n + s.tp - 1) / s.tp;
        while (hi - lo > 1) {
            const int step = (hi - lo + 63) / 64, cand = lo + lane * step;
            const bool in = cand < hi && steps_before(before, q.n, s.tp, cand) + (long)cand * s.anew <= off;
            const int idx = __popcll(__ballot(in)) - 1;
            lo += idx * step;
            hi = min(hi, lo + step);
        }
        i = uniform(lo);
        unit = uniform((int)(off - (i ? steps_before(before, q.n, s.tp, i) + (long)i * s.anew : 0)));
    };
    if (a.B <= 64) {  // a sequence a lane, every wave for itself: one round of loads, no barrier
        const int own_b = min(lane, a.B - 1);
        const Tokens own = new_tokens(a.q_starts, own_b, a.T);
        const int own_before = length(own_b) - own.n, tiles = lane < a.B ? (own.n + s.tp - 1) / s.tp : 0;
        const int longest = tiles ? tile_steps(own_before, own.n, s.tp, tiles - 1) : 0;
        const long steps = steps_before(own_before, own.n, s.tp, tiles) + (long)tiles * s.anew;
        long upto = steps;
        int all = tiles;
        for (int d = 1; d < a.B; d <<= 1) {
            const long u = __shfl_up(upto, d, 64);
            const int v = __shfl_up(all, d, 64);
            if (lane >= d) upto += u, all += v;
        }
        const long total = of_lane(upto, a.B - 1);
        all = __builtin_amdgcn_readlane(all, a.B - 1);
        share = uniform_long(share_of(total));
        // Shares of one row tile each, where they are little longer: a team that goes on in
        // the middle of a tile begins it as well.
        int whole = (int)min(share_of(total - (long)all * s.anew), 0x7FFFFFFFL), parts = 0, need = s.teams + 1;
        while (all <= s.teams && whole <= share + s.anew) {
            parts = (longest + whole - 1) / whole;
            need = tiles * parts;
            for (int d = 1; d < a.B; d <<= 1) {
                const int v = __shfl_up(need, d, 64);
                if (lane >= d) need += v;
            }
            const int last = __builtin_amdgcn_readlane(need, a.B - 1);
            if (last <= s.teams) break;
            whole = max(whole + 1, (int)((long)whole * last / s.teams));
            need = s.teams + 1;
        }
        whole = uniform(whole);
        const bool aligned = __builtin_amdgcn_readlane(need, a.B - 1) <= s.teams;
        const long from = team * share;
        const unsigned long long behind = __ballot(aligned ? need > team : upto > from);
        if (team < s.teams && behind) {
            b = __builtin_ctzll(behind);
            q = {__builtin_amdgcn_readlane(own.first, b), __builtin_amdgcn_readlane(own.n, b)};
            before = __builtin_amdgcn_readlane(own_before, b);
            if (aligned) {
                const int k = __builtin_amdgcn_readlane(parts, b), r = team - __builtin_amdgcn_readlane(need - tiles * parts, b);
                share = whole;
                i = uniform(r / k);
                unit = s.anew + (r - i * k) * whole;
                left = max(min(whole, tile_steps(before, q.n, s.tp, i) + s.anew - unit), 0);
            } else {
                left = min(total, from + share) - from;
                seek(from - of_lane(upto - steps, b));
            }
        }
    } else {
        long *pre = reinterpret_cast<long *>(lds_raw);
        block_prefix<NW>(a.B, pre, reinterpret_cast<long *>(exchange), [&](int b) {
            const Tokens q = new_tokens(a.q_starts, b, a.T);
            const int tiles = (q.n + s.tp - 1) / s.tp;
            return steps_before(length(b) - q.n, q.n, s.tp, tiles) + (long)tiles * s.anew;
        });
        const long total = pre[a.B];
        share = uniform_long(share_of(total));
        const long from = team * share;
        left = team < s.teams ? min(total, from + share) - from : 0;
        if (left > 0) {
            b = uniform(find_sequence(pre, a.B, from));
            q = uniform(new_tokens(a.q_starts, b, a.T));
            before = uniform(length(b)) - q.n;
            seek(from - pre[b]);
        }
    }
    __syncthreads();
    if (t < 16) flags[t] = 0;
    unsigned epoch = 0;  // steps so far: a step's flag is its number
    Shared mine{0, 0, 0, 0};

    // ---- the first row tile's queries and table entries, under way with the constants
    const int half = lane >> 5, l15 = lane & 15, l31 = lane & 31, g4 = lane >> 4;
    const int own_row = (CS == 4 ? (cs >> 1) * 16 : 0) + l15;  // whose weights this lane makes; and, with both halves, own_row + 16
    int j0 = i * s.tp;                                         // the row tile's first token
    // (token, head) of a row of the tile
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
    // queries: fragments of 16 rows by 32 values
    bf16x8 qf[QR][18];
    auto load_queries = [&] {
        const Rsrc rq = make_rsrc(a.q + ((size_t)(q.first + j0) * a.H + (a.H > R ? g * R : 0)) * SKG_LATENT_ROW, left > 0 ? R * SKG_LATENT_ROW * 2u : 0u);
#pragma unroll
        for (int x = 0; x < QR; ++x) {
            int qt, qh;
            const int r = rg * 32 + own_row + 16 * x;  // rows of a tile lie one after another
            const unsigned off = place(r, qt, qh) ? (unsigned)(r * SKG_LATENT_ROW + g4 * 8) * 2u : kOOB;
#pragma unroll
            for (int k = 0; k < 18; ++k) qf[x][k] = __builtin_bit_cast(bf16x8, load16<kCacheDefault>(rq, off + k * 64));
        }
    };
    const bool wide = a.page_shift >= 5;
    auto table_entry = [&](int step) {
        const long e = ((long)step * kTile + here(threadIdx.x & 63) * (wide ? kTile : 8)) >> a.page_shift;
        return e < a.W ? a.table[(size_t)b * a.W + e] : -1;
    };
    load_queries();
    int page = left > 0 ? table_entry(max(unit - s.anew, 0)) : -1;

    // ---- constants of the lane
    unsigned src[LOADS];
#pragma unroll
    for (int k = 0; k < LOADS; ++k) {
        const int p = k * 64 + lane, row = p / PIECES, c = p % PIECES, tr = wave * WR + row;
        const int piece = E4M3 ? (c & ~3) | ((c & 3) ^ swz4(tr)) : (c & ~7) | ((c & 7) ^ swz8(tr));
        src[k] = (unsigned)(row * ROWB + piece * 16);
    }
    // fragments of keys, 16 rows by 32 values
    unsigned koff[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int row = step_half * 16 + l15;
        koff[j] = (unsigned)(row * ROWB) + (unsigned)(E4M3 ? ((j * 2 + (g4 >> 1)) ^ swz4(row)) * 16 + (g4 & 1) * 8
                                                           : ((j * 4 + g4) ^ swz8(row)) * 16);
    }
    // and of values, 32 columns by 16 rows: this lane's column from rows 4 half + 0 .. 3
    // and 8 + 4 half + 0 .. 3, as the scores' registers have them
    unsigned voff[2][E4M3 ? 1 : 2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int dg = g4 & 1;
        if constexpr (E4M3) {
            const int k = l15 >> 1, row = (k >> 2) * 8 + 4 * half + (k & 3);
            voff[j][0] = (unsigned)(row * ROWB + (((j * 2 + dg) ^ swz4(row)) * 16) + (l15 & 1) * 8 + cs * DB * 32);
        } else {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int row = 8 * y + 4 * half + (l15 >> 2);
                voff[j][y] = (unsigned)(row * ROWB + (((j * 4 + dg * 2 + ((l15 & 3) >> 1)) ^ swz8(row)) * 16) + (l15 & 1) * 8 + cs * DB * 64);
            }
        }
    }
    // Weights of 16 cache rows by 16 rows, four of a row a lane: into a row's 32 in the
    // order in which the second product's lanes take eight of them, the row's four
    // 16-byte pieces permuted.  Scores likewise, in the order of the cache rows.
    const unsigned put_at = (unsigned)((rg * 32 + own_row) * 64 + (((step_half * 2 + (g4 & 1)) ^ ((own_row >> 2) & 3)) * 16) + (g4 >> 1) * 8);
    const unsigned get_at = (unsigned)((rg * 32 + l31) * 64 + ((half ^ ((l31 >> 2) & 3)) * 16));
    const unsigned ring = (unsigned)uniform((int)lds_address(lds_raw + wave * WR * ROWB));
    const float kv_scale = E4M3 ? a.scale[0] : 1.0f;
    const float factor = a.factor * kv_scale;
    // Both are numbers of fp32, their product may be none: then one after the other, so that
    // a score of 0 is 0 and one that fits is there.
    bool in_two = false;
    if constexpr (E4M3) in_two = !(__builtin_fabsf(factor) < __builtin_inff());

    // ---- row tiles of the share, one after another
    while (left > 0) {
        const int steps = tile_steps(before, q.n, s.tp, i);
        const int units = uniform((int)min((long)(steps + s.anew - unit), left));
        const int at = max(unit - s.anew, 0), n = max(unit + units - s.anew, 0) - at;  // this workgroup's steps of it
        if (n == 0) break;  // the share ends in front of them
        const int lim0 = max(before + j0 + 1, 0);                  // rows that it sees
        const int most = max(before + min(j0 + s.tp, q.n), 0);     // and the last one
        // how many cache rows the rows whose weights this lane makes see
        int lim[QR];
#pragma unroll
        for (int x = 0; x < QR; ++x) {
            int tok, head;
            lim[x] = place(rg * 32 + own_row + 16 * x, tok, head) ? max(before + tok + 1, 0) : 0;
        }

        // Where this wave's rows of 64 steps lie in the cache, and how many bytes of them
        // there are, one step a lane; of 16 steps in fours where a step may have several
        // pages.  held: whose page is one of the cache's, a bit a lane.
        int first = 0;
        const unsigned known = wide ? 64 : 16;  // steps
        unsigned place_lo = 0, place_hi = 0, place_bytes = 0;
        unsigned long long held = 0;
        auto fill = [&](int step, int page) {
            const int lane = here(threadIdx.x & 63);
            first = step;
            const long row = (long)step * kTile + lane * (wide ? kTile : 8);
            wait_vmcnt_lds<0>();
            const bool ok = (unsigned)page < (unsigned)a.pages;
            held = __ballot(ok);
            const int in_step = wide ? WR * wave : WR * wave & 7;
            const size_t at_row = ((size_t)(ok ? page : 0) << a.page_shift) + (size_t)(row & ((1 << a.page_shift) - 1)) + in_step;
            const size_t p = (size_t)(uintptr_t)a.cache + at_row * ROWB;
            place_lo = (unsigned)p;
            place_hi = (unsigned)(p >> 32);
            place_bytes = ok ? (unsigned)(min(max((long)most - (row + in_step), 0L), (long)WR) * ROWB) : 0u;
        };
        // Its wait is for the queries as well: the compiler then waits for no load inside the
        // loop over the ring.
        fill(at, page);
        // The sums take 128 of the 256 registers that vector instructions reach; the queries,
        // which only the matrix instruction reads, go to the others.
        if constexpr (QR == 2) {
#pragma unroll
            for (int x = 0; x < QR; ++x)
#pragma unroll
                for (int k = 0; k < 18; ++k) asm volatile("" : "+a"(qf[x][k]));
        }

        f32x16 acc[DB];
        float m, l;  // of row l31
        bool careful = false;
        for (;;) {
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[d][r] = 0.0f;
            m = -__builtin_inff();
            l = 0.0f;
            float own_ref[QR], own_most[QR];  // of this lane's rows: m, or 0 where there is none; m + 8
            f32x4 last[QR];                   // and scores of the step to come
#pragma unroll
            for (int x = 0; x < QR; ++x) {
                own_ref[x] = 0.0f;
                own_most[x] = -__builtin_inff();
            }

            unsigned seen = 0;  // four bits a step, the newest lowest: groups of 8 rows whose page is one
            // Step `step` to ring slot `slot`: the table's entries, where the rows are, and then the
            // loads, number k of LOADS each.  Behind the last step no row is there, and the
            // loads bring zeros.
            Rsrc rs;
            unsigned dst;
            auto look_up = [&](int step) {
                if (__builtin_expect((unsigned)(step - first) >= known, 0)) fill(step, table_entry(step));
            };
            auto locate = [&](int step, int slot) {
                const int i0 = (step - first) * (wide ? 1 : 4), own = i0 + (wide ? 0 : WR * wave >> 3);
                const unsigned bits = (unsigned)(held >> i0) & (wide ? 1u : 15u);
                seen = seen << 4 | (wide ? bits * 15u : bits);
                const size_t p = (size_t)(unsigned)__builtin_amdgcn_readlane((int)place_hi, own) << 32 | (unsigned)__builtin_amdgcn_readlane((int)place_lo, own);
                rs = make_rsrc(reinterpret_cast<const void *>(p), (unsigned)__builtin_amdgcn_readlane((int)place_bytes, own));
                dst = ring + slot * TILE;
            };
            auto load = [&](auto number) {
                constexpr int k = decltype(number)::value;
                if constexpr (k < LOADS) {
                    if ((k + 1) * 64 <= WR * PIECES || lane < WR * PIECES - k * 64) ring_load16<k * 1024>(rs, dst, src[k]);
                }
            };
            auto read_keys = [&](const unsigned char *tile, int c, Key(&x)[2]) {
#pragma unroll
                for (int e = 0; e < 2; ++e) x[e] = *reinterpret_cast<const Key *>(tile + koff[e] + c * (E4M3 ? 64 : 128));
            };
            auto read_values = [&](const unsigned char *tile, int d, Value(&x)[2]) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const unsigned char *v = tile + e * 16 * ROWB + (d >> 1) * (E4M3 ? 64 : 128);
                    if constexpr (E4M3) x[e] = lds_transposed8(v + voff[d & 1][0]);
                    else x[e] = __builtin_shufflevector(lds_transposed4(v + voff[d & 1][0]), lds_transposed4(v + voff[d & 1][1]), 0, 1, 2, 3, 4, 5, 6, 7);
                }
            };
            // Ninth c of the scores of a step, 16 by 16 QR a wave; the keys are read ahead.
            f32x4 y[QR][YN];
            Key kf[KD][2];
            auto score = [&](const unsigned char *next, int c) {
                if (c + KD - 1 < 9) read_keys(next, c + KD - 1, kf[(c + KD - 1) % KD]);
                arrived(kf[c % KD]);
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int x = 0; x < QR; ++x)
                        y[x][e % YN] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(kf[c % KD][e]), qf[x][2 * c + e], y[x][e % YN], 0, 0, 0);
            };
            auto first_keys = [&](const unsigned char *next) {
#pragma unroll
                for (int x = 0; x < QR; ++x) y[x][0] = y[x][YN - 1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < KD - 1; ++c) read_keys(next, c, kf[c]);
            };
            // Columns 32 d .. + 31 of the wave's part: their sums of a step.
            bf16x8 pf[2];
            Value vf[VD][2];
            auto sum = [&](int d) {
                arrived(vf[d % VD]);
#pragma unroll
                for (int e = 0; e < 2; ++e) acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16(vf[d % VD][e]), pf[e], acc[d], 0, 0, 0);
            };
            // The scores' weights to where all waves read them, in three parts.  Behind the
            // last step the scores are those of zeros, and unused.
            auto scaled = [&](int row0, unsigned bits) {
#pragma unroll
                for (int x = 0; x < QR; ++x) last[x] = (y[x][0] + y[x][1]) * factor;
                bool rare = row0 + kTile > lim0 || bits != 15u;
                if constexpr (E4M3) rare |= in_two;
                if (__builtin_expect(rare, 0)) {
                    if constexpr (E4M3) {
                        if (in_two) {
#pragma unroll
                            for (int x = 0; x < QR; ++x) last[x] = (y[x][0] + y[x][1]) * kv_scale * a.factor;
                        }
                    }
                    const bool held = bits >> (step_half * 2 + (g4 >> 1)) & 1u;
#pragma unroll
                    for (int x = 0; x < QR; ++x)
#pragma unroll
                        for (int r = 0; r < 4; ++r) last[x][r] = held && row0 + step_half * 16 + g4 * 4 + r < lim[x] ? last[x][r] : -__builtin_inff();
                }
            };
            auto warn = [&](int parity, unsigned number) {
                bool over = false;
#pragma unroll
                for (int x = 0; x < QR; ++x) over |= fmaxf(fmaxf(last[x][0], last[x][1]), fmaxf(last[x][2], last[x][3])) > own_most[x];
                if (__builtin_expect(__any(over), 0)) {
                    if (lane == 0) flags[parity] = number;
                }
            };
            auto weigh = [&](int parity) {
#pragma unroll
                for (int x = 0; x < QR; ++x) {
                    float w[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) w[r] = __builtin_amdgcn_exp2f(last[x][r] - own_ref[x]);
                    *reinterpret_cast<uint2 *>(exchange + parity * RG * kWeights * 2 + put_at + x * 16 * 64) = to_bf16x4(w[0], w[1], w[2], w[3]);
                }
            };

#pragma unroll
            for (int k = 0; k < kRing - 1; ++k) {
                look_up(at + k);
                locate(at + k, k);
                each<LOADS>(load);
            }
            wait_vmcnt_lds<2 * LOADS>();
            barrier_nofence();
            ++epoch;
            first_keys(lds_raw);
#pragma unroll
            for (int c = 0; c < 9; ++c) score(lds_raw, c);
            scaled(at * kTile, seen >> 8 & 15u);
            warn(0, epoch);
            weigh(0);
            int slot = 0;
            for (int k = 0; k < n; ++k) {
                // the next step's rows are there when the one behind it may be under way
                wait_vmcnt_lds<LOADS>();
                barrier_nofence();
                // weights of column l31, the lane's (token, head), in the second product's order
                const unsigned flag = flags[k & 1];
#pragma unroll
                for (int v = 0; v < 2; ++v) pf[v] = *reinterpret_cast<const bf16x8 *>(exchange + (k & 1) * RG * kWeights * 2 + (get_at ^ (v * 32)));
                const unsigned bits = seen >> 8 & 15u, next_bits = seen >> 4 & 15u;
                const unsigned char *tile = lds_raw + slot * TILE;
                const int free_slot = (slot + kRing - 1) & (kRing - 1);  // every wave is done with the step before
                slot = (slot + 1) & (kRing - 1);
                const unsigned char *next = lds_raw + slot * TILE;
                const int row0 = (at + k) * kTile;
                look_up(at + k + kRing - 1);
                first_keys(next);
                score(next, 0);
                locate(at + k + kRing - 1, free_slot);
                each<3>([&](auto c) {
                    load(c);
                    score(next, c + 1);
                });
                if (__builtin_expect((unsigned)uniform((int)flag) == epoch, 0)) {
                    // a maximum has grown: new weights of all scores, old sums multiplied
                    __syncthreads();
                    const int lane = here(threadIdx.x & 63), half = lane >> 5, l31 = lane & 31, l15 = lane & 15, g4 = lane >> 4;
                    const int own_row = (CS == 4 ? (cs >> 1) * 16 : 0) + l15;
                    float *all = reinterpret_cast<float *>(exchange);
#pragma unroll
                    for (int x = 0; x < QR; ++x)
                        *reinterpret_cast<f32x4 *>(all + (rg * 32 + own_row + 16 * x) * 32 + (((step_half * 4 + g4) ^ (own_row & 7)) * 4)) = last[x];
                    __syncthreads();
                    float z[16];
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        *reinterpret_cast<f32x4 *>(z + 4 * v) = *reinterpret_cast<const f32x4 *>(all + (rg * 32 + l31) * 32 + ((2 * v + half) ^ (l31 & 7)) * 4);
                    float top = z[0];
#pragma unroll
                    for (int r = 1; r < 16; ++r) top = fmaxf(top, z[r]);
                    top = fmaxf(m, other_half_max(top));
                    const float down = top == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(m - top);
                    const float ref = top == -__builtin_inff() ? 0.0f : top;
                    m = top;
                    l *= down;
#pragma unroll
                    for (int d = 0; d < DB; ++d)
#pragma unroll
                        for (int r = 0; r < 16; ++r) acc[d][r] *= down;
#pragma unroll
                    for (int r = 0; r < 16; ++r) z[r] = __builtin_amdgcn_exp2f(z[r] - ref);
                    pf[0] = to_bf16x8(z);
                    pf[1] = to_bf16x8(z + 8);
#pragma unroll
                    for (int x = 0; x < QR; ++x) {
                        own_ref[x] = __shfl(ref, own_row + 16 * x, 64);
                        own_most[x] = __shfl(m, own_row + 16 * x, 64) + 8.0f;
                    }
                    __syncthreads();
                }
                ++epoch;
                const bool masked = row0 + kTile > lim0 || bits != 15u;
                if (__builtin_expect(careful && masked, 0)) {
                    // Rows with infinities or NaN that some of the tile's tokens see and some do
                    // not: their products by vector instructions for those that do, and zeros
                    // in their place for the matrix instruction.
                    __syncthreads();
                    const int t = here(threadIdx.x), lane = t & 63, half = lane >> 5, l31 = lane & 31;
                    unsigned char *bad_rows = reinterpret_cast<unsigned char *>(flags + 4);
                    bool bad = false;
                    for (int e = 0; e < ROWB * 512 / 576 / 8 / 4; ++e) {
                        const unsigned w = *reinterpret_cast<const unsigned *>(
                            tile + ((wave & 3) * 8 + (lane >> 3)) * ROWB + (lane & 7) * (ROWB * 512 / 576 / 8) + e * 4);
                        if constexpr (E4M3) {
                            const unsigned u = w & 0x7F7F7F7Fu;
                            bad |= ((u + 0x01010101u) & 0x80808080u) != 0;
                        } else {
                            bad |= (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
                        }
                    }
                    const unsigned long long any = __ballot(bad);
                    unsigned rows8 = 0;
#pragma unroll
                    for (int r = 0; r < 8; ++r) rows8 |= ((any >> (8 * r)) & 0xFFull ? 1u : 0u) << r;
                    if (lane == 0) bad_rows[wave & 3] = (unsigned char)rows8;  // each four waves the same
                    __syncthreads();
                    const unsigned flagged = (unsigned)uniform((int)flags[4]);
                    const int col_lim = [&] {
                        int tok, head;
                        return place(rg * 32 + l31, tok, head) ? max(before + tok + 1, 0) : 0;
                    }();
                    for (unsigned f = flagged; f; f &= f - 1) {
                        const int e = __builtin_ctz(f), r = (e >> 3) * 4 + (e & 3), eh = (e >> 2) & 1;
                        float own = 0.0f;
#pragma unroll
                        for (int u = 0; u < 16; ++u) own = u == r ? (float)pf[u >> 3][u & 7] : own;
                        const float w = __shfl(own, l31 + 32 * eh, 64);
                        const bool sees = row0 + e < col_lim && (bits >> (e >> 3) & 1u);
#pragma unroll
                        for (int d = 0; d < DB; ++d)
#pragma unroll
                            for (int v = 0; v < 4; ++v) {
                                const int col = (cs * DB + d) * 32 + 8 * v + 4 * half;
                                float y[4];
                                if constexpr (E4M3) {
                                    const int c = col >> 4;
                                    const unsigned x = *reinterpret_cast<const unsigned *>(
                                        tile + e * ROWB + ((c & ~3) | ((c & 3) ^ swz4(e))) * 16 + (col & 15));
                                    const bf16x8 c8 = e4m3_to_bf16(i32x2{(int)x, 0});
#pragma unroll
                                    for (int u = 0; u < 4; ++u) y[u] = (float)c8[u];
                                } else {
                                    const int c = col >> 3;
                                    const uint2 x = *reinterpret_cast<const uint2 *>(
                                        tile + e * ROWB + ((c & ~7) | ((c & 7) ^ swz8(e))) * 16 + (col & 7) * 2);
                                    y[0] = bf16_lo(x.x);
                                    y[1] = bf16_hi(x.x);
                                    y[2] = bf16_lo(x.y);
                                    y[3] = bf16_hi(x.y);
                                }
#pragma unroll
                                for (int u = 0; u < 4; ++u)
                                    if (sees) acc[d][4 * v + u] = __builtin_fmaf(w, y[u], acc[d][4 * v + u]);
                                __builtin_amdgcn_sched_barrier(0);  // one after another: rare, and short of registers
                            }
                    }
                    __syncthreads();
                    for (unsigned f = flagged; f; f &= f - 1)
                        for (int e = t; e < ROWB * 512 / 576 / 4; e += 64 * NW)
                            *reinterpret_cast<unsigned *>(const_cast<unsigned char *>(tile) + __builtin_ctz(f) * ROWB + e * 4) = 0;
                    __syncthreads();
                }
                each<5>([&](auto e) {
                    constexpr int c = decltype(e)::value + 4;
                    load(std::integral_constant<int, c - 1>{});
                    if (c >= 10 - VD) read_values(tile, c - (10 - VD), vf[c >= 10 - VD ? c - (10 - VD) : 0]);
                    score(next, c);
                });
                load(std::integral_constant<int, 8>{});
#pragma unroll
                for (int d = 0; d < DB; ++d) {
                    if (d + VD - 1 < DB) read_values(tile, d + VD - 1, vf[(d + VD - 1) % VD]);
                    sum(d);
                    if (d == 0) scaled(row0 + kTile, next_bits);
                    if (d == 1) warn((k + 1) & 1, epoch);
                    if (d == 2) weigh((k + 1) & 1);
                    if (d == 2) l = add_bf16x8(pf[1], add_bf16x8(pf[0], l));
                }
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
            const unsigned long long found = __ballot(bad);
            if (lane == 0) flags[8 + wave] = found != 0;
            __syncthreads();
            unsigned some = 0;
#pragma unroll
            for (int w = 0; w < NW; ++w) some |= flags[8 + w];
            __syncthreads();
            if (!uniform((int)some)) break;
            careful = true;
            fill(at, table_entry(at));
        }
        l = other_half_sum(l);

        if (at == 0 && n == steps) {
            const Quotient by(kv_scale, l);
            const int lane = here(threadIdx.x & 63), half = lane >> 5, l31 = lane & 31;
            int tok, head;
            if (place(rg * 32 + l31, tok, head)) {
                uint16_t *o = a.out + ((size_t)(q.first + tok) * a.H + head) * SKG_LATENT + cs * DB * 32 + 4 * half;
#pragma unroll
                for (int d = 0; d < DB; ++d)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        *reinterpret_cast<uint2 *>(o + d * 32 + 8 * v) =
                            to_bf16x4(by.of(acc[d][4 * v]), by.of(acc[d][4 * v + 1]), by.of(acc[d][4 * v + 2]), by.of(acc[d][4 * v + 3]));
            }
        } else {
            // a part: the sums in the registers' order, then maxima and sums of weights
            const int lane = here(threadIdx.x & 63), half = lane >> 5, l31 = lane & 31;
            float *part = a.ws + (2 * (size_t)group + (at == 0 ? 1 : 0)) * part_floats<RG>();
            int tok, head;
            if (place(rg * 32 + l31, tok, head)) {  // rows of no token or head are not handed on
#pragma unroll
                for (int d = 0; d < DB; ++d)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        *reinterpret_cast<f32x4 *>(part + (((rg * 16 + cs * DB + d) * 4 + v) * 64 + lane) * 4) =
                            f32x4{acc[d][4 * v], acc[d][4 * v + 1], acc[d][4 * v + 2], acc[d][4 * v + 3]};
                if (cs == 0 && half == 0) *reinterpret_cast<f32x2 *>(part + R * SKG_LATENT + (rg * 32 + l31) * 2) = f32x2{m, l};
            }
            if (at == 0) mine = Shared{b, i, group, 1 + (int)((steps - n + share - 1) / share)};
        }
        if (s.by_tile && at == 0 && t == 0)
            records[b * s.hg + g] = n == steps ? Shared{b, i, group, 1} : mine;

        left -= units;
        unit = 0;
        if (left > 0 && ++i * s.tp >= q.n) {
            i = 0;
            do {
                ++b;
                q = uniform(new_tokens(a.q_starts, b, a.T));
            } while (q.n == 0);  // steps are left, so there is one
            before = uniform(length(b)) - q.n;
        }
        if (left > 0) {
            j0 = i * s.tp;
            load_queries();
            page = table_entry(0);
        }
    }
    if (!s.by_tile && t == 0) records[group] = mine;
}

// Row tiles that several workgroups shared.  One workgroup for a record and 32
// columns.  Up to four parts: a wave joins 8 of the columns in the order of the steps.
// More: a wave adds up every fourth part, then the waves' sums are added in their order.
template <int RG>
__global__ void __launch_bounds__(256) latent_combine_kernel(Shape s, const float *scale, int G) {
    constexpr int R = 32 * RG;
    __shared__ f32x4 sums[4][4][64];
    __shared__ f32x2 stats[4][64];
    const LatentArgs &a = s.a;
    const int d = blockIdx.x;  // neighbouring workgroups lie on different XCDs: those of one record on all of them
    const Shared e = reinterpret_cast<const Shared *>(a.ws + 2 * (size_t)G * part_floats<RG>())[blockIdx.y];
    if (e.parts < 2) return;
    const int group = e.group, g = group % s.hg;
    const Tokens q = new_tokens(a.q_starts, e.b, a.T);
    const int t = threadIdx.x, wave = t >> 6, lane = t & 63, half = lane >> 5;
    const float kv_scale = scale ? scale[0] : 1.0f;
    auto part = [&](int p) { return a.ws + (2 * (size_t)(group + p * s.hg) + (p == 0 ? 1 : 0)) * part_floats<RG>(); };
    auto columns = [&](int rg, int v) { return (((rg * 16 + d) * 4 + v) * 64 + lane) * 4; };
    // (token, head) of a row of the tile
    auto place = [&](int r, int &tok, int &head) {
        tok = e.i * s.tp;
        head = g * R + r;
        if (a.H > R) return head < a.H;
        const int x = r / a.H;
        head = r - x * a.H;
        const bool ok = x < s.tp && tok + x < q.n;
        tok += x;
        return ok;
    };
    auto store = [&](int tok, int head, f32x4 sum, float l) {
        const Quotient by(kv_scale, l);
        *reinterpret_cast<uint2 *>(a.out + ((size_t)(q.first + tok) * a.H + head) * SKG_LATENT + d * 32 + 8 * wave + 4 * half) =
            to_bf16x4(by.of(sum[0]), by.of(sum[1]), by.of(sum[2]), by.of(sum[3]));
    };
    constexpr int U = 4;  // parts whose loads are under way together
    if (e.parts <= U) {
        f32x2 ml[RG][U];
        f32x4 y[RG][U];
        int tok[RG], head[RG];
        bool live[RG];
#pragma unroll
        for (int rg = 0; rg < RG; ++rg) {
            const int r = rg * 32 + (lane & 31);
            live[rg] = place(r, tok[rg], head[rg]);
#pragma unroll
            for (int p = 0; p < U; ++p)
                if (p < e.parts && live[rg]) {
                    ml[rg][p] = *reinterpret_cast<const f32x2 *>(part(p) + R * SKG_LATENT + 2 * r);
                    y[rg][p] = *reinterpret_cast<const f32x4 *>(part(p) + columns(rg, wave));
                }
        }
#pragma unroll
        for (int rg = 0; rg < RG; ++rg) {
            if (!live[rg]) continue;
            float m = -__builtin_inff(), l = 0.0f;
            f32x4 sum[1] = {};
#pragma unroll
            for (int p = 0; p < U; ++p)
                if (p < e.parts) {
                    const f32x4 one[1] = {y[rg][p]};
                    add_part(m, l, sum, ml[rg][p], one);
                }
            store(tok[rg], head[rg], sum[0], l);
        }
        return;
    }
    for (int rg = 0; rg < RG; ++rg) {
        const int r = rg * 32 + (lane & 31);
        int tok, head;
        const bool live = place(r, tok, head);
        if (!__any(live)) continue;  // the same in every wave
        float m = -__builtin_inff(), l = 0.0f;
        f32x4 sum[4] = {};
        for (int p0 = live ? wave : e.parts; p0 < e.parts; p0 += 4 * U) {
            f32x2 ml[U];
            f32x4 y[U][4];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (p0 + 4 * u >= e.parts) break;
                const float *x = part(p0 + 4 * u);
                ml[u] = *reinterpret_cast<const f32x2 *>(x + R * SKG_LATENT + 2 * r);
#pragma unroll
                for (int v = 0; v < 4; ++v) y[u][v] = *reinterpret_cast<const f32x4 *>(x + columns(rg, v));
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (p0 + 4 * u >= e.parts) break;
                add_part(m, l, sum, ml[u], y[u]);
            }
        }
        stats[wave][lane] = f32x2{m, l};
#pragma unroll
        for (int v = 0; v < 4; ++v) sums[wave][v][lane] = sum[v];
        __syncthreads();
        // wave v joins the four waves' sums of its 4 columns a lane
        m = -__builtin_inff();
        l = 0.0f;
        f32x4 one[1] = {};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const f32x4 y[1] = {sums[w][wave][lane]};
            add_part(m, l, one, stats[w][lane], y);
        }
        __syncthreads();
        if (live) store(tok, head, one[0], l);
    }
}

namespace {

template <int RG, int CS, bool E4M3>
int go(const LatentArgs &a, hipStream_t stream) {
    constexpr int R = 32 * RG;
    constexpr int G = groups_of(RG, E4M3);
    Shape s{a, a.H > R ? 1 : R / a.H, a.H > R ? (a.H + R - 1) / R : 1, 0, E4M3 ? 4 : 6, E4M3 ? 8 : 12, 0};
    s.teams = G / s.hg;
    s.by_tile = !a.q_starts && (long)a.B * s.hg <= G;
    static std::atomic<unsigned long long> done{0};
    constexpr size_t lds = lds_bytes<RG, E4M3>();
    const hipError_t e = allow_dynamic_lds((const void *)latent_attention_kernel<RG, CS, E4M3>, lds, done);
    if (e != hipSuccess) return (int)e;
    hipLaunchKernelGGL((latent_attention_kernel<RG, CS, E4M3>), dim3(G), dim3(64 * RG * CS), lds, stream, s);
    const hipError_t f = hipGetLastError();
    if (f != hipSuccess) return (int)f;
    hipLaunchKernelGGL((latent_combine_kernel<RG>), dim3(16, s.by_tile ? a.B * s.hg : G), dim3(256), 0, stream, s, a.scale, G);
    return (int)hipGetLastError();
}

template <bool E4M3>
int by_rows(const LatentArgs &a, int rows, hipStream_t stream) {
    return rows == 32 ? go<1, 4, E4M3>(a, stream) : go<2, 2, E4M3>(a, stream);
}

}  // namespace

// 64 rows read the cache half as often and waste fewer rows where H does not divide 32,
// but fill the device with fewer tiles and hand on twice as much.  Measured, 32 against
// 64 (bf16, us): 512 tokens of 128 heads over 8192 rows 1095, 860; 150 tokens of 20 heads
// over 2000 to 9000 rows, 12 sequences, 130, 74; 128 tokens of 16 heads over 16000 rows
// 105, 92, 64 over 4000 31, 38; 100 tokens of 7 heads over 12000, 3 sequences, 37, 43; 4
// tokens of 128 heads over 6000, 4 sequences, 24, 35; 100 tokens of 128 heads over 200 34,
// 27 (more tiles of 32 rows than workgroups).  The same in e4m3, which has twice the
// workgroups for 32 rows: 1009, 920; 101, 76; 105, 100 and 37, 41; 42, 45; 31, 40; 29, 28.
// What a table lets sequences be they seldom are, and then 64 rows cost most where the
// tiles are few: 128 heads (bf16), 32 tokens of sequences of 4000 rows 51, 48, of 24000
// 208, 172; 16 heads, 64 tokens of 2 sequences of 2000 25, 35, of 24000 75, 67; 128 heads, 4 of 6000
// 25, 35, of 100000 92, 85.  So below 32 tiles the table's width does not count.
int latent_rows(int B, int T, int H, long capacity, bool e4m3) {
    auto tiles = [&](int rows) {  // of the call if its tokens are spread evenly
        const long tp = H > rows ? 1 : rows / H, hg = H > rows ? (H + rows - 1) / rows : 1;
        return B * ((((long)T + B - 1) / B + tp - 1) / tp) * hg;
    };
    const long few = tiles(64), many = tiles(32);
    if (few == many) return 32;
    // steps of one of 256 workgroups if all sequences are as long as the table lets them be
    const double share = (double)few * capacity / kTile / 256;
    return few >= 256 || (many > 2 * few && share >= 20) || (few >= 32 && share >= 48) || (!e4m3 && many > 256) ? 64 : 32;
}

size_t latent_workspace_bytes(int rows, bool e4m3) {
    const size_t groups = groups_of(rows / 32, e4m3);
    return groups * (2 * rows * (SKG_LATENT + 2) * 4 + sizeof(Shared));
}

int launch_latent_attention(const LatentArgs &a, bool e4m3, int rows, hipStream_t stream) {
    return e4m3 ? by_rows<true>(a, rows, stream) : by_rows<false>(a, rows, stream);
}

}  // namespace skg
