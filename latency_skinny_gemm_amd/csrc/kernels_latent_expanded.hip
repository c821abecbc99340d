// kernels_latent_expanded.hip -- attention of prompts over expanded keys and
// values: a head's key is 128 values of its own and 64 that all heads share.
//
// A workgroup takes 128 query tokens of one head, a wave 32 of them; steps of 32
// keys and values come to an LDS ring by direct loads.  Scores are made
// transposed, so that a lane has eight keys of one token in the registers in which
// the second product takes its weights.  A step's weights are made between the next
// one's scores, so that vector and matrix instructions run beside each other; weights
// are 2^(score - m), m a maximum that follows only when a score is over m + 8.
//
// 4096 tokens, 128 heads: 722 us, 950 TFLOP/s, at 1.9 GHz of 2.4.  The matrix pipes are busy
// 46 % of the cycles; a SIMD's two waves each issue instructions in 36 % of them, wait for
// counters and barriers in 26 % and for a unit to take the next instruction in 37 %.  Waves
// of 64 tokens, one a SIMD, which read LDS half as often, took 784 us for 723; blocks of 16
// rows by 64 bytes in LDS, loaded 64 bytes a row, 811.
//
// Query tokens that fill less than half of the device have their keys shared among
// workgroups, two a CU in all; a second kernel joins the parts (500 tokens of 32 heads
// over 8100 keys: 155 us in one part, 89 + 8 in four).
#include <algorithm>

#include "internal.h"
#include "latent_common.h"
#include "latent_internal.h"
#include "lds_limit.h"

namespace skg {

namespace {

#define INLINE __attribute__((always_inline))

constexpr int kRows = 128;              // query tokens a workgroup
constexpr int kStep = 32, kSlots = 3;   // keys a step, steps in LDS
constexpr int kGroups = 512;            // workgroups that the device holds: two a CU
constexpr int kKvRow = 2 * (SKG_EXPANDED_NOPE + SKG_EXPANDED_V);  // bytes
constexpr int kOwnRow = 2 * SKG_EXPANDED_NOPE, kRopeRow = 2 * SKG_LATENT_ROPE;
// A step in LDS: blocks of 1 KB, each one direct load, keys' and shared parts' with a gap.
constexpr int kOwnBlock = 1024 + 16, kSharedBlock = 1024 + 32;
constexpr int kShared = 8 * kOwnBlock, kKeyBytes = kShared + 4 * kSharedBlock, kValueBytes = 8 * 1024;
constexpr int kLoads = 5;  // a wave's direct loads a step: 8 keys, their shared parts, 8 values
constexpr int kFlags = kSlots * (kKeyBytes + kValueBytes);
constexpr size_t kExpandedLds = std::max<size_t>(kFlags + 64, (SKG_LATENT_MAX_B + 1) * 8 + 64);
// A part's least number of steps: 100 tokens of 16 heads over 4000 keys 33, 24, 25 us with
// 4, 8 and 16 (82 in one part), over 1000 18, 18 and 27.
constexpr int kLeast = 8;
constexpr int kAhead = 5;                                        // fragments of keys under way
constexpr size_t kPart = (size_t)kRows * (SKG_EXPANDED_V + 2);   // floats of a part: sums, maxima, sums of weights
constexpr int kQuery = SKG_EXPANDED_NOPE + SKG_LATENT_ROPE;

// Tile n of 128 query tokens: its sequence's tokens and keys, and its place there.
struct Place {
    Tokens q, kv;
    int i;
    bool there;
};
__device__ __forceinline__ Place place_of(const ExpandedArgs &a, int n, unsigned char *lds) {
    if (a.B <= 64) {  // a sequence a lane, every wave for itself: one round of loads, no barrier
        const int lane = threadIdx.x & 63, b = min(lane, a.B - 1);
        const Tokens q = new_tokens(a.q_starts, b, a.T), kv = new_tokens(a.kv_starts, b, a.S);
        const int tiles = lane < a.B ? (q.n + kRows - 1) / kRows : 0;
        int upto = tiles;
        for (int d = 1; d < a.B; d <<= 1) {
            const int u = __shfl_up(upto, d, 64);
            if (lane >= d) upto += u;
        }
        const unsigned long long behind = __ballot(upto > n);
        if (!behind) return {{0, 0}, {0, 0}, 0, false};
        const int at = __builtin_ctzll(behind);
        auto of = [&](int v) INLINE { return __builtin_amdgcn_readlane(v, at); };
        return {{of(q.first), of(q.n)}, {of(kv.first), of(kv.n)}, n - of(upto - tiles), true};
    }
    long *pre = reinterpret_cast<long *>(lds);
    block_prefix<4>(a.B, pre, pre + a.B + 1, [&](int s) INLINE { return (long)((new_tokens(a.q_starts, s, a.T).n + kRows - 1) / kRows); });
    if (n >= pre[a.B]) return {{0, 0}, {0, 0}, 0, false};
    const int b = uniform(find_sequence(pre, a.B, n)), i = uniform(n - (int)pre[b]);
    __syncthreads();
    return {uniform(new_tokens(a.q_starts, b, a.T)), uniform(new_tokens(a.kv_starts, b, a.S)), i, true};
}
// Keys that token j of a place's sequence sees.
__device__ __forceinline__ int keys_of(const ExpandedArgs &a, const Place &p, int j) {
    return max(a.causal ? p.kv.n - p.q.n + j + 1 : p.kv.n, 0);
}
// The parts of a tile whose last token sees `most` keys.
__device__ __forceinline__ int parts_of(const ExpandedArgs &a, int most) { return max(1, min(a.parts, most / (kStep * kLeast))); }

}  // namespace

__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2))) latent_expanded_kernel(ExpandedArgs a, int tiles) {
    extern __shared__ __attribute__((aligned(16))) unsigned char lds_raw[];
    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    // a head's tiles lie on one XCD, those with the most keys first; with parts, all tiles of
    // a part beside each other, since they read the same keys
    const unsigned total = (unsigned)tiles * (unsigned)a.H * (unsigned)a.parts, per = (total + 7) / 8;
    const unsigned id = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if ((blockIdx.x >> 3) >= per || id >= total) return;
    const int n = tiles - 1 - (int)(id % (unsigned)tiles), h = (int)(id / (unsigned)(tiles * a.parts));
    const int part = (int)(id / (unsigned)tiles) - h * a.parts;
    const Place at_tile = place_of(a, n, lds_raw);
    if (!at_tile.there) return;
    const Tokens q = at_tile.q, kv = at_tile.kv;
    const int i = at_tile.i;
    auto sees = [&](int j) INLINE { return keys_of(a, at_tile, j); };
    const int half = lane >> 5, l15 = lane & 15, l31 = lane & 31, g4 = lane >> 4;
    const int j = i * kRows + wave * 32 + l31;
    const int lim = j < q.n ? sees(j) : 0;
    const int lim0 = sees(i * kRows + wave * 32);  // of the wave's first token
    const int wave_most = i * kRows + wave * 32 < q.n ? sees(min(i * kRows + wave * 32 + 32, q.n) - 1) : 0;  // and its last
    const int most = sees(min(i * kRows + kRows, q.n) - 1);
    // this part's steps
    const int parts = parts_of(a, most);
    if (part >= parts) return;
    const int steps = (most + kStep - 1) / kStep;
    const int first = (int)((long)steps * part / parts), end = (int)((long)steps * (part + 1) / parts);

    // A block holds four rows of 16 pieces of 16 bytes (a head's keys, its values), or eight
    // of 8 (shared parts): four pieces of each row, then the next four.  Four lanes load 64
    // bytes of a row, and a fragment's address is one register and a constant.  A fragment
    // read takes one piece of 16 rows at once, 64 bytes apart in a block: the gaps shift
    // four blocks of keys, and an exchange of neighbouring pieces in every other four
    // shared rows two times two, to different banks of LDS's 64.  A transposed read takes
    // 256 bytes in a row.
    const unsigned row_bytes = (unsigned)a.H * kKvRow, rope_bytes = (unsigned)a.rope_stride * 2;
    unsigned src[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) src[k] = (unsigned)(k * 4 + ((lane >> 2) & 3)) * row_bytes + (unsigned)(g4 * 64 + (lane & 3) * 16);
    const unsigned rope_src = (unsigned)((lane >> 2) & 7) * rope_bytes + (unsigned)(half * 64 + ((lane & 3) ^ ((lane >> 4) & 1)) * 16);
    const int key_at = (l31 >> 2) * kOwnBlock + (l31 & 3) * 64 + half * 16;
    const int shared_at = kShared + (l31 >> 3) * kSharedBlock + (l31 & 7) * 64 + (half ^ ((l31 >> 2) & 1)) * 16;
    const int value_at = half * 1024 + (l15 >> 2) * 64 + (g4 & 1) * 32 + (l15 & 3) * 8;
    const unsigned ring = uniform((int)lds_address(lds_raw));
    // a step's keys, and the values of the step before; steps are brought in order
    struct Next {
        const uint16_t *own, *shared;  // this wave's rows
        int row;
        unsigned value_bytes;
    };
    auto rewind = [&]() INLINE {
        const int row = first * kStep + wave * 8;
        const size_t at = (size_t)kv.first + row;
        return Next{a.kv + (at * a.H + h) * (kKvRow / 2), a.k_rope + at * a.rope_stride, row, 0u};
    };
    struct Loads {
        Rsrc own, shared, values;
        unsigned key_at, value_at;
    };
    auto loads = [&](Next &n, int key_slot, int value_slot) INLINE {
        const int rows = min(uniform(most - n.row), 8);
        const unsigned bytes = rows > 0 ? (unsigned)(rows - 1) * row_bytes + kOwnRow : 0u;
        const unsigned shared = rows > 0 ? (unsigned)(rows - 1) * rope_bytes + kRopeRow : 0u;
        const Loads x{make_rsrc(n.own, bytes), make_rsrc(n.shared, shared),
                      make_rsrc(n.own - (size_t)(kStep / 2) * row_bytes + SKG_EXPANDED_NOPE, n.value_bytes),
                      ring + key_slot * kKeyBytes, ring + value_slot * kValueBytes};
        n.own += (size_t)(kStep / 2) * row_bytes;
        n.shared += (size_t)kStep * a.rope_stride;
        n.row += kStep;
        n.value_bytes = bytes;
        return x;
    };
    auto load = [&](const Loads &x, auto part) INLINE {
        constexpr int k = decltype(part)::value;
        if constexpr (k < 2) ring_load16<k * kOwnBlock>(x.own, x.key_at + wave * 2 * kOwnBlock, src[k]);
        else if constexpr (k == 2) ring_load16<kShared>(x.shared, x.key_at + wave * kSharedBlock, rope_src);
        else ring_load16<kSlots * kKeyBytes + (k - 3) * 1024>(x.values, x.value_at + wave * 2048, src[k - 3]);
    };

    // the first steps, and under way with them the queries
    Next next;
    auto bring = [&]() INLINE {
        next = rewind();
        each<3>([&](auto k) INLINE {
            const Loads x = loads(next, k, (k + 2) % kSlots);
            each<kLoads>([&](auto p) INLINE { load(x, p); });
        });
    };
    if (steps > 0) bring();
    bf16x8 qf[12];
    {
        const uint16_t *p = a.q + ((size_t)(q.first + (j < q.n ? j : 0)) * a.H + h) * kQuery + half * 8;
#pragma unroll
        for (int k = 0; k < 12; ++k) {
            u32x4 v{0, 0, 0, 0};
            if (j < q.n) v = *reinterpret_cast<const u32x4 *>(p + k * 16);
            qf[k] = __builtin_bit_cast(bf16x8, v);
        }
    }
    wait_vmcnt_lds<0>();  // here, so that the compiler waits for no load inside the loop over the ring

    unsigned char *flags = lds_raw + kFlags;
    f32x16 acc[4], z;
    float m, ref, l, top, x[16];  // ref: m, 0 for -inf; top: z's maximum; x: scores over m, logarithms of weights
    bf16x8 pf[2];
    auto nothing = [&]() INLINE {
#pragma unroll
        for (int d = 0; d < 4; ++d)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[d][r] = 0.0f;
        m = -__builtin_inff();
        ref = 0.0f;
        l = 0.0f;
    };
    auto read_key = [&](const unsigned char *keys, int c) INLINE {
        return *reinterpret_cast<const u32x4 *>(c < 8 ? keys + key_at + (c >> 1) * 256 + (c & 1) * 32 : keys + shared_at + ((c - 8) >> 1) * 512 + (c & 1) * 32);
    };
    auto read_values = [&](const unsigned char *values, int d, s16x8 (&v)[2]) INLINE {
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            const unsigned char *p = values + value_at + kSlots * kKeyBytes + kk * 4096 + d * 256;
            v[kk] = __builtin_shufflevector(lds_transposed4(p), lds_transposed4(p + 2048), 0, 1, 2, 3, 4, 5, 6, 7);
        }
    };
    auto weigh = [&](int c) INLINE {  // two of the weights, in the place where they are written
        bf16x2 w{(__bf16)__builtin_amdgcn_exp2f(x[2 * c]), (__bf16)__builtin_amdgcn_exp2f(x[2 * c + 1])};
        asm volatile("" : "+v"(w));
        pf[c >> 2][(c & 3) * 2] = w.x, pf[c >> 2][(c & 3) * 2 + 1] = w.y;
        l = __builtin_amdgcn_fdot2_f32_bf16(w, bf16x2{(__bf16)1.0f, (__bf16)1.0f}, l, false);
    };
    auto masked = [&](int row0) INLINE {
        if (row0 + kStep > lim0) {
            const int left = here(lim) - row0 - 4 * half;
#pragma unroll
            for (int r = 0; r < 16; ++r) z[r] = 8 * (r >> 2) + (r & 3) < left ? z[r] : -__builtin_inff();
        }
    };
    auto scaled = [&]() INLINE {
        top = other_half_max(top) * a.factor;
        if (__any(top > m + 8.0f)) {
            const float next = fmaxf(m, top);
            const float down = next == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(m - next);
            m = next;
            ref = next == -__builtin_inff() ? 0.0f : next;
            l *= down;
#pragma unroll
            for (int d = 0; d < 4; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[d][r] *= down;
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) x[r] = __builtin_fmaf(z[r], a.factor, -ref);
    };
    using Keys = u32x4[kAhead][1];
    using Values = s16x8[2][2];
    auto first_keys = [&](Keys &kf, const unsigned char *keys) INLINE {
#pragma unroll
        for (int c = 0; c < kAhead - 1; ++c) kf[c][0] = read_key(keys, c);
    };
    // the scores of a step, and between them what `beside` does
    auto scores = [&](Keys &kf, const unsigned char *keys, auto beside) INLINE {
#pragma unroll
        for (int r = 0; r < 16; ++r) z[r] = 0.0f;
        each<12>([&](auto c) INLINE {
            if constexpr (c + kAhead - 1 < 12) kf[(c + kAhead - 1) % kAhead][0] = read_key(keys, c + kAhead - 1);
            arrived(kf[c % kAhead]);
            z = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16(kf[c % kAhead][0]), qf[c], z, 0, 0, 0);
            beside(c);
        });
    };
    // this step's sums, and between them the maximum of the next one's scores
    auto sums = [&](const unsigned char *values, Values &vf) INLINE {
        top = -__builtin_inff();
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            if (d + 1 < 4) read_values(values, d + 1, vf[(d + 1) & 1]);
            arrived(vf[d & 1]);
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16(vf[d & 1][kk]), pf[kk], acc[d], 0, 0, 0);
#pragma unroll
                for (int r = 0; r < 2; ++r) top = fmaxf(top, z[d * 4 + kk * 2 + r]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    // keys whose values hold an infinity or NaN, in a step that some tokens do not see:
    // their products by vector instructions for those that do, zeros for the matrix
    // instruction
    auto apart = [&](unsigned char *values, int row0) INLINE {
        unsigned *const word = reinterpret_cast<unsigned *>(flags);
        if (t == 0) *word = 0;
        __syncthreads();
        for (int e = 0; e < 2; ++e) {
            const int block = e * 4 + wave;
            const u32x4 w = *reinterpret_cast<const u32x4 *>(values + block * 1024 + lane * 16);
            bool bad = false;
#pragma unroll
            for (int u = 0; u < 4; ++u) bad |= (w[u] & 0x7F80u) == 0x7F80u || (w[u] & 0x7F800000u) == 0x7F800000u;
            if (bad) atomicOr(word, 1u << (block * 4 + ((lane >> 2) & 3)));
        }
        __syncthreads();
        const unsigned flagged = __builtin_amdgcn_readfirstlane(*word);
        auto at = [&](int row, int c) INLINE { return values + (row >> 2) * 1024 + (c >> 2) * 256 + (row & 3) * 64 + (c & 3) * 16; };
        for (unsigned f = flagged; f; f &= f - 1) {
            const int r0 = __builtin_ctz(f), r = (r0 >> 3) * 4 + (r0 & 3), kh = (r0 >> 2) & 1;
            float own_p = 0.0f;
#pragma unroll
            for (int u = 0; u < 16; ++u) own_p = u == r ? (float)pf[u >> 3][u & 7] : own_p;
            const float pk = __shfl(own_p, l31 + 32 * kh, 64);
            const bool in = row0 + r0 < lim;
#pragma unroll
            for (int d = 0; d < 4; ++d)
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(at(r0, d * 4 + v) + half * 8);
                    const float y[4] = {bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)};
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        if (in) acc[d][4 * v + u] = __builtin_fmaf(pk, y[u], acc[d][4 * v + u]);
                }
        }
        __syncthreads();
        for (unsigned f = flagged; f; f &= f - 1)
            if (t < 64) *reinterpret_cast<unsigned *>(at(__builtin_ctz(f), t >> 2) + (t & 3) * 4) = 0;
        __syncthreads();
    };
    auto begin = [&]() INLINE {
        nothing();
        wait_vmcnt_lds<2 * kLoads>();
        barrier_nofence();
        Keys kf;
        first_keys(kf, lds_raw);
        scores(kf, lds_raw, [](auto) INLINE {});
        masked(first * kStep);
        top = z[0];
#pragma unroll
        for (int r = 1; r < 16; ++r) top = fmaxf(top, z[r]);
    };
    // step k, with its values in slot `at` and the next one's keys in the slot after
    auto step = [&](int k, int at, auto careful) INLINE {
        const int after = (at + 1) % kSlots, last = (at + 2) % kSlots;
        const Loads more = loads(next, at, last);
        wait_vmcnt_lds<kLoads>();
        barrier_nofence();
        const int row0 = k * kStep;
        unsigned char *const values = lds_raw + at * kValueBytes, *const keys = lds_raw + after * kKeyBytes;
        Keys kf;
        Values vf;
        const bool seen = row0 < wave_most;
        if (seen) {
            first_keys(kf, keys);
            __builtin_amdgcn_sched_barrier(0);
            scaled();
            scores(kf, keys, [&](auto c) INLINE {
                if constexpr (c < kLoads) load(more, c);
                if constexpr (c >= 2 && c < 10) weigh(c - 2);
                if constexpr (c == 11) read_values(values, 0, vf[0]);
            });
        } else {
            each<kLoads>([&](auto p) INLINE { load(more, p); });
        }
        if constexpr (decltype(careful)::value) {
            if (!seen) pf[0] = pf[1] = bf16x8{};
            if (row0 + kStep > sees(i * kRows)) {
                apart(values + kSlots * kKeyBytes, row0);
                read_values(values, 0, vf[0]);
            }
        }
        if (!seen) return;
        masked(row0 + kStep);
        sums(values, vf);
    };
    if (steps > 0) {
        begin();
        int k = first;
        for (; k + 3 <= end; k += 3) each<3>([&](auto slot) INLINE { step(k + slot, slot, std::false_type{}); });
        for (int slot = 0; k < end; ++k, ++slot) step(k, slot, std::false_type{});
        wait_vmcnt_lds<0>();
        __syncthreads();
        // see kernels_latent_attention.hip: infinities and NaN of keys that a token does not see
        if (sees(i * kRows) < min(most, end * kStep)) {
            bool bad = false;
#pragma unroll
            for (int d = 0; d < 4; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r) bad |= not_finite(acc[d][r]);
            const unsigned long long found = __ballot(bad && j < q.n);
            if (lane == 0) flags[wave] = found != 0;
            __syncthreads();
            const unsigned some = __builtin_amdgcn_readfirstlane(*reinterpret_cast<const unsigned *>(flags));
            __syncthreads();
            if (__builtin_expect(some, 0)) {
                bring();
                begin();
                for (int k = first; k < end; ++k) step(k, (k - first) % kSlots, std::true_type{});
                wait_vmcnt_lds<0>();
            }
        }
    } else {
        nothing();
    }
    l = other_half_sum(l);
    if (parts > 1) {
        // sums as they lie in the waves' registers, each wave's register beside the others'
        float *ws = a.ws + ((size_t)((h * tiles + n) * a.parts) + part) * kPart;
#pragma unroll
        for (int d = 0; d < 4; ++d)
#pragma unroll
            for (int v = 0; v < 4; ++v)
                *reinterpret_cast<f32x4 *>(ws + ((d * 4 + v) * 256 + t) * 4) = f32x4{acc[d][4 * v], acc[d][4 * v + 1], acc[d][4 * v + 2], acc[d][4 * v + 3]};
        if (half == 0) *reinterpret_cast<f32x2 *>(ws + kRows * SKG_EXPANDED_V + (wave * 32 + l31) * 2) = f32x2{m, l};
        return;
    }
    if (j >= q.n) return;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint16_t *o = a.out + ((size_t)(q.first + j) * a.H + h) * SKG_EXPANDED_V + 4 * half;
#pragma unroll
    for (int d = 0; d < 4; ++d)
#pragma unroll
        for (int v = 0; v < 4; ++v)
            *reinterpret_cast<uint2 *>(o + d * 32 + 8 * v) =
                to_bf16x4(acc[d][4 * v] * inv, acc[d][4 * v + 1] * inv, acc[d][4 * v + 2] * inv, acc[d][4 * v + 3] * inv);
}

// Joins the parts of a tile in their order: a workgroup has 32 of the values of its 128
// tokens, a lane the same places as in the kernel above.  Bytes: 34 MB in 8.2 us.
__global__ void __launch_bounds__(256) latent_expanded_join_kernel(ExpandedArgs a, int tiles) {
    extern __shared__ __attribute__((aligned(16))) unsigned char lds_raw[];
    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int d = blockIdx.x & 3, n = (int)(blockIdx.x >> 2) % tiles, h = (int)(blockIdx.x >> 2) / tiles;
    const Place at = place_of(a, n, lds_raw);
    if (!at.there) return;
    const int parts = parts_of(a, keys_of(a, at, min(at.i * kRows + kRows, at.q.n) - 1));
    const int row = wave * 32 + (lane & 31), j = at.i * kRows + row;
    if (parts == 1 || j >= at.q.n) return;
    const float *ws = a.ws + (size_t)((h * tiles + n) * a.parts) * kPart;
    float m = -__builtin_inff(), l = 0.0f;
    f32x4 sum[4] = {};
    for (int p = 0; p < parts; ++p, ws += kPart) {
        f32x4 y[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) y[v] = *reinterpret_cast<const f32x4 *>(ws + ((d * 4 + v) * 256 + t) * 4);
        add_part(m, l, sum, *reinterpret_cast<const f32x2 *>(ws + kRows * SKG_EXPANDED_V + row * 2), y);
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint16_t *o = a.out + ((size_t)(at.q.first + j) * a.H + h) * SKG_EXPANDED_V + d * 32 + 4 * (lane >> 5);
#pragma unroll
    for (int v = 0; v < 4; ++v) *reinterpret_cast<uint2 *>(o + 8 * v) = to_bf16x4(sum[v][0] * inv, sum[v][1] * inv, sum[v][2] * inv, sum[v][3] * inv);
}

// Tiles of query tokens: each sequence has at most one that is not full.
static long tiles_of(int B, int T) { return B == 1 ? (T + kRows - 1) / kRows : std::min<long>(T, T / kRows + B); }

int latent_expanded_parts(int B, int T, int S, int H) {
    const long total = tiles_of(B, T) * H;
    return (int)std::max<long>(1, std::min<long>(kGroups / total, S / (kStep * kLeast)));
}
size_t latent_expanded_workspace_bytes() { return kGroups * kPart * 4; }

int launch_latent_expanded(const ExpandedArgs &a, hipStream_t stream) {
    const long tiles = tiles_of(a.B, a.T), total = tiles * a.H * a.parts;
    static std::atomic<unsigned long long> done{0};
    const hipError_t e = allow_dynamic_lds((const void *)latent_expanded_kernel, kExpandedLds, done);
    if (e != hipSuccess) return (int)e;
    hipLaunchKernelGGL(latent_expanded_kernel, dim3((unsigned)((total + 7) / 8 * 8)), dim3(256), kExpandedLds, stream, a, (int)tiles);
    if (a.parts > 1) {
        const size_t lds = a.B > 64 ? ((size_t)a.B + 1) * 8 + 64 : 0;
        static std::atomic<unsigned long long> join_done{0};
        const hipError_t f = allow_dynamic_lds((const void *)latent_expanded_join_kernel, (SKG_LATENT_MAX_B + 1) * 8 + 64, join_done);
        if (f != hipSuccess) return (int)f;
        hipLaunchKernelGGL(latent_expanded_join_kernel, dim3((unsigned)(tiles * a.H * 4)), dim3(256), lds, stream, a, (int)tiles);
    }
    return (int)hipGetLastError();
}

}  // namespace skg
