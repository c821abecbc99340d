// kernels_latent_expanded.hip -- attention of prompts over expanded keys and
// values: a head's key is 128 values of its own and 64 that all heads share.
//
// A workgroup takes 128 query tokens of one head, a wave 32 of them; steps of 32
// keys and values come to an LDS ring by direct loads.  Scores are made
// transposed, so that a lane has eight keys of one token in the registers in which
// the second product takes its weights.
#include <algorithm>

#include "internal.h"
#include "latent_common.h"
#include "latent_internal.h"
#include "lds_limit.h"

namespace skg {

namespace {

constexpr int kStep = 32, kSlots = 3;
constexpr int kKvRow = 2 * (SKG_EXPANDED_NOPE + SKG_EXPANDED_V);  // bytes
constexpr int kOwnRow = 2 * SKG_EXPANDED_NOPE, kRopeRow = 2 * SKG_LATENT_ROPE, kValueRow = 2 * SKG_EXPANDED_V;
constexpr int kKeyBytes = kStep * (kOwnRow + kRopeRow), kValueBytes = kStep * kValueRow;
constexpr int kLoads = 5;  // a wave's direct loads a step: 8 keys, their shared parts, 8 values
constexpr int kFlags = kSlots * (kKeyBytes + kValueBytes);
constexpr size_t kExpandedLds = std::max<size_t>(kFlags + 64, (SKG_LATENT_MAX_B + 1) * 8 + 64);
constexpr int kRows = 128;
constexpr int kAhead = 4;  // keys' fragments under way
constexpr int kQuery = SKG_EXPANDED_NOPE + SKG_LATENT_ROPE;

}  // namespace

__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2))) latent_expanded_kernel(ExpandedArgs a, int tiles) {
    extern __shared__ __attribute__((aligned(16))) unsigned char lds_raw[];
    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    // a head's tiles lie on one XCD, those with the most keys first
    const unsigned total = (unsigned)tiles * (unsigned)a.H, per = (total + 7) / 8;
    const unsigned id = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if ((blockIdx.x >> 3) >= per || id >= total) return;
    const int h = (int)(id / (unsigned)tiles), n = tiles - 1 - (int)(id % (unsigned)tiles);

    int b = 0, i = n;
    if (a.B > 1) {
        long *pre = reinterpret_cast<long *>(lds_raw);
        block_prefix<4>(a.B, pre, pre + a.B + 1, [&](int s) { return (long)((new_tokens(a.q_starts, s, a.T).n + kRows - 1) / kRows); });
        if (n >= pre[a.B]) return;
        b = uniform(find_sequence(pre, a.B, n));
        i = uniform(n - (int)pre[b]);
        __syncthreads();
    }
    const Tokens q = uniform(new_tokens(a.q_starts, b, a.T)), kv = uniform(new_tokens(a.kv_starts, b, a.S));
    if (i * kRows >= q.n) return;
    const int before = a.causal ? kv.n - q.n : kv.n - 1;  // token j sees keys 0 .. before + j (causal) or before
    auto sees = [&](int j) { return max(a.causal ? before + j + 1 : kv.n, 0); };
    const int half = lane >> 5, l15 = lane & 15, l31 = lane & 31, g4 = lane >> 4;
    const int j = i * kRows + wave * 32 + l31;
    const bool live = j < q.n;
    const int lim = live ? sees(j) : 0;
    const int lim0 = sees(i * kRows + wave * 32);                          // of the wave's first token
    const int wave_most = sees(min(i * kRows + wave * 32 + 31, q.n - 1));  // and its last
    const int most = sees(min(i * kRows + kRows - 1, q.n - 1));

    bf16x8 qf[12];
    {
        const uint16_t *p = a.q + ((size_t)(q.first + (live ? j : 0)) * a.H + h) * kQuery + half * 8;
#pragma unroll
        for (int k = 0; k < 12; ++k) {
            u32x4 v{0, 0, 0, 0};
            if (live) v = *reinterpret_cast<const u32x4 *>(p + k * 16);
            qf[k] = __builtin_bit_cast(bf16x8, v);
        }
    }
    wait_vmcnt_lds<0>();  // here, so that the compiler waits for no load inside the loop over the ring
    // direct loads: a head's keys and values in rows of 16 pieces, the shared parts of 8
    const unsigned row_bytes = (unsigned)a.H * kKvRow;
    unsigned src[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int row = k * 4 + g4;
        src[k] = (unsigned)row * row_bytes + (unsigned)((l15 ^ swz16(wave * 8 + row)) * 16);
    }
    const unsigned rope_bytes = (unsigned)a.rope_stride * 2;
    const unsigned rope_src = (unsigned)(lane >> 3) * rope_bytes + (unsigned)(((lane & 7) ^ swz8(wave * 8 + (lane >> 3))) * 16);
    unsigned koff[8], roff[4], voff[2][4];
#pragma unroll
    for (int c = 0; c < 8; ++c) koff[c] = (unsigned)l31 * kOwnRow + (unsigned)(((c * 2 + half) ^ swz16(l31)) * 16);
#pragma unroll
    for (int c = 0; c < 4; ++c) roff[c] = (unsigned)(kStep * kOwnRow) + (unsigned)l31 * kRopeRow + (unsigned)(((c * 2 + half) ^ swz8(l31)) * 16);
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const int row = 8 * y + 4 * half + (l15 >> 2);
            voff[y][d] = (unsigned)(kSlots * kKeyBytes + row * kValueRow + ((d * 4 + (g4 & 1) * 2 + ((l15 & 3) >> 1)) ^ swz16(row)) * 16 + (l15 & 1) * 8);
        }
    const unsigned ring = uniform((int)lds_address(lds_raw));
    // a step's keys, and the values of the step before; steps are brought in order
    struct Next {
        const uint16_t *own, *shared;  // this wave's rows
        int row;
        unsigned value_bytes;
    };
    auto rewind = [&] {
        const size_t at = (size_t)kv.first + wave * 8;
        return Next{a.kv + (at * a.H + h) * (kKvRow / 2), a.k_rope + at * a.rope_stride, wave * 8, 0u};
    };
    auto issue = [&](Next &n, int key_slot, int value_slot) {
        const int rows = min(uniform(most - n.row), 8);
        const unsigned bytes = rows > 0 ? (unsigned)(rows - 1) * row_bytes + kOwnRow : 0u;
        const unsigned shared = rows > 0 ? (unsigned)(rows - 1) * rope_bytes + kRopeRow : 0u;
        const unsigned keys = ring + key_slot * kKeyBytes, values = ring + value_slot * kValueBytes;
        const Rsrc rk = make_rsrc(n.own, bytes), rr = make_rsrc(n.shared, shared);
        const Rsrc rv = make_rsrc(n.own - (size_t)(kStep / 2) * row_bytes + SKG_EXPANDED_NOPE, n.value_bytes);
        each<2>([&](auto k) { ring_load16<k * 1024>(rk, keys + wave * 8 * kOwnRow, src[k]); });
        ring_load16<kStep * kOwnRow>(rr, keys + wave * 1024, rope_src);
        each<2>([&](auto k) { ring_load16<kSlots * kKeyBytes + k * 1024>(rv, values + wave * 8 * kValueRow, src[k]); });
        n.own += (size_t)(kStep / 2) * row_bytes;
        n.shared += (size_t)kStep * a.rope_stride;
        n.row += kStep;
        n.value_bytes = bytes;
    };

    unsigned char *flags = lds_raw + kFlags;
    const int steps = (most + kStep - 1) / kStep;
    f32x16 acc[4];
    float m = 0.0f, l = 0.0f, x[16];  // x: scores over m, logarithms of weights
    bf16x8 pf[2];
    auto read_key = [&](const unsigned char *keys, int c) { return *reinterpret_cast<const u32x4 *>(keys + (c < 8 ? koff[c] : roff[c - 8])); };
    auto read_values = [&](const unsigned char *values, int d, s16x8 (&v)[2]) {
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            const s16x4 v0 = lds_transposed4(values + voff[0][d] + kk * 16 * kValueRow);
            const s16x4 v1 = lds_transposed4(values + voff[1][d] + kk * 16 * kValueRow);
            v[kk] = __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    };
    auto weigh = [&](int part) {  // four of the weights
        bf16x4 w;
#pragma unroll
        for (int r = 0; r < 4; ++r) w[r] = (__bf16)__builtin_amdgcn_exp2f(x[part * 4 + r]);
#pragma unroll
        for (int r = 0; r < 4; ++r) pf[part >> 1][(part & 1) * 4 + r] = w[r];
        const bf16x2 one{(__bf16)1.0f, (__bf16)1.0f};
        l = __builtin_amdgcn_fdot2_f32_bf16(__builtin_shufflevector(w, w, 0, 1), one, l, false);
        l = __builtin_amdgcn_fdot2_f32_bf16(__builtin_shufflevector(w, w, 2, 3), one, l, false);
    };
    auto masked = [&](f32x16 &z, int row0) {
        if (row0 + kStep > lim0) {
            const int left = here(lim) - row0 - 4 * half;
#pragma unroll
            for (int r = 0; r < 16; ++r) z[r] = 8 * (r >> 2) + (r & 3) < left ? z[r] : -__builtin_inff();
        }
    };
    auto scaled = [&](const f32x16 &z, float top) {
        top = other_half_max(top) * a.factor;
        if (__any(top > m + 8.0f)) {
            const float next = fmaxf(m, top);
            const float down = next == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(m - next);
            m = next;
            l *= down;
#pragma unroll
            for (int d = 0; d < 4; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[d][r] *= down;
        }
        const float ref = m == -__builtin_inff() ? 0.0f : m;
#pragma unroll
        for (int r = 0; r < 16; ++r) x[r] = __builtin_fmaf(z[r], a.factor, -ref);
    };
    // the scores of a step, and between them the weights of the one before
    auto scores = [&](const unsigned char *keys, auto weights) {
        f32x16 z;
        u32x4 kf[kAhead][1];
#pragma unroll
        for (int c = 0; c < kAhead - 1; ++c) kf[c][0] = read_key(keys, c);
#pragma unroll
        for (int r = 0; r < 16; ++r) z[r] = 0.0f;
#pragma unroll
        for (int c = 0; c < 12; ++c) {
            if (c + kAhead - 1 < 12) kf[(c + kAhead - 1) % kAhead][0] = read_key(keys, c + kAhead - 1);
            arrived(kf[c % kAhead]);
            z = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16(kf[c % kAhead][0]), qf[c], z, 0, 0, 0);
            if constexpr (decltype(weights)::value)
                if (c % 3 == 0) weigh(c / 3);
        }
        return z;
    };
    // this step's sums, and between them the maximum of the next one's scores
    auto sums = [&](const unsigned char *values, s16x8 (&vf)[2][2], const f32x16 &z) {
        float top = -__builtin_inff();
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            if (d + 1 < 4) read_values(values, d + 1, vf[(d + 1) & 1]);
            arrived(vf[d & 1]);
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16(vf[d & 1][kk]), pf[kk], acc[d], 0, 0, 0);
#pragma unroll
            for (int r = 0; r < 4; ++r) top = fmaxf(top, z[d * 4 + r]);
        }
        return top;
    };
    // keys whose values hold an infinity or NaN, in a step that some tokens do not see:
    // their products by vector instructions for those that do, zeros for the matrix
    // instruction
    auto apart = [&](unsigned char *values, int row0) {
        bool bad = false;
        for (int e = 0; e < 8; ++e) {
            const unsigned w = *reinterpret_cast<const unsigned *>(values + (wave * 8 + (lane >> 3)) * kValueRow + (lane & 7) * 32 + e * 4);
            bad |= (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
        }
        const unsigned long long any = __ballot(bad);
        unsigned rows8 = 0;
#pragma unroll
        for (int r = 0; r < 8; ++r) rows8 |= ((any >> (8 * r)) & 0xFFull ? 1u : 0u) << r;
        if (lane == 0) flags[wave] = (unsigned char)rows8;
        __syncthreads();
        const unsigned flagged = __builtin_amdgcn_readfirstlane(*reinterpret_cast<const unsigned *>(flags));
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
                    const int c = d * 4 + v;
                    const uint2 w = *reinterpret_cast<const uint2 *>(values + r0 * kValueRow + (c ^ swz16(r0)) * 16 + half * 8);
                    const float y[4] = {bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)};
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        if (in) acc[d][4 * v + u] = __builtin_fmaf(pk, y[u], acc[d][4 * v + u]);
                }
        }
        __syncthreads();
        for (unsigned f = flagged; f; f &= f - 1)
            if (t < 64) *reinterpret_cast<unsigned *>(values + __builtin_ctz(f) * kValueRow + t * 4) = 0;
        __syncthreads();
    };
    Next next;
    auto begin = [&] {
#pragma unroll
        for (int d = 0; d < 4; ++d)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[d][r] = 0.0f;
        m = -__builtin_inff();
        l = 0.0f;
        next = rewind();
        issue(next, 0, 2);
        issue(next, 1, 0);
        issue(next, 2, 1);
        wait_vmcnt_lds<2 * kLoads>();
        barrier_nofence();
        f32x16 z = scores(lds_raw, std::false_type{});
        masked(z, 0);
        float top = z[0];
#pragma unroll
        for (int r = 1; r < 16; ++r) top = fmaxf(top, z[r]);
        scaled(z, top);
    };
    // step k, with its values in slot `at` and the next one's keys in the slot after
    auto step = [&](int k, int at, auto careful) {
        const int after = (at + 1) % kSlots, last = (at + 2) % kSlots;
        wait_vmcnt_lds<kLoads>();
        barrier_nofence();
        issue(next, at, last);
        const int row0 = k * kStep;
        unsigned char *const values = lds_raw + at * kValueBytes;
        const bool seen = row0 < wave_most;
        f32x16 z;
        s16x8 vf[2][2];
        if (seen) z = scores(lds_raw + after * kKeyBytes, std::true_type{});
        if constexpr (decltype(careful)::value) {
            if (!seen) pf[0] = pf[1] = bf16x8{};
            if (row0 + kStep > sees(i * kRows)) apart(values + kSlots * kKeyBytes, row0);
        }
        if (!seen) return;
        read_values(values, 0, vf[0]);
        masked(z, row0 + kStep);
        scaled(z, sums(values, vf, z));
    };
    if (steps > 0) {
        begin();
        for (int k = 0;; k += 3) {
            step(k, 0, std::false_type{});
            if (k + 1 >= steps) break;
            step(k + 1, 1, std::false_type{});
            if (k + 2 >= steps) break;
            step(k + 2, 2, std::false_type{});
            if (k + 3 >= steps) break;
        }
        wait_vmcnt_lds<0>();
        __syncthreads();
        // see kernels_latent_attention.hip: infinities and NaN of keys that a token does not see
        if (sees(i * kRows) < most) {
            bool bad = false;
#pragma unroll
            for (int d = 0; d < 4; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r) bad |= not_finite(acc[d][r]);
            const unsigned long long found = __ballot(bad && live);
            if (lane == 0) flags[wave] = found != 0;
            __syncthreads();
            const unsigned some = __builtin_amdgcn_readfirstlane(*reinterpret_cast<const unsigned *>(flags));
            __syncthreads();
            if (__builtin_expect(some, 0)) {
                begin();
                for (int k = 0; k < steps; ++k) step(k, k % kSlots, std::true_type{});
                wait_vmcnt_lds<0>();
            }
        }
    } else {
#pragma unroll
        for (int d = 0; d < 4; ++d)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[d][r] = 0.0f;
    }
    l = other_half_sum(l);
    if (!live) return;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint16_t *o = a.out + ((size_t)(q.first + j) * a.H + h) * SKG_EXPANDED_V + 4 * half;
#pragma unroll
    for (int d = 0; d < 4; ++d)
#pragma unroll
        for (int v = 0; v < 4; ++v)
            *reinterpret_cast<uint2 *>(o + d * 32 + 8 * v) =
                to_bf16x4(acc[d][4 * v] * inv, acc[d][4 * v + 1] * inv, acc[d][4 * v + 2] * inv, acc[d][4 * v + 3] * inv);
}

int launch_latent_expanded(const ExpandedArgs &a, hipStream_t stream) {
    // each sequence has at most one tile that is not full
    const long tiles = a.B == 1 ? (a.T + kRows - 1) / kRows : std::min<long>(a.T, a.T / kRows + a.B);
    const long total = tiles * a.H;
    static std::atomic<unsigned long long> done{0};
    const hipError_t e = allow_dynamic_lds((const void *)latent_expanded_kernel, kExpandedLds, done);
    if (e != hipSuccess) return (int)e;
    hipLaunchKernelGGL(latent_expanded_kernel, dim3((unsigned)((total + 7) / 8 * 8)), dim3(256), kExpandedLds, stream, a, (int)tiles);
    return (int)hipGetLastError();
}

}  // namespace skg
