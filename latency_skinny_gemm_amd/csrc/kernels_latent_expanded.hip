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
constexpr int kRopeRow = 2 * SKG_LATENT_ROPE;
constexpr int kSlotBytes = kStep * (kKvRow + kRopeRow);
constexpr int kLoads = 5;  // a wave's direct loads a step: 8 rows of keys and values, 8 shared parts
constexpr size_t kExpandedLds = std::max<size_t>(kSlots * kSlotBytes + 64, (SKG_LATENT_MAX_B + 1) * 8 + 64);
constexpr int kRows = 128;
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
    // direct loads: rows of 32 pieces, permuted among 16, and of 8
    const unsigned row_bytes = (unsigned)a.H * kKvRow;
    unsigned src[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int p = k * 64 + lane, row = p >> 5, c = p & 31;
        src[k] = (unsigned)row * row_bytes + (unsigned)((c ^ swz16(wave * 8 + row)) * 16);
    }
    const unsigned rope_bytes = (unsigned)a.rope_stride * 2;
    const unsigned rope_src = (unsigned)(lane >> 3) * rope_bytes + (unsigned)(((lane & 7) ^ swz8(wave * 8 + (lane >> 3))) * 16);
    unsigned koff[8], roff[4], voff[2][4];
#pragma unroll
    for (int c = 0; c < 8; ++c) koff[c] = (unsigned)l31 * kKvRow + (unsigned)(((c * 2 + half) ^ swz16(l31)) * 16);
#pragma unroll
    for (int c = 0; c < 4; ++c) roff[c] = (unsigned)(kStep * kKvRow) + (unsigned)l31 * kRopeRow + (unsigned)(((c * 2 + half) ^ swz8(l31)) * 16);
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const int row = 8 * y + 4 * half + (l15 >> 2);
            voff[y][d] = (unsigned)(row * kKvRow + 2 * SKG_EXPANDED_NOPE + ((d * 4 + (g4 & 1) * 2 + ((l15 & 3) >> 1)) ^ swz16(row)) * 16 + (l15 & 1) * 8);
        }
    const unsigned ring = uniform((int)lds_address(lds_raw));
    auto issue = [&](int step, int slot) {
        const int row = step * kStep + wave * 8, rows = min(max(most - row, 0), 8);
        const size_t at = (size_t)kv.first + (rows ? row : 0);
        const Rsrc rk = make_rsrc(a.kv + (at * a.H + h) * (kKvRow / 2), rows ? (unsigned)(rows - 1) * row_bytes + kKvRow : 0u);
        const Rsrc rr = make_rsrc(a.k_rope + at * a.rope_stride, rows ? (unsigned)(rows - 1) * rope_bytes + kRopeRow : 0u);
        const unsigned dst = ring + slot * kSlotBytes;
        each<4>([&](auto k) { ring_load16<k * 1024>(rk, dst + wave * 8 * kKvRow, src[k]); });
        ring_load16<kStep * kKvRow>(rr, dst + wave * 1024, rope_src);
    };

    unsigned char *flags = lds_raw + kSlots * kSlotBytes;
    const int steps = (most + kStep - 1) / kStep;
    f32x16 acc[4];
    float m, l;
    bool careful = false;
    for (;;) {
#pragma unroll
        for (int d = 0; d < 4; ++d)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[d][r] = 0.0f;
        m = -__builtin_inff();
        l = 0.0f;
        for (int k = 0; k < kSlots - 1; ++k)
            if (k < steps) issue(k, k);
        int slot = 0, fill = kSlots - 1;
        for (int k = 0; k < steps; ++k) {
            if (k + 1 < steps) wait_vmcnt_lds<kLoads>();
            else wait_vmcnt_lds<0>();
            barrier_nofence();
            if (k + kSlots - 1 < steps) issue(k + kSlots - 1, fill);
            const unsigned char *tile = lds_raw + slot * kSlotBytes;
            slot = slot + 1 == kSlots ? 0 : slot + 1;
            fill = fill + 1 == kSlots ? 0 : fill + 1;
            const int row0 = k * kStep;
            const bool masked = row0 + kStep > lim0;
            float p[16];
            bf16x8 pf[2] = {};
            if (row0 < wave_most) {
                f32x16 z;
#pragma unroll
                for (int r = 0; r < 16; ++r) z[r] = 0.0f;
#pragma unroll
                for (int c = 0; c < 12; ++c) {
                    const bf16x8 kf = *reinterpret_cast<const bf16x8 *>(tile + (c < 8 ? koff[c] : roff[c - 8]));
                    z = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[c], z, 0, 0, 0);
                }
                if (masked) {
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        z[r] = row0 + 8 * (r >> 2) + 4 * half + (r & 3) < lim ? z[r] : -__builtin_inff();
                }
                float top = z[0];
#pragma unroll
                for (int r = 1; r < 16; ++r) top = fmaxf(top, z[r]);
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
                for (int r = 0; r < 16; ++r) p[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(z[r], a.factor, -ref));
                pf[0] = to_bf16x8(p);
                pf[1] = to_bf16x8(p + 8);
                l = add_bf16x8(pf[1], add_bf16x8(pf[0], l));
            }
            if (__builtin_expect(careful && row0 + kStep > sees(i * kRows), 0)) {
                // keys whose values hold an infinity or NaN, in a step that some tokens do
                // not see: their products by vector instructions for those that do, zeros
                // for the matrix instruction
                bool bad = false;
                for (int e = 0; e < 8; ++e) {
                    const unsigned w = *reinterpret_cast<const unsigned *>(
                        tile + (wave * 8 + (lane >> 3)) * kKvRow + 2 * SKG_EXPANDED_NOPE + (lane & 7) * 32 + e * 4);
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
                            const uint2 w = *reinterpret_cast<const uint2 *>(tile + r0 * kKvRow + 2 * SKG_EXPANDED_NOPE + (c ^ swz16(r0)) * 16 + half * 8);
                            const float y[4] = {bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)};
#pragma unroll
                            for (int u = 0; u < 4; ++u)
                                if (in) acc[d][4 * v + u] = __builtin_fmaf(pk, y[u], acc[d][4 * v + u]);
                        }
                }
                __syncthreads();
                for (unsigned f = flagged; f; f &= f - 1)
                    if (t < 64) *reinterpret_cast<unsigned *>(const_cast<unsigned char *>(tile) + __builtin_ctz(f) * kKvRow + 2 * SKG_EXPANDED_NOPE + t * 4) = 0;
                __syncthreads();
            }
            if (row0 < wave_most) {
#pragma unroll
                for (int d = 0; d < 4; ++d) {
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk) {
                        const s16x4 x = lds_transposed4(tile + voff[0][d] + kk * 16 * kKvRow);
                        const s16x4 y = lds_transposed4(tile + voff[1][d] + kk * 16 * kKvRow);
                        acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                            __builtin_bit_cast(bf16x8, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7)), pf[kk], acc[d], 0, 0, 0);
                    }
                }
            }
        }
        wait_vmcnt_lds<0>();
        __syncthreads();
        // see kernels_latent_attention.hip: infinities and NaN of keys that a token does not see
        if (careful || sees(i * kRows) >= most) break;
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
        if (!some) break;
        careful = true;
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
