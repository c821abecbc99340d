// kernels_heads.hip -- out[t, h] = W[h] x[t, h]: a product per head, into and out
// of the absorbed form of latent attention.
//
// A wave keeps 32 of a head's N columns and the whole K (up to 512) in registers
// as fragments of the matrix instruction, loaded straight from memory, and takes 16 tokens after
// the other.  The two fragments' columns interleave by four, so that a lane ends
// with eight consecutive outputs.  One token, 128 heads, 512 by 128: 4.6 us, 16.8 MB of
// weights at 3.7 TB/s.
#include <algorithm>

#include "internal.h"
#include "latent_common.h"
#include "latent_internal.h"
#include "lds_limit.h"

namespace skg {

template <int KS>
__global__ void __launch_bounds__(256) heads_kernel(HeadsArgs a, int n_tiles, int t_step, int t_parts) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int u = (int)blockIdx.x * 4 + wave;  // (head, token part, column tile)
    const int n_tile = u % n_tiles, rest = u / n_tiles, part = rest % t_parts, h = rest / t_parts;
    if (h >= a.H) return;
    const int l15 = lane & 15, g4 = lane >> 4;
    const int t0 = part * t_step, t1 = min(a.T, t0 + t_step);
    const uint16_t *w = a.W + ((size_t)h * a.N) * a.K;
    bf16x8 wf[2][KS];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int n = min(n_tile * 32 + (l15 >> 2) * 8 + x * 4 + (l15 & 3), a.N - 1);
#pragma unroll
        for (int k = 0; k < KS; ++k)
            wf[x][k] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4 *>(w + (size_t)n * a.K + k * 32 + g4 * 8));
    }
    const int n0 = n_tile * 32 + g4 * 8;
    for (int t = t0; t < t1; t += 16) {
        const int tok = t + l15;
        const uint16_t *x = a.x + (size_t)min(tok, a.T - 1) * a.xt + (size_t)h * a.xh + g4 * 8;
        bf16x8 xf[KS];
#pragma unroll
        for (int k = 0; k < KS; ++k) xf[k] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4 *>(x + k * 32));
        f32x4 c[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int y = 0; y < 2; ++y) c[y] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[y][k], xf[k], c[y], 0, 0, 0);
        if (tok < a.T && n0 < a.N) {
            const uint2 lo = to_bf16x4(c[0][0], c[0][1], c[0][2], c[0][3]), hi = to_bf16x4(c[1][0], c[1][1], c[1][2], c[1][3]);
            *reinterpret_cast<u32x4 *>(a.out + (size_t)tok * a.ot + (size_t)h * a.oh + n0) = u32x4{lo.x, lo.y, hi.x, hi.y};
        }
    }
}

// The same for many tokens: the four waves of a workgroup, 128 columns, take the
// tokens' rows from a ring in LDS, so that a row is read once for them and a step's
// rows are on their way while earlier ones are multiplied.  K a multiple of 128.  2048
// tokens, 128 heads, 128 by 512: 80 us, 352 MB at 4.4 TB/s (170 by the kernel above).
constexpr int kHeadsRing = 4;
template <int KS>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2))) heads_ring_kernel(HeadsArgs a, int n_tiles, int t_step, int t_parts) {
    constexpr int SLOT = KS * 1024, LOADS = KS / 4, PIECES = KS * 4;  // 16 tokens; a wave's loads; a row's pieces
    static_assert(KS % 4 == 0, "whole loads for each wave");
    extern __shared__ __attribute__((aligned(16))) unsigned char lds_raw[];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int u = (int)blockIdx.x, n_tile = u % n_tiles, rest = u / n_tiles, part = rest % t_parts, h = rest / t_parts;
    const int l15 = lane & 15, g4 = lane >> 4;
    const int t0 = part * t_step, t1 = min(a.T, t0 + t_step), steps = (t1 - t0 + 15) / 16;
    const unsigned row_bytes = (unsigned)a.xt * 2u;
    unsigned src[LOADS];
#pragma unroll
    for (int k = 0; k < LOADS; ++k) {
        const int p = (k * 4 + wave) * 64 + lane, row = p / PIECES, c = p % PIECES;
        src[k] = (unsigned)row * row_bytes + (unsigned)((c ^ swz16(row)) * 16);
    }
    const unsigned ring = (unsigned)uniform((int)lds_address(lds_raw + wave * 1024));
    auto issue = [&](int step, int slot) {
        const int t = t0 + step * 16, rows = min(max(t1 - t, 0), 16);
        const Rsrc rs = make_rsrc(a.x + (size_t)(rows ? t : t0) * a.xt + (size_t)h * a.xh, rows ? (unsigned)(rows - 1) * row_bytes + KS * 64u : 0u);
        each<LOADS>([&](auto k) { ring_load16<k * 4096>(rs, ring + slot * SLOT, src[k]); });
    };
    const int n_first = n_tile * 128 + wave * 32;
    const uint16_t *w = a.W + ((size_t)h * a.N) * a.K;
    u32x4 wf[2][KS];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int n = min(n_first + (l15 >> 2) * 8 + x * 4 + (l15 & 3), a.N - 1);
#pragma unroll
        for (int k = 0; k < KS; ++k) wf[x][k] = *reinterpret_cast<const u32x4 *>(w + (size_t)n * a.K + k * 32 + g4 * 8);
    }
    wait_vmcnt_lds<0>();  // here, so that the compiler waits for no load inside the loop
#pragma unroll
    for (int k = 0; k < kHeadsRing - 1; ++k) issue(k, k);
    const int n0 = n_first + g4 * 8;
    uint16_t *o = a.out + (size_t)(t0 + l15) * a.ot + (size_t)h * a.oh + n0;
    int slot = 0;
    for (int k = 0; k < steps; ++k) {
        wait_vmcnt_lds<(kHeadsRing - 2) * LOADS>();
        barrier_nofence();
        issue(k + kHeadsRing - 1, (slot + kHeadsRing - 1) & (kHeadsRing - 1));
        const unsigned char *row = lds_raw + slot * SLOT + l15 * (KS * 64);
        slot = (slot + 1) & (kHeadsRing - 1);
        f32x4 c[2] = {};
        u32x4 xf[2][4];
        auto read = [&](int q, u32x4(&x)[4]) {
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = *reinterpret_cast<const u32x4 *>(row + ((q * 16 + e * 4 + g4) ^ swz16(l15)) * 16);
        };
        read(0, xf[0]);
#pragma unroll
        for (int q = 0; q < KS / 4; ++q) {
            if (q + 1 < KS / 4) read(q + 1, xf[(q + 1) & 1]);
            arrived(xf[q & 1]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int y = 0; y < 2; ++y) c[y] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(wf[y][q * 4 + e]), as_bf16(xf[q & 1][e]), c[y], 0, 0, 0);
        }
        if (t0 + k * 16 + l15 < t1 && n0 < a.N) {
            const uint2 lo = to_bf16x4(c[0][0], c[0][1], c[0][2], c[0][3]), hi = to_bf16x4(c[1][0], c[1][1], c[1][2], c[1][3]);
            *reinterpret_cast<u32x4 *>(o + (size_t)k * 16 * a.ot) = u32x4{lo.x, lo.y, hi.x, hi.y};
        }
    }
    wait_vmcnt_lds<0>();  // no load to LDS outlives the loop
}

// The ring from the tokens on whose rows it saves more than its start costs (direct
// against ring, 128 heads, us: K = 512, 16 tokens 8.2, 8.3, 32 10.1, 8.1, 128 24, 10;
// K = 128, 96 tokens 11.4, 13.0, 128 13.7, 13.0, 256 23, 18).  A row of 16 tokens
// spans less than 2 GiB.
bool heads_ring(int T, int K, long x_token_stride) { return K % 128 == 0 && (long)T * K >= 16384 && x_token_stride < 1L << 26; }

namespace {

template <int KS>
int go(const HeadsArgs &a, hipStream_t stream) {
    if constexpr (KS % 4 == 0) {
        if (heads_ring(a.T, a.K, a.xt)) {
            static std::atomic<unsigned long long> done{0};
            const hipError_t e = allow_dynamic_lds((const void *)heads_ring_kernel<KS>, kHeadsRing * KS * 1024, done);
            if (e != hipSuccess) return (int)e;
            const int tiles = (a.N + 127) / 128;
            // two workgroups a CU, twice
            const long want = std::max<long>(1, 1024 / ((long)a.H * tiles));
            const int step = (int)std::min<long>(512, std::max<long>(64, ((a.T + want - 1) / want + 15) / 16 * 16));
            const int parts = (a.T + step - 1) / step;
            hipLaunchKernelGGL((heads_ring_kernel<KS>), dim3((unsigned)((long)a.H * parts * tiles)), dim3(256), kHeadsRing * KS * 1024, stream, a, tiles, step, parts);
            return (int)hipGetLastError();
        }
    }
    const int n_tiles = (a.N + 31) / 32;
    // tokens a wave: all up to 128, however many waves that makes
    const int step = std::min(128, (a.T + 15) / 16 * 16);
    const int parts = (a.T + step - 1) / step;
    const long waves = (long)a.H * parts * n_tiles;
    hipLaunchKernelGGL((heads_kernel<KS>), dim3((unsigned)((waves + 3) / 4)), dim3(256), 0, stream, a, n_tiles, step, parts);
    return (int)hipGetLastError();
}

template <int KS>
int by_k(const HeadsArgs &a, hipStream_t stream) {
    if constexpr (KS == 0) return (int)hipErrorInvalidValue;
    else return a.K == KS * 32 ? go<KS>(a, stream) : by_k<KS - 1>(a, stream);
}

}  // namespace

int launch_heads(const HeadsArgs &a, hipStream_t stream) { return by_k<16>(a, stream); }

}  // namespace skg
