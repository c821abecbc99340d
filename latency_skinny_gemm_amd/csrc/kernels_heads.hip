// kernels_heads.hip -- out[t, h] = W[h] x[t, h]: a product per head, into and out
// of the absorbed form of latent attention.
//
// A wave keeps 32 of a head's N columns and the whole K (up to 512) in registers
// as fragments of the matrix instruction, loaded straight from memory, and takes 16 tokens after
// the other.  The two fragments' columns interleave by four, so that a lane ends
// with eight consecutive outputs.
#include <algorithm>

#include "internal.h"
#include "latent_common.h"
#include "latent_internal.h"

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

namespace {

template <int KS>
int go(const HeadsArgs &a, hipStream_t stream) {
    const int n_tiles = (a.N + 31) / 32;
    // tokens a wave: as many waves as fill the card, then up to 128
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
