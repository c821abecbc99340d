// kernels_moe.hip -- the routed experts' feed-forward: the pairs (token,
// choice) sorted by expert, the two products over the sorted rows, and the
// weighted sum of each token's choices.
#include "device_common.h"
#include "internal.h"
#include "moe_internal.h"
#include "mx_common.h"

namespace skg {

// Workgroup e gathers the pairs of expert e, in the order of their index,
// after those of the experts before it, and lists its row tiles.  Each
// workgroup counts every expert's pairs itself (LDS counters), so no
// workgroup waits for another.  Pairs whose id is outside [0, E) are left out.
__global__ void __launch_bounds__(256)
    moe_sort_kernel(const int *__restrict__ ids, int P, int E, int tile_rows,
                    int *__restrict__ pairs, MoeTile *__restrict__ tiles, int *__restrict__ count) {
    extern __shared__ int hist[];  // [E]
    __shared__ int mine[4], before[4], tbefore[4], ttotal[4];
    const int e = blockIdx.x, t = threadIdx.x, lane = t & 63, wave = t >> 6;
    for (int i = t; i < E; i += 256) hist[i] = 0;
    __syncthreads();
    // wave w takes the w-th quarter of the pairs, in whole groups of 64
    const int q = ((P + 255) / 256) * 64, p0 = wave * q, p1 = min(P, p0 + q);
    int eq = 0;
    for (int p = p0 + lane; p < p1; p += 64) {
        const int id = ids[p];
        if ((unsigned)id < (unsigned)E) atomicAdd(&hist[id], 1);
        eq += id == e;
    }
    for (int d = 32; d > 0; d >>= 1) eq += __shfl_xor(eq, d, 64);
    if (lane == 0) mine[wave] = eq;
    __syncthreads();
    int b = 0, tb = 0, tt = 0;  // rows and tiles of the experts before e, tiles of all
    for (int i = t; i < E; i += 256) {
        const int c = hist[i], ct = (c + tile_rows - 1) / tile_rows;
        b += i < e ? c : 0;
        tb += i < e ? ct : 0;
        tt += ct;
    }
    for (int d = 32; d > 0; d >>= 1) {
        b += __shfl_xor(b, d, 64);
        tb += __shfl_xor(tb, d, 64);
        tt += __shfl_xor(tt, d, 64);
    }
    if (lane == 0) {
        before[wave] = b;
        tbefore[wave] = tb;
        ttotal[wave] = tt;
    }
    __syncthreads();
    const int row0 = before[0] + before[1] + before[2] + before[3];
    const int tile0 = tbefore[0] + tbefore[1] + tbefore[2] + tbefore[3];
    if (e == 0 && t == 0) count[0] = ttotal[0] + ttotal[1] + ttotal[2] + ttotal[3];
    const int n = mine[0] + mine[1] + mine[2] + mine[3];
    for (int i = t; i * tile_rows < n; i += 256)
        tiles[tile0 + i] = MoeTile{e, row0, n, tile0};
    int at = row0;
    for (int w = 0; w < wave; ++w) at += mine[w];
    for (int p = p0; p < p1; p += 64) {
        const bool here = p + lane < p1 && ids[p + lane] == e;
        const unsigned long long m = __ballot(here);
        if (here) pairs[at + __popcll(m & ((1ull << lane) - 1ull))] = p + lane;
        at += __popcll(m);
    }
}

// out[t, n] = sum_j weights[t, j] * y[t * k + j, n], j ascending, in fp32.
__global__ void __launch_bounds__(256)
    moe_combine_kernel(const float *__restrict__ y, const int *__restrict__ ids,
                       const float *__restrict__ weights, uint16_t *__restrict__ out, int k, int H,
                       int E) {
    const int t = blockIdx.x, n = (blockIdx.y * 256 + threadIdx.x) * 4;
    if (n >= H) return;
    f32x4 s{0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < k; ++j) {
        const size_t p = (size_t)t * k + j;
        if ((unsigned)ids[p] >= (unsigned)E) continue;
        const float w = weights[p];
        const f32x4 v = *reinterpret_cast<const f32x4 *>(y + p * H + n);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = __builtin_fmaf(w, v[i], s[i]);
    }
    uint2 r;
    r.x = f32_to_bf16_rne(s[0]) | (unsigned)f32_to_bf16_rne(s[1]) << 16;
    r.y = f32_to_bf16_rne(s[2]) | (unsigned)f32_to_bf16_rne(s[3]) << 16;
    *reinterpret_cast<uint2 *>(out + (size_t)t * H + n) = r;
}

namespace {

// The workspace, piece by piece, each 256-byte aligned.
struct MoeSpace {
    size_t xq, xe, h, he, y, pairs, tiles, count, bytes;
};

MoeSpace moe_space(int T, int k, int H, int I, int E, int fmt) {
    MoeSpace s{};
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t here = at;
        at += (n + 255) / 256 * 256;
        return here;
    };
    const size_t P = (size_t)T * k;
    s.xq = take((size_t)T * mx_code_stride(fmt, H));
    s.xe = take((size_t)T * mx_scale_stride(H));
    s.h = take(P * mx_code_stride(fmt, I));
    s.he = take(P * mx_scale_stride(I));
    s.y = take(P * H * 4);
    s.pairs = take(P * 4);
    s.tiles = take((size_t)moe_max_tiles((long)P, E, 16) * sizeof(MoeTile));
    s.count = take(4);
    s.bytes = at;
    return s;
}

}  // namespace

// Whether each pair reads its expert's weights for itself.
static bool moe_unsorted(const MoeArgs &a) {
    return ((long)a.T * a.k <= 16 || a.T == 1) && mxfp4_row_lds_bytes(a.fmt, a.H) <= kMxRowMaxLds;
}

int moe_tile_rows(int T, int k, int E) {
    const long avg = (long)T * k / E;
    return avg <= 8 ? 16 : avg <= 20 ? 32 : 64;
}

size_t moe_workspace_bytes(int T, int k, int H, int I, int E, int fmt) {
    return moe_space(T, k, H, I, E, fmt).bytes;
}

int launch_moe(const MoeArgs &a, void *workspace, hipStream_t stream) {
    const MoeSpace s = moe_space(a.T, a.k, a.H, a.I, a.E, a.fmt);
    uint8_t *b = (uint8_t *)workspace;
    if (moe_unsorted(a)) return launch_moe_rows(a, b + s.h, b + s.he, stream);
    const int P = a.T * a.k, rows = moe_tile_rows(a.T, a.k, a.E);
    const int tiles = moe_max_tiles(P, a.E, rows);
    const MoeLists lists{(const MoeTile *)(b + s.tiles), (const int *)(b + s.count),
                         (const int *)(b + s.pairs)};
    int e = launch_quant_mx(a.x, b + s.xq, b + s.xe, a.fmt, a.T, a.H, true, stream);
    if (e != (int)hipSuccess) return e;
    hipLaunchKernelGGL(moe_sort_kernel, dim3((unsigned)a.E), dim3(256), (size_t)a.E * 4, stream,
                       a.ids, P, a.E, rows, (int *)(b + s.pairs), (MoeTile *)(b + s.tiles),
                       (int *)(b + s.count));
    e = (int)hipGetLastError();
    if (e != (int)hipSuccess) return e;
    e = launch_moe_gate_up(a, lists, b + s.xq, b + s.xe, b + s.h, b + s.he, rows, tiles, stream);
    if (e != (int)hipSuccess) return e;
    e = launch_moe_down(a, lists, b + s.h, b + s.he, (float *)(b + s.y), rows, tiles, stream);
    if (e != (int)hipSuccess) return e;
    hipLaunchKernelGGL(moe_combine_kernel, dim3((unsigned)a.T, (unsigned)((a.H / 4 + 255) / 256)),
                       dim3(256), 0, stream, (const float *)(b + s.y), a.ids, a.weights, a.out, a.k,
                       a.H, a.E);
    return (int)hipGetLastError();
}

}  // namespace skg
