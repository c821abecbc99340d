// kernels_moe.hip -- the routed experts' feed-forward: the pairs (token,
// choice) sorted by expert, the two products over the sorted rows, and the
// weighted sum of each token's choices.
#include <math.h>

#include "device_common.h"
#include "internal.h"
#include "moe_internal.h"
#include "mx_common.h"

namespace skg {

namespace {
constexpr int kPrepThreads = 1024;
constexpr int kPrepWaves = kPrepThreads / 64;
constexpr int kIdsInFlight = 8;  // loads of ids a lane has out at once

struct PrepArgs {
    const uint16_t *x;
    uint8_t *xq, *xe;
    unsigned n8, k8, q_stride, e_stride;
    const int *ids;
    int P, E, tile_rows, tall;
    int *pairs;
    MoeTile *tiles;
    int *count;
};

// Sum over the workgroup of three values per thread, in every thread.
__device__ __forceinline__ int3 block_sum(int3 v, int (*lds)[3]) {
    for (int d = 32; d > 0; d >>= 1) {
        v.x += __shfl_xor(v.x, d, 64);
        v.y += __shfl_xor(v.y, d, 64);
        v.z += __shfl_xor(v.z, d, 64);
    }
    if ((threadIdx.x & 63) == 0) {
        int *o = lds[threadIdx.x >> 6];
        o[0] = v.x;
        o[1] = v.y;
        o[2] = v.z;
    }
    __syncthreads();
    v = int3{0, 0, 0};
    for (int w = 0; w < kPrepWaves; ++w) {
        v.x += lds[w][0];
        v.y += lds[w][1];
        v.z += lds[w][2];
    }
    return v;
}

// Workgroup e < E gathers the pairs of expert e, in the order of their index,
// after those of the experts before it, and lists its row tiles.  Each
// workgroup counts every expert's pairs itself (LDS counters; integer sums, so
// their order does not matter) and none waits for another: the ids are read E
// times from L2, 16 waves with eight loads each in flight.  Pairs whose id is
// outside [0, E) are left out.
//
// 8192 pairs of 128 experts take 8.5 us, with the quantising of 2048 x 2880 in
// the same launch, and 320 pairs of 64 experts 4.9: two passes over the ids, one
// load after another, and the barriers between them.
__device__ __forceinline__ void sort_pairs(const PrepArgs &a, int *hist) {
    __shared__ int mine[kPrepWaves], sums[kPrepWaves][3];
    const int e = blockIdx.x, t = threadIdx.x, lane = t & 63, wave = t >> 6;
    for (int i = t; i < a.E; i += kPrepThreads) hist[i] = 0;
    __syncthreads();
    // wave w takes the w-th run of the pairs, in whole groups of 64
    const int run = ((a.P + kPrepThreads - 1) / kPrepThreads) * 64;
    const int p0 = min(a.P, wave * run), p1 = min(a.P, p0 + run);
    int eq = 0;
    for (int p = p0; p < p1; p += 64 * kIdsInFlight) {
        int id[kIdsInFlight];
#pragma unroll
        for (int i = 0; i < kIdsInFlight; ++i) {
            const int q = p + i * 64 + lane;
            id[i] = q < p1 ? a.ids[q] : -1;
        }
#pragma unroll
        for (int i = 0; i < kIdsInFlight; ++i) {
            if ((unsigned)id[i] < (unsigned)a.E) atomicAdd(&hist[id[i]], 1);
            eq += __popcll(__ballot(id[i] == e));
        }
    }
    if (lane == 0) mine[wave] = eq;
    __syncthreads();
    int3 v{0, 0, 0};  // rows and tiles of the experts before e, tiles of all
    for (int i = t; i < a.E; i += kPrepThreads) {
        const int c = hist[i], h = moe_tile_height(c, a.tile_rows, a.tall), ct = (c + h - 1) / h;
        v.x += i < e ? c : 0;
        v.y += i < e ? ct : 0;
        v.z += ct;
    }
    v = block_sum(v, sums);
    if (e == 0 && t == 0) a.count[0] = v.z;
    const int n = hist[e], height = moe_tile_height(n, a.tile_rows, a.tall);
    for (int i = t; i * height < n; i += kPrepThreads) a.tiles[v.y + i] = MoeTile{e, v.x, n, v.y};
    int at = v.x;
    for (int w = 0; w < wave; ++w) at += mine[w];
    for (int p = p0; p < p1; p += 64 * kIdsInFlight) {
        int id[kIdsInFlight];
#pragma unroll
        for (int i = 0; i < kIdsInFlight; ++i) {
            const int q = p + i * 64 + lane;
            id[i] = q < p1 ? a.ids[q] : -1;
        }
#pragma unroll
        for (int i = 0; i < kIdsInFlight; ++i) {
            const bool here = id[i] == e;
            const unsigned long long m = __ballot(here);
            if (here) a.pairs[at + __popcll(m & ((1ull << lane) - 1ull))] = p + i * 64 + lane;
            at += __popcll(m);
        }
    }
}
}  // namespace

// What the products need first, in one launch: workgroups [0, E) sort, the
// rest quantise x.
template <int FMT>
__global__ void __launch_bounds__(kPrepThreads) moe_prepare_kernel(PrepArgs a) {
    extern __shared__ int hist[];  // [E]
    if ((int)blockIdx.x < a.E) {
        sort_pairs(a, hist);
    } else {
        const unsigned i = (blockIdx.x - a.E) * kPrepThreads + threadIdx.x;
        if (i < a.n8) quant_padded8<FMT>(a.x, a.xq, a.xe, i, a.k8, a.q_stride, a.e_stride);
    }
}

// out[t, n] = sum_j weights[t, j] * y[t * k + j, n], j ascending, in fp32: y is
// kept in fp32, so that the sum is rounded once.  2048 tokens of four choices of
// 2880: 18 us for 106 MB, 5.9 TB/s (y from the last-level cache); 40 tokens 4.8.
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

// Whether each pair reads its expert's weights for itself (two launches)
// instead of sorting (four).  Sorting saves the weights of the experts that
// several pairs share, and its tiles stream at 5.9 TB/s against 5.0 (4.5 in e4m3,
// whose rows are taken apart pair by pair), for about 14 us more.  Both sides measured
// from 1 to 20 tokens at (E, k, H, I) = (128, 4, 2880, 2880), (32, 4, 2880, 1440) and
// (256, 8, 2048, 512): 1 token of the first 16.4 us against 30.7 (e2m1 14.5, 27.7);
// they cross at 16-20, 20-24 and 112-120 pairs (20, 24 and 128-160), where this does.
static bool moe_unsorted(const MoeArgs &a) {
    const double P = (double)a.T * a.k, E = a.E;
    const double shared = E * (1.0 - pow(1.0 - 1.0 / E, P));        // experts that P pairs meet
    const double expert_us = 3.0 * a.H * a.I * 17 / 32 * 1e-6;      // at 1 TB/s
    return P * expert_us / (a.fmt == kMxE4m3 ? 4.5 : 5.0) - shared * expert_us / 5.9 < 14.0 &&
           mxfp4_row_lds_bytes(a.fmt, a.H) <= kMxRowMaxLds &&
           a.k * mxfp4_row_lds_bytes(a.fmt, a.I) <= kMxRowMaxLds;
}

// Measured at the same sizes from 1 to 1024 tokens of e2m1: 16 and 32 rows differ
// by a few per cent up to 4 pairs an expert, 32 wins by 3-7 % to 16, and 64 from
// about 32 on (128 experts: 394 against 379 us there).  e4m3, in us at 16, 32 and
// 64 rows: 5 pairs an expert (32 of 2880 x 1440) 47, 51, 69; 12 50, 54, 74; 16 (128
// of 2880 x 2880) 342, 307, 356; 64 647, 537, 585; 128 1074, 869, 916; 512 513, 415,
// 416; 2048 1987, 1636, 1586.
int moe_tile_rows(int T, int k, int E, int fmt) {
    const long avg = (long)T * k / E;
    if (fmt == kMxE4m3) return avg <= 14 ? 16 : avg <= 640 ? 32 : 64;
    return avg <= 4 ? 16 : avg <= 24 ? 32 : 64;
}

// Whether the tiles of some experts may be taller than 64 rows: in e2m1, with
// enough of them that fewer, longer workgroups still fill the card.  4096 tokens of
// 128 experts of 2880 x 2880, 4 a token: 581 -> 546 us; 512 of 64 of 4096 x 1408, 8 a
// token: 162 -> 157, but 256: 130 -> 131; 1024 of 32 of 2880 x 1440: 104 -> 114.
static int moe_tall(const MoeArgs &a, int rows) {
    const long tiles = (long)a.T * a.k / 64 + a.E / 2;
    return a.fmt == kMxE2m1 && rows == 64 && tiles * ((a.I + 127) / 128) >= 4 * kNumCusMI355X;
}

int moe_way(const MoeArgs &a) {
    if (moe_unsorted(a)) return 0;
    const int rows = moe_tile_rows(a.T, a.k, a.E, a.fmt);
    return moe_tall(a, rows) ? 96 : rows;
}

size_t moe_workspace_bytes(int T, int k, int H, int I, int E, int fmt) {
    return moe_space(T, k, H, I, E, fmt).bytes;
}

int launch_moe(const MoeArgs &a, void *workspace, hipStream_t stream) {
    const MoeSpace s = moe_space(a.T, a.k, a.H, a.I, a.E, a.fmt);
    uint8_t *b = (uint8_t *)workspace;
    if (moe_unsorted(a)) return launch_moe_rows(a, b + s.h, b + s.he, stream);
    const int P = a.T * a.k, rows = moe_tile_rows(a.T, a.k, a.E, a.fmt);
    const int tiles = moe_max_tiles(P, a.E, rows);
    const MoeLists lists{(const MoeTile *)(b + s.tiles), (const int *)(b + s.count),
                         (const int *)(b + s.pairs), moe_tall(a, rows)};
    const unsigned n8 = (unsigned)((size_t)a.T * a.H / 8);
    const PrepArgs prep{a.x, b + s.xq, b + s.xe, n8, (unsigned)a.H / 8,
                        (unsigned)mx_code_stride(a.fmt, a.H), (unsigned)mx_scale_stride(a.H),
                        a.ids, P, a.E, rows, lists.tall, (int *)(b + s.pairs), (MoeTile *)(b + s.tiles),
                        (int *)(b + s.count)};
    const dim3 grid((unsigned)a.E + (n8 + kPrepThreads - 1) / kPrepThreads);
    if (a.fmt == kMxE4m3)
        hipLaunchKernelGGL(moe_prepare_kernel<kMxE4m3>, grid, dim3(kPrepThreads), (size_t)a.E * 4, stream, prep);
    else
        hipLaunchKernelGGL(moe_prepare_kernel<kMxE2m1>, grid, dim3(kPrepThreads), (size_t)a.E * 4, stream, prep);
    int e = (int)hipGetLastError();
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
