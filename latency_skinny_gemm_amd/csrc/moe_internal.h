// moe_internal.h -- shapes, layouts and launchers of the operators of
// include/skinny_moe.h.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "skinny_moe.h"

namespace skg {

// ---------------------------------------------------------------- MXFP4 layout
// Weights in column groups of 16, K in steps of 128 (one matrix instruction)
// and chunks of 4 steps (one dword of scale bytes per lane); see
// kernels_mx.hip.
constexpr int mxfp4_groups(int N) { return (N + 15) / 16; }
constexpr int mxfp4_steps(int K) { return (K + 127) / 128; }
constexpr int mxfp4_chunks(int K) { return (mxfp4_steps(K) + 3) / 4; }
constexpr size_t mxfp4_group_bytes(int K) {
    return (size_t)mxfp4_steps(K) * 1024 + (size_t)mxfp4_chunks(K) * 256;
}
constexpr size_t mxfp4_packed_bytes(int E, int N, int K) {
    return (size_t)E * mxfp4_groups(N) * mxfp4_group_bytes(K);
}
// Scale rows of quantised activations in a workspace: whole 16-byte pieces,
// one a chunk.
constexpr int mx_scale_stride(int K) { return mxfp4_chunks(K) * 16; }
// Their code rows: whole steps, and whole 128-byte lines, so that a line is
// asked for once.
constexpr int mx_code_stride(int fmt, int K) {
    return fmt == SKG_MX_E4M3 ? mxfp4_steps(K) * 128 : (mxfp4_steps(K) + 1) / 2 * 128;
}

// ---------------------------------------------------------------- launchers
// Each returns a hipError_t as int.  fmt: kMxE4m3 or kMxE2m1.
// padded: rows of mx_code_stride and mx_scale_stride bytes, else dense ones.
int launch_quant_mx(const void *x, void *q, void *e8, int fmt, int M, int K, bool padded,
                    hipStream_t stream);
int launch_dequant_mx(const void *q, const void *e8, int fmt, void *out, int M, int K,
                      hipStream_t stream);
int launch_pad_scales(const void *e8, void *out, int M, int K, hipStream_t stream);
int launch_mxfp4_pack(const void *q, const void *e8, void *out, int E, int N, int K,
                      hipStream_t stream);
int launch_rmsnorm(const void *x, const void *residual, const void *weight, float eps,
                   int out_format, const float *scale, void *y, void *e8, void *residual_out,
                   int M, int K, hipStream_t stream);
int launch_route(const void *logits, int dtype, const float *bias, const skinny_route_options &o,
                 float *weights, int *ids, int T, int E, hipStream_t stream);

// A product with packed weights.
struct Mxfp4Args {
    const uint8_t *x;   // bf16 rows (xe null) or codes
    int xs;             // codes: bytes from row to row
    const uint8_t *xe;  // scale bytes, es a row
    int es;
    int fmt;
    const uint8_t *W;
    const uint16_t *bias;
    void *out;
    int out_f32;
    int M, N, K;
};
// Codes with padded scale rows, any number of rows.
int launch_mxfp4(const Mxfp4Args &a, hipStream_t stream);
// Blocks of few rows, a workgroup each for 16 columns: codes, or bf16 rows
// quantised on the way.
constexpr int kMxRowsBf16 = 16, kMxRowsCodes = 32;
int launch_mxfp4_rows(const Mxfp4Args &a, int blocks, hipStream_t stream);
// The tile that a product of this size takes, as dense() lists them.
int dense_tile(int M, int N, int fmt);
// Time in us of the tiles, quantising included.
double mxfp4_tile_time(int M, int N, int K, int fmt);

// ---------------------------------------------------------------- experts
// Pairs (token, choice) sorted by expert, and the row tiles of the grouped
// products.
// A tile's expert, whole: its tiles are first .. first + ceil(rows / height) - 1,
// over sorted rows row .. row + rows - 1.
struct MoeTile {
    int expert;
    int row;
    int rows;
    int first;
};
// Rows a tile may hold, by the average number of pairs an expert gets.
int moe_tile_rows(int T, int k, int E, int fmt);
// The height of the tiles of an expert with n rows: 96 (tall) instead of 64 where
// that makes fewer of them, and so fewer readings of its weights.
#ifdef __HIPCC__
__host__ __device__
#endif
constexpr int moe_tile_height(int n, int rows, int tall) {
    return tall && (n + 95) / 96 < (n + 63) / 64 ? 96 : rows;
}
// The most tiles of that height the pairs can make.
constexpr int moe_max_tiles(long P, int E, int rows) {
    return (int)((P < E ? P : E) + P / rows);
}

struct MoeArgs {
    const uint16_t *x;      // bf16 [T][H]
    const int *ids;         // [T][k]
    const float *weights;   // [T][k]
    const uint8_t *W13;     // packed [E][2I][H]
    const uint8_t *W2;      // packed [E][H][I]
    uint16_t *out;          // bf16 [T][H]
    int fmt;
    int T, k, H, I, E;
};
struct MoeLists {
    const MoeTile *tiles;
    const int *count;  // tiles in use
    const int *pairs;  // sorted row -> pair t * k + j
    int tall;          // tiles of 64 rows may be 96 high
};
// rows: height of the tiles (16, 32 or 64); tiles: bound on their number.
int launch_moe_gate_up(const MoeArgs &m, const MoeLists &s, const uint8_t *xq, const uint8_t *xe,
                       uint8_t *h, uint8_t *he, int rows, int tiles, hipStream_t stream);
int launch_moe_down(const MoeArgs &m, const MoeLists &s, const uint8_t *h, const uint8_t *he,
                    float *y, int rows, int tiles, hipStream_t stream);
// LDS of a row's codes and scale bytes, in whole steps, and the most of it.
// The pad puts the same piece of neighbouring rows into different banks.
constexpr int kRowLdsPad = 64;
constexpr size_t mxfp4_row_lds_bytes(int fmt, int K) {
    return (size_t)mxfp4_steps(K) * ((fmt == SKG_MX_E4M3 ? 128 : 64) + 4) + kRowLdsPad;
}
constexpr size_t kMxRowMaxLds = 124 * 1024;
// How a call is done: 0 unsorted, else the height of its tiles (96: some of them).
int moe_way(const MoeArgs &a);
// Few pairs, unsorted: h and he have a row per pair; combines as well.
int launch_moe_rows(const MoeArgs &m, uint8_t *h, uint8_t *he, hipStream_t stream);
// Bytes of workspace the experts need.
size_t moe_workspace_bytes(int T, int k, int H, int I, int E, int fmt);
int launch_moe(const MoeArgs &a, void *workspace, hipStream_t stream);

}  // namespace skg
