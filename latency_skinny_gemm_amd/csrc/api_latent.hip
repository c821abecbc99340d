// api_latent.hip -- entry points of include/skinny_latent.h: argument checks on the
// host before any HIP call, workspace, launches.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "internal.h"
#include "latent_internal.h"
#include "spans.h"

using namespace skg;

namespace {

constexpr double kLog2e = 1.4426950408889634;
constexpr float kMostScale = 2e38f;  // times log2 e it is still a number of fp32

// A product of sizes that reach 2^31 each, at most `most`.
bool within(double product, double most) { return product <= most; }

int check_batch(const skinny_latent_batch *b) {
    if (!b || b->B < 0 || b->T < 0 || b->table_width < 0 || b->page_size < 1 || b->pages < 0) return SKG_ERR_INVALID_ARG;
    if (b->B > SKG_LATENT_MAX_B || b->page_size < 8 || b->page_size > 65536 || (b->page_size & (b->page_size - 1)) != 0 ||
        !within((double)b->table_width * b->page_size, 0x7FFFFF00))
        return SKG_ERR_UNSUPPORTED;
    if (!b->q_starts && b->T != b->B) return SKG_ERR_INVALID_ARG;
    return SKG_OK;
}
int check_batch_pointers(const skinny_latent_batch *b) {
    if ((!b->table && b->table_width > 0) || !b->kv_lens) return SKG_ERR_INVALID_ARG;
    if (!aligned(b->table, 4) || !aligned(b->kv_lens, 4) || !aligned(b->q_starts, 4)) return SKG_ERR_ALIGNMENT;
    return SKG_OK;
}
int shift_of(int page_size) { return __builtin_ctz((unsigned)page_size); }

// Bytes that T x H rows of n bf16 values reach over.
size_t strided_bytes(long T, long H, long ts, long hs, long n) {
    return T && H ? (size_t)((T - 1) * ts + (H - 1) * hs + n) * 2 : 0;
}
// Rows of n bf16 values, T tokens by H heads, with strides.
struct Rows {
    const void *p;
    long T, H, ts, hs, n;
    Span span() const { return {p, strided_bytes(T, H, ts, hs, n)}; }
};
// Blocks of a and b that begin at every multiple of one period do not meet.
bool blocks_apart(const Rows &a, long wa, const Rows &b, long wb, long period) {
    if (wa > period || wb > period) return false;
    const uintptr_t p = (uintptr_t)period * 2, x = (uintptr_t)a.p % p, y = (uintptr_t)b.p % p;
    const uintptr_t d = y >= x ? y - x : y + p - x;  // from a's blocks to b's
    return d >= (uintptr_t)wa * 2 && d + (uintptr_t)wb * 2 <= p;
}
// Whether two tensors share memory.  What their spans have in common may be columns of
// one matrix that both are slices of: by tokens, or by heads where these go on
// evenly from token to token.
bool overlap(const Rows &a, const Rows &b) {
    if (!overlap(a.span(), b.span())) return false;
    if (a.ts != b.ts || a.ts == 0) return true;
    if (blocks_apart(a, (a.H - 1) * a.hs + a.n, b, (b.H - 1) * b.hs + b.n, a.ts)) return false;
    const bool even = a.hs > 0 && a.hs == b.hs && a.ts % a.hs == 0;
    return !(even && blocks_apart(a, a.n, b, b.n, a.hs));
}
bool strides_ok(long ts, long hs) { return ts >= 0 && hs >= 0 && ts % 8 == 0 && hs % 8 == 0; }
// Rows of an output are apart: tokens outside of heads, or the other way round.
bool rows_apart(long T, long H, long ts, long hs, long n) {
    const bool inner_heads = (H < 2 || hs >= n) && (T < 2 || ts >= (H - 1) * hs + n);
    const bool inner_tokens = (T < 2 || ts >= n) && (H < 2 || hs >= (T - 1) * ts + n);
    return inner_heads || inner_tokens;
}
bool strides_fit(long T, long H, long ts, long hs) {
    return within((double)T * ts + (double)H * hs, (double)(1L << 40));
}

}  // namespace

extern "C" int skinny_latent_append(const skinny_latent_batch *batch, const void *kv, long kv_stride,
                                    const void *weight, float eps, const float *rotations,
                                    int rotation_rows, int rope_style, void *cache, int cache_dtype,
                                    const float *scale, void *latent_out, const void *q,
                                    long q_token_stride, long q_head_stride, void *q_out,
                                    long out_token_stride, long out_head_stride, int H,
                                    hipStream_t stream) {
    int rc = check_batch(batch);
    if (rc != SKG_OK) return rc;
    if ((rope_style != SKG_ROPE_PAIRS && rope_style != SKG_ROPE_HALVES) || rotation_rows < 0 || H < 0 || !(eps >= 0.0f) ||
        (cache_dtype != SKG_DTYPE_BF16 && cache_dtype != SKG_DTYPE_FP8) ||
        (scale != nullptr) != (cache_dtype == SKG_DTYPE_FP8) || (q == nullptr) != (q_out == nullptr) ||
        (q == nullptr) != (H == 0))
        return SKG_ERR_INVALID_ARG;
    const long T = batch->T, rows = (long)batch->pages * batch->page_size;
    if (kv_stride < SKG_LATENT_ROW || !strides_ok(kv_stride, 0) || (q && (!strides_ok(q_token_stride, q_head_stride) || !strides_ok(out_token_stride, out_head_stride))))
        return SKG_ERR_INVALID_ARG;
    if (H > SKG_LATENT_MAX_H || rotation_rows < (long)batch->table_width * batch->page_size ||
        !within((double)T * (4.0 * H + 64), 0x7FFFFFFF) || !strides_fit(T, 1, kv_stride, 0) ||
        (q && (!strides_fit(T, H, q_token_stride, q_head_stride) || !strides_fit(T, H, out_token_stride, out_head_stride))))
        return SKG_ERR_UNSUPPORTED;
    if (T == 0 || batch->B == 0) return SKG_OK;
    if (rotation_rows == 0) return SKG_ERR_UNSUPPORTED;  // tokens without a row are turned by the first
    rc = check_batch_pointers(batch);
    if (rc != SKG_OK) return rc;
    if (!kv || !rotations || (!cache && rows > 0)) return SKG_ERR_INVALID_ARG;
    if (q && !rows_apart(T, H, out_token_stride, out_head_stride, SKG_LATENT_ROPE)) return SKG_ERR_INVALID_ARG;
    if (!aligned(kv, 16) || !aligned(weight, 16) || !aligned(rotations, 16) || !aligned(cache, 16) || !aligned(scale, 4) ||
        !aligned(latent_out, 16) || !aligned(q, 16) || !aligned(q_out, 16))
        return SKG_ERR_ALIGNMENT;
    const bool e4m3 = cache_dtype == SKG_DTYPE_FP8;
    const bool in_place = q == q_out && q_token_stride == out_token_stride && q_head_stride == out_head_stride;
    const Rows kv_rows{kv, T, 1, kv_stride, 0, SKG_LATENT_ROW}, q_rows{q, T, H, q_token_stride, q_head_stride, SKG_LATENT_ROPE},
        q_out_rows{q_out, T, H, out_token_stride, out_head_stride, SKG_LATENT_ROPE};
    const Span written[] = {{cache, (size_t)rows * SKG_LATENT_ROW * (e4m3 ? 1 : 2)}, {latent_out, (size_t)T * SKG_LATENT_ROW * 2}};
    const Span outs[] = {written[0], written[1], q_out_rows.span()};
    const Span read[] = {kv_rows.span(), q_rows.span()};
    const Span ins[] = {{weight, SKG_LATENT * 2},
                        {rotations, (size_t)rotation_rows * SKG_LATENT_ROPE * 4},
                        {scale, 4},
                        {batch->table, (size_t)batch->B * batch->table_width * 4},
                        {batch->kv_lens, (size_t)batch->B * 4},
                        {batch->q_starts, ((size_t)batch->B + 1) * 4}};
    if (any_overlap(outs, ins) || any_overlap(written, read) || overlap(q_out_rows, kv_rows) ||
        (!in_place && overlap(q_out_rows, q_rows)))
        return SKG_ERR_INVALID_ARG;
    const LatentAppendArgs a{(const uint16_t *)kv, (const uint16_t *)weight, (const uint16_t *)q, rotations, scale,
                             batch->table, batch->kv_lens, batch->q_starts, (uint8_t *)cache, (uint16_t *)latent_out,
                             (uint16_t *)q_out, kv_stride, q_token_stride, q_head_stride, out_token_stride,
                             out_head_stride, eps, batch->B, batch->T, batch->table_width, shift_of(batch->page_size),
                             batch->pages, H};
    return hip_status(launch_latent_append(a, rope_style, e4m3, stream));
}

extern "C" int skinny_latent_attention(const skinny_latent_batch *batch, const void *q, const void *cache,
                                       int cache_dtype, const float *scale, float softmax_scale,
                                       void *out, int H, hipStream_t stream) {
    int rc = check_batch(batch);
    if (rc != SKG_OK) return rc;
    if (H < 1 || !(softmax_scale > 0.0f) || softmax_scale > kMostScale || (cache_dtype != SKG_DTYPE_BF16 && cache_dtype != SKG_DTYPE_FP8) ||
        (scale != nullptr) != (cache_dtype == SKG_DTYPE_FP8))
        return SKG_ERR_INVALID_ARG;
    if (H > SKG_LATENT_MAX_H || !within((double)batch->T * H, (double)(1L << 31))) return SKG_ERR_UNSUPPORTED;
    if (batch->T == 0 || batch->B == 0) return SKG_OK;
    rc = check_batch_pointers(batch);
    if (rc != SKG_OK) return rc;
    const long rows = (long)batch->pages * batch->page_size;
    if (!q || !out || (!cache && rows > 0)) return SKG_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(cache, 16) || !aligned(out, 16) || !aligned(scale, 4)) return SKG_ERR_ALIGNMENT;
    const bool e4m3 = cache_dtype == SKG_DTYPE_FP8;
    const size_t n = (size_t)batch->T * H;
    const Span outs[] = {{out, n * SKG_LATENT * 2}};
    const Span ins[] = {{q, n * SKG_LATENT_ROW * 2},
                        {cache, (size_t)rows * SKG_LATENT_ROW * (e4m3 ? 1 : 2)},
                        {scale, 4},
                        {batch->table, (size_t)batch->B * batch->table_width * 4},
                        {batch->kv_lens, (size_t)batch->B * 4},
                        {batch->q_starts, ((size_t)batch->B + 1) * 4}};
    if (any_overlap(outs, ins)) return SKG_ERR_INVALID_ARG;
    const int tile = latent_rows(batch->B, batch->T, H, (long)batch->table_width * batch->page_size, e4m3);
    float *ws = nullptr;
    unsigned *tk = nullptr;
    rc = acquire(stream, latent_workspace_bytes(tile, e4m3) / 4, 0, &ws, &tk);
    if (rc != SKG_OK) return rc;
    const LatentArgs a{(const uint16_t *)q, (const uint8_t *)cache, scale, batch->table, batch->kv_lens, batch->q_starts,
                       (uint16_t *)out, ws, (float)(softmax_scale * kLog2e), batch->B, batch->T, batch->table_width,
                       shift_of(batch->page_size), batch->pages, H};
    return hip_status(launch_latent_attention(a, e4m3, tile, stream));
}

extern "C" int skinny_latent_attention_expanded(const void *q, const void *kv, const void *k_rope,
                                                long k_rope_stride, const int *q_starts,
                                                const int *kv_starts, void *out, float softmax_scale,
                                                int causal, int B, int T, int S, int H,
                                                hipStream_t stream) {
    if (B < 0 || T < 0 || S < 0 || H < 1 || !(softmax_scale > 0.0f) || softmax_scale > kMostScale || (causal != 0 && causal != 1) ||
        k_rope_stride < SKG_LATENT_ROPE || k_rope_stride % 8 != 0)
        return SKG_ERR_INVALID_ARG;
    // a step's rows within 2 GiB of their first
    if (B > SKG_LATENT_MAX_B || H > SKG_LATENT_MAX_H || k_rope_stride > 1 << 24 || !within((double)T * H, 0x7FFFFFFF) ||
        !within(((double)T / 128 + B + 1) * H, (double)(1 << 23)))
        return SKG_ERR_UNSUPPORTED;
    if (B == 0 || T == 0) return SKG_OK;
    if (!q || !q_starts || !kv_starts || !out || (S > 0 && (!kv || !k_rope))) return SKG_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(kv, 16) || !aligned(k_rope, 16) || !aligned(out, 16) || !aligned(q_starts, 4) ||
        !aligned(kv_starts, 4))
        return SKG_ERR_ALIGNMENT;
    const size_t n = (size_t)T * H;
    const Span outs[] = {{out, n * SKG_EXPANDED_V * 2}};
    const Span ins[] = {{q, n * (SKG_EXPANDED_NOPE + SKG_LATENT_ROPE) * 2},
                        {kv, (size_t)S * H * (SKG_EXPANDED_NOPE + SKG_EXPANDED_V) * 2},
                        {k_rope, strided_bytes(S, 1, k_rope_stride, 0, SKG_LATENT_ROPE)},
                        {q_starts, ((size_t)B + 1) * 4},
                        {kv_starts, ((size_t)B + 1) * 4}};
    if (any_overlap(outs, ins)) return SKG_ERR_INVALID_ARG;
    const int parts = latent_expanded_parts(B, T, S, H);
    float *ws = nullptr;
    unsigned *tk = nullptr;
    if (parts > 1) {
        const int rc = acquire(stream, latent_expanded_workspace_bytes() / 4, 0, &ws, &tk);
        if (rc != SKG_OK) return rc;
    }
    const ExpandedArgs a{(const uint16_t *)q, (const uint16_t *)kv, (const uint16_t *)k_rope, q_starts, kv_starts,
                         (uint16_t *)out, k_rope_stride, (float)(softmax_scale * kLog2e), causal, B, T, S, H, parts, ws};
    return hip_status(launch_latent_expanded(a, stream));
}

extern "C" int skinny_heads_gemm(const void *x, long x_token_stride, long x_head_stride, const void *W,
                                 void *out, long out_token_stride, long out_head_stride, int T, int H,
                                 int N, int K, hipStream_t stream) {
    if (T < 0 || H < 1 || N < 0 || K < 0 || !strides_ok(x_token_stride, x_head_stride) ||
        !strides_ok(out_token_stride, out_head_stride))
        return SKG_ERR_INVALID_ARG;
    if (H > SKG_LATENT_MAX_H || K < 32 || K > 512 || K % 32 != 0 || N % 8 != 0 || N >= 1 << 20 ||
        !strides_fit(T, H, x_token_stride, x_head_stride) || !strides_fit(T, H, out_token_stride, out_head_stride) ||
        !within(((double)T / 128 + 1) * H * (N / 32 + 1), (double)(1 << 24)))
        return SKG_ERR_UNSUPPORTED;
    if (T == 0 || N == 0) return SKG_OK;
    if (!x || !W || !out || !rows_apart(T, H, out_token_stride, out_head_stride, N)) return SKG_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(W, 16) || !aligned(out, 16)) return SKG_ERR_ALIGNMENT;
    const Rows x_rows{x, T, H, x_token_stride, x_head_stride, K}, out_rows{out, T, H, out_token_stride, out_head_stride, N};
    if (overlap(out_rows, x_rows) || overlap(out_rows.span(), {W, (size_t)H * N * K * 2})) return SKG_ERR_INVALID_ARG;
    const HeadsArgs a{(const uint16_t *)x, (const uint16_t *)W, (uint16_t *)out, x_token_stride, x_head_stride,
                      out_token_stride, out_head_stride, T, H, N, K};
    return hip_status(launch_heads(a, stream));
}

// For the tests: the forms that calls take (the rows of a workgroup, the parts that
// share a tile's keys at most, whether rows of x come through a ring).
extern "C" int skg_latent_rows(int B, int T, int H, long capacity, int e4m3) { return latent_rows(B, T, H, capacity, e4m3 != 0); }
extern "C" int skg_latent_parts(int B, int T, int S, int H) { return latent_expanded_parts(B, T, S, H); }
extern "C" int skg_heads_ring(int T, int K, long x_token_stride) { return heads_ring(T, K, x_token_stride); }

extern "C" int skinny_latent_reserve(int H, hipStream_t stream) {
    if (H < 1) return SKG_ERR_INVALID_ARG;
    if (H > SKG_LATENT_MAX_H) return SKG_ERR_UNSUPPORTED;
    float *ws = nullptr;
    unsigned *tk = nullptr;
    const size_t bytes = std::max({latent_workspace_bytes(64, false), latent_workspace_bytes(32, true), latent_expanded_workspace_bytes()});
    return acquire(stream, bytes / 4, 0, &ws, &tk);
}
