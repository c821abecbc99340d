/*
 * skinny_latent.h -- C ABI of latent attention on AMD MI355X (gfx950):
 * attention whose keys and values are linear functions of one latent vector a
 * token, which all heads share, beside the products of skinny_gemm.h that make
 * that vector (K = 7168, N = 576, or N = 2112 with the queries' own latent):
 *
 *   skinny_latent_append              norm and rotation of new tokens' latents
 *                                     into a paged cache, rotation of queries
 *   skinny_latent_attention           attention over that cache in the absorbed
 *                                     form: single tokens and chunks
 *   skinny_latent_attention_expanded  attention of prompts over expanded keys
 *                                     and values
 *   skinny_heads_gemm                 a product per head, into and out of the
 *                                     absorbed form
 *
 * One decode step of a layer, q = [T, H, 192], kv = [T, 576]:
 *   skinny_latent_append(kv, q[..., 128:]) -> cache, ql[..., 512:]
 *   skinny_heads_gemm(q[..., :128], Wk [H, 512, 128]) -> ql[..., :512]
 *   skinny_latent_attention(ql [T, H, 576]) -> o [T, H, 512]
 *   skinny_heads_gemm(o, Wv [H, 128, 512]) -> [T, H, 128]
 *
 * Conventions are skinny_gemm.h's: DEVICE tensors owned by the caller on the
 * current device, row-major, dense except where a stride is an argument (in
 * elements; the last dimension is always dense); work enqueued on `stream`
 * without synchronising; SKG_OK or a negative SKG_ERR_*, with every argument
 * checked on the host before any HIP call; outputs must not overlap inputs
 * (except where said) or each other, from their first value to their last;
 * tensors of the same strides may be different columns of one matrix.  Calls of one stream share its workspace
 * (skinny_latent_reserve); nothing is kept from one call for the next.
 */
#ifndef SKINNY_LATENT_H
#define SKINNY_LATENT_H

#include "skinny_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SKG_LATENT 512                             /* latent values of a cache row */
#define SKG_LATENT_ROPE 64                         /* then rotated ones */
#define SKG_LATENT_ROW (SKG_LATENT + SKG_LATENT_ROPE)
#define SKG_EXPANDED_NOPE 128                      /* expanded: a head's own key part */
#define SKG_EXPANDED_V 128                         /* and its value */
#define SKG_LATENT_MAX_B 8192
#define SKG_LATENT_MAX_H 1024

/* Which tokens are new, and where a sequence's rows lie.  Sequence b has
 * kv_lens[b] rows in the cache, its new tokens' among them: row p at
 * cache[table[b][p / page_size]][p % page_size].  Its new tokens are
 * q_starts[b] .. q_starts[b + 1] - 1 of the call's T (q_starts NULL: token b,
 * T == B), the last of them row kv_lens[b] - 1.
 * The contents are the device's and are not checked on the host.  Lengths are
 * taken between 0 and table_width * page_size, q_starts between 0 and T.  A
 * page outside [0, pages) holds no rows: nothing is written to it, and its keys
 * are not seen.  A new token that falls before row 0 has none and sees none.
 * Tokens of the call that belong to no sequence (behind the last one) are not
 * read, and their outputs are left as they were.  q_starts must not descend. */
typedef struct skinny_latent_batch {
    const int *table;    /* int32 [B, table_width] */
    const int *kv_lens;  /* int32 [B] */
    const int *q_starts; /* int32 [B + 1] or NULL */
    int B, T;            /* B <= 8192 */
    int table_width;     /* pages a sequence may have */
    int page_size;       /* rows a page: a power of two from 8 to 65536 */
    int pages;           /* pages of the cache */
} skinny_latent_batch;

#define SKG_ROPE_PAIRS 0  /* value 2i turns with value 2i + 1 */
#define SKG_ROPE_HALVES 1 /* value i turns with value i + 32 */

/* For every new token, c = kv[t][0:512], r = kv[t][512:576]:
 *   row = (c / sqrt(mean(c^2) + eps) * weight, rotated r), in fp64, rounded
 *   once to the cache's type: bf16, or e4m3 of row / *scale, clamped to +-448
 *   (NaN stays).  weight NULL: c as it is.
 * A pair (a, b) is turned by row p of `rotations` (fp32 [rotation_rows, 64],
 * 32 cosines, then 32 sines; p the token's row in its sequence) to
 * (a cos - b sin, a sin + b cos).
 * latent_out (NULL: none): bf16 [T, 576], the row unscaled.
 * q (NULL: none, H == 0): bf16 [T, H, 64], turned in fp32 into q_out, which may
 * be q itself with the same strides.
 * kv bf16 with kv_stride values from row to row; weight bf16 [512]; cache
 * [pages, page_size, 576] of cache_dtype (SKG_DTYPE_BF16, or SKG_DTYPE_FP8 with
 * scale, one fp32).  Strides are multiples of 8, tensors 16-byte aligned
 * (scale 4).  rotation_rows >= max(1, table_width * page_size); new tokens before row 0
 * are turned by row 0.  Two sequences that hold one page write to it in no order. */
int skinny_latent_append(const skinny_latent_batch *batch, const void *kv, long kv_stride,
                         const void *weight, float eps, const float *rotations, int rotation_rows,
                         int rope_style, void *cache, int cache_dtype, const float *scale,
                         void *latent_out, const void *q, long q_token_stride, long q_head_stride,
                         void *q_out, long out_token_stride, long out_head_stride, int H,
                         hipStream_t stream);

/* out[t, h] = sum_p w_p row_p[0:512], w = softmax over p of
 * softmax_scale * (q[t, h] . row_p), over the rows p of t's sequence up to its
 * own.  Rows of an e4m3 cache stand for code * *scale; softmax_scale * *scale may
 * leave fp32 where the scores themselves do not.  q bf16 [T, H, 576],
 * out bf16 [T, H, 512], dense.  Scores, maxima, sums and outputs are held in
 * fp32; the weights before their division, up to 2^8, are rounded to bf16 for the
 * matrix instruction.  So a value of the cache times its sequence's length must stay
 * below 2^119, and a sum of 576 products of queries and codes or values below 2^128.
 * A token that sees no row gets zeros.  A row that a token does not see has no
 * effect on it, whatever it holds; nor has what a page holds behind the
 * sequence's end.  Results do not depend on the order in which workgroups run.
 * 0 < softmax_scale <= 2e38.
 * All that the host knows of the lengths is table_width, by which it chooses how many
 * rows a workgroup takes where there are tiles enough: a table much wider than the
 * longest sequence costs time (128 tokens of 16 heads, 2 sequences of 2000 rows: 32 us,
 * with room for 100000 37) and may move an output by a rounding, as other sums are
 * joined. */
int skinny_latent_attention(const skinny_latent_batch *batch, const void *q, const void *cache,
                            int cache_dtype, const float *scale, float softmax_scale, void *out,
                            int H, hipStream_t stream);

/* Prompts in the expanded form: q bf16 [T, H, 192], kv bf16 [S, H, 256] (a head's
 * 128 key values, then its 128 values), k_rope bf16 [S, 64] with k_rope_stride
 * values from row to row (the rotated key that all heads share: columns 512 to
 * 575 of latent_out, say), out bf16 [T, H, 128].
 *   out[t, h] = sum_s w_s kv[s, h, 128:], w = softmax over s of
 *   softmax_scale * (q[t, h, :128] . kv[s, h, :128] + q[t, h, 128:] . k_rope[s]).
 * Sequence b has new tokens q_starts[b] .. q_starts[b + 1] - 1 and keys
 * kv_starts[b] .. kv_starts[b + 1] - 1 (int32 [B + 1] each, taken between 0 and
 * T or S, not descending).  causal: its last token sees all its keys, the one
 * before one fewer, and so on; else every token sees all.  Empty rows, unseen
 * keys, precision and order as above.  Tensors 16-byte aligned, k_rope_stride a
 * multiple of 8.  0 < softmax_scale <= 2e38. */
int skinny_latent_attention_expanded(const void *q, const void *kv, const void *k_rope,
                                     long k_rope_stride, const int *q_starts, const int *kv_starts,
                                     void *out, float softmax_scale, int causal, int B, int T,
                                     int S, int H, hipStream_t stream);

/* out[t, h, n] = sum_k x[t, h, k] * W[h, n, k], accumulated in fp32 and rounded
 * once.  x bf16 [T, H, K] and out bf16 [T, H, N] with strides from token to
 * token and from head to head, W bf16 [H, N, K] dense.  K % 32 == 0, K <= 512,
 * N % 8 == 0, N < 2^20, H <= 1024; strides multiples of 8, tensors 16-byte aligned.
 * T == 0 or N == 0 is a no-op. */
int skinny_heads_gemm(const void *x, long x_token_stride, long x_head_stride, const void *W,
                      void *out, long out_token_stride, long out_head_stride, int T, int H, int N,
                      int K, hipStream_t stream);

/* Workspace of `stream` for skinny_latent_attention calls of H heads, any B, T and
 * lengths, and for all skinny_latent_attention_expanded calls (those whose query
 * tokens are few for their keys use it).  It holds what workgroups that share a
 * sequence hand on.  As skinny_gemm_reserve: before graph capture. */
int skinny_latent_reserve(int H, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SKINNY_LATENT_H */
