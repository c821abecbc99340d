/*
 * skinny_moe.h -- C ABI of the operators around the small-M products of a
 * mixture-of-experts decode step on AMD MI355X (gfx950):
 *
 *   skinny_rmsnorm       residual addition and root-mean-square norm, with a
 *                        bf16, static e4m3 or MX e4m3 output
 *   skinny_route         router logits -> the chosen experts and weights
 *   skinny_quant_mx      bf16 -> MX codes (e4m3 or e2m1), skinny_dequant_mx back
 *   skinny_mxfp4_pack    row-major MXFP4 weights -> the products' layout
 *   skinny_gemm_mxfp4    product of few rows with an MXFP4 weight
 *   skinny_moe_mxfp4     the routed experts' feed-forward in MXFP4
 *
 * One step of a layer, with the products of skinny_gemm.h:
 *   skinny_rmsnorm -> skinny_gemm_bf16_f32 (router) -> skinny_route ->
 *   skinny_moe_mxfp4.
 *
 * Conventions are skinny_gemm.h's: dense row-major DEVICE tensors without
 * strides, owned by the caller, on the current device; work enqueued on
 * `stream` without synchronising; SKG_OK or a negative SKG_ERR_*, with every
 * argument checked on the host before any HIP call; outputs must not overlap
 * inputs (except where said) or each other.  Calls of one stream share its
 * workspace (skinny_moe_reserve); nothing is kept from one call for the next.
 *
 * MX (microscaling) tensors: 32 consecutive values of a row share one e8m0
 * byte e, the factor 2^(e - 127); 255 means NaN.  Codes are e4m3fn bytes, or
 * e2m1 (+-{0, 0.5, 1, 1.5, 2, 3, 4, 6}) two to a byte, the even index in the
 * low half.  Scales are row-major [rows][K / 32].
 */
#ifndef SKINNY_MOE_H
#define SKINNY_MOE_H

#include "skinny_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------ MX codes */
#define SKG_MX_E4M3 0 /* one byte a value */
#define SKG_MX_E2M1 4 /* half a byte a value */

/* q, e8m0 = MX codes of x.  Per block of 32: e is the smallest with
 * amax <= largest * 2^(e - 127) (largest code 448 or 6), at least 0; codes are
 * x * 2^(127 - e) rounded to nearest, ties to even; an all-zero block takes
 * e = 127, a block with an infinity or NaN e = 255 (the whole block is NaN).
 * x: bf16 [M, K], 16-byte aligned; q: [M, K] e4m3 or [M, K/2] e2m1 bytes,
 * 16-byte aligned; e8m0: [M, K/32].  K % 32 == 0, M * K < 2^31.  M == 0 is a
 * no-op. */
int skinny_quant_mx(const void *x, void *q, void *e8m0, int format, int M, int K,
                    hipStream_t stream);

/* out[m, k] = bf16(code * 2^(e - 127)): exact unless bf16's range is left. */
int skinny_dequant_mx(const void *q, const void *e8m0, int format, void *out, int M, int K,
                      hipStream_t stream);

/* ------------------------------------------------------------ norm */
#define SKG_NORM_BF16 0 /* y: bf16 */
#define SKG_NORM_E4M3 1 /* y: e4m3fn codes of y / *scale, clamped to +-448: what
                           skinny_gemm_fp8 takes with sx = scale */
#define SKG_NORM_MX 2   /* y: MX e4m3 codes with e8m0: what skinny_gemm_fp8 takes
                           in mode SKG_FP8_MX32, and skinny_gemm_mxfp4 */

/* s = x + residual (fp32; residual NULL: s = x), residual_out = bf16(s),
 * y = s / sqrt(mean_k(s^2) + eps) * weight, in fp32, rounded once to the
 * output's type.  The norm is of the fp32 sum, not of its bf16 rounding.  The
 * squares are added up in fp64, so that rows of any size have their norm.
 * x, residual, residual_out, (bf16 out) [M, K]; weight bf16 [K]; scale: one
 * fp32 (SKG_NORM_E4M3 only, else NULL); e8m0 [M, K/32] (SKG_NORM_MX only,
 * else NULL).  residual and residual_out are given together or not at all, and
 * residual_out may be the same memory as residual or x.  16-byte aligned
 * tensors (scale 4, e8m0 1).  K % 8 == 0 (MX: % 32), K <= 65536, M * K < 2^40,
 * eps >= 0. */
int skinny_rmsnorm(const void *x, const void *residual, const void *weight, float eps,
                   int out_format, const float *scale, void *y, void *e8m0, void *residual_out,
                   int M, int K, hipStream_t stream);

/* ------------------------------------------------------------ routing */
#define SKG_SCORE_SOFTMAX 0
#define SKG_SCORE_SIGMOID 1
#define SKG_ROUTE_MAX_E 1024
#define SKG_ROUTE_MAX_K 64
#define SKG_ROUTE_MAX_GROUPS 64

typedef struct skinny_route_options {
    int scores;      /* SKG_SCORE_* */
    int k;           /* experts chosen per token */
    int groups;      /* experts come in `groups` groups of E / groups (1: no groups) */
    int top_groups;  /* groups a token may choose from */
    int renormalize; /* 1: a token's weights are divided by their sum */
    float factor;    /* then multiplied by this */
} skinny_route_options;

/* Scores p = softmax(l) or sigmoid(l) of a token's logits l; the choice goes
 * by p + bias (by l for softmax without a bias, the same order without p's
 * rounding).  A group's value is the sum of its two best keys (sigmoid) or its
 * best key (softmax); the top_groups best groups stay.  The k best keys of
 * those are chosen, best first; equal keys and equal groups in the order of
 * their index.  weights[t, j] = p of the choice, without the bias, over the
 * sum of the chosen ones if renormalize, times factor; where that sum (or
 * softmax's) is 0 the weights are 0.
 * A NaN logit counts as -inf: chosen after every number, with weight 0; +inf
 * logits share softmax's whole weight.
 * logits: fp32 or bf16 [T, E] (dtype SKG_DTYPE_F32 or SKG_DTYPE_BF16); bias:
 * fp32 [E] or NULL; weights: fp32 [T, k]; ids: int32 [T, k].
 * 1 <= E <= 1024, k <= 64, groups <= 64, E % groups == 0,
 * k <= top_groups * (E / groups).  T == 0 is a no-op. */
int skinny_route(const void *logits, int dtype, const float *bias,
                 const skinny_route_options *options, float *weights, int *ids, int T, int E,
                 hipStream_t stream);

/* ------------------------------------------------------------ MXFP4 products */
/* Weights W[E, N, K] in MXFP4, laid out once for the products below: q
 * [E, N, K/2] and e8m0 [E, N, K/32] -> `packed`, skinny_mxfp4_packed_bytes
 * bytes, 16-byte aligned.  E == 1 for skinny_gemm_mxfp4.  K % 32 == 0, E <=
 * 65535, N and K < 2^20.  skinny_mxfp4_packed_bytes returns 0 for sizes out of
 * this domain. */
size_t skinny_mxfp4_packed_bytes(int E, int N, int K);
int skinny_mxfp4_pack(const void *q, const void *e8m0, void *packed, int E, int N, int K,
                      hipStream_t stream);

/* out[m, n] = sum_k x[m, k] * W[n, k] (+ bias[n]), accumulated in fp32 by the
 * scaled matrix instruction and rounded once to out_dtype (SKG_DTYPE_BF16 or
 * SKG_DTYPE_F32).  x is either bf16 [M, K] (x_e8m0 NULL), quantised here as by
 * skinny_quant_mx to x_format, or MX codes of x_format with their scales
 * x_e8m0.  bias: bf16 [N] or NULL.  1 <= M <= 512; x 16-byte aligned, out to
 * its type's size.  M == 0 or N == 0 is a no-op. */
int skinny_gemm_mxfp4(const void *x, const void *x_e8m0, int x_format, const void *packed,
                      const void *bias, void *out, int out_dtype, int M, int N, int K,
                      hipStream_t stream);

/* The routed experts' feed-forward, out bf16 [T, H]:
 *   out[t] = sum_j weights[t, j] * W2[e] . q( silu(g) * u ),  e = ids[t, j],
 *   (g, u) = W13[e] . q(x[t]),
 * q the MX quantisation to x_format, sums in fp32, one rounding to bf16.
 * x bf16 [T, H]; ids int32 [T, k]; weights fp32 [T, k]; W13 packed
 * [E, 2I, H] (I rows of g, then I of u); W2 packed [E, H, I].  A choice whose
 * id lies outside [0, E) contributes nothing (an expert held elsewhere); a
 * token with none left gets zeros.  H % 32 == 0, I % 32 == 0, E <= 1024,
 * k <= 64, T * k * max(H, I) * 4 < 2^40, and T * k, T * H and T * k * I at most
 * 2^31 - 1 with H and I rounded up to 128 there.
 * T == 0 is a no-op. */
int skinny_moe_mxfp4(const void *x, const int *ids, const float *weights, const void *w13,
                     const void *w2, void *out, int x_format, int T, int k, int H, int I, int E,
                     hipStream_t stream);

/* Workspace of `stream` for skinny_gemm_mxfp4 calls of up to max_M x max_K
 * (M, K; any N) and skinny_moe_mxfp4 calls of up to (max_T, k, H, I, E); either set of
 * sizes may be 0.  As skinny_gemm_reserve: before graph capture, and a larger
 * call outside capture grows it by itself, as told there.  The experts take about
 * T * (k * (4 * H + I) + H) bytes of it; a server reserves for its longest prompt. */
int skinny_moe_reserve(int max_M, int max_K, int max_T, int k, int H, int I, int E,
                       hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SKINNY_MOE_H */
