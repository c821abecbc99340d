// latent_internal.h -- arguments and launchers of the operators of
// include/skinny_latent.h.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "skinny_latent.h"

namespace skg {

struct LatentAppendArgs {
    const uint16_t *kv, *weight, *q;
    const float *rotations, *scale;
    const int *table, *kv_lens, *q_starts;
    uint8_t *cache;
    uint16_t *latent_out, *q_out;
    long kv_stride, q_token, q_head, o_token, o_head;
    float eps;
    int B, T, W, page_shift, pages, H;
};
int launch_latent_append(const LatentAppendArgs &a, int style, bool e4m3, hipStream_t stream);

struct LatentArgs {
    const uint16_t *q;
    const uint8_t *cache;
    const float *scale;  // e4m3 caches
    const int *table, *kv_lens, *q_starts;
    uint16_t *out;
    float *ws;
    float factor;  // softmax scale * log2 e
    int B, T, W, page_shift, pages, H;
};
// Rows (token, head) a workgroup takes at once: 32 or 64.  capacity: cache rows that a
// sequence's pages may hold.
int latent_rows(int B, int T, int H, long capacity, bool e4m3);
size_t latent_workspace_bytes(int rows, bool e4m3);
int launch_latent_attention(const LatentArgs &a, bool e4m3, int rows, hipStream_t stream);

struct ExpandedArgs {
    const uint16_t *q, *kv, *k_rope;
    const int *q_starts, *kv_starts;
    uint16_t *out;
    long rope_stride;
    float factor;
    int causal, B, T, S, H;
    int parts;  // workgroups that share a tile's keys, at most
    float *ws;  // parts > 1
};
int latent_expanded_parts(int B, int T, int S, int H);
size_t latent_expanded_workspace_bytes();
int launch_latent_expanded(const ExpandedArgs &a, hipStream_t stream);

struct HeadsArgs {
    const uint16_t *x, *W;
    uint16_t *out;
    long xt, xh, ot, oh;
    int T, H, N, K;
};
bool heads_ring(int T, int K, long x_token_stride);  // x through an LDS ring, else straight from memory
int launch_heads(const HeadsArgs &a, hipStream_t stream);

}  // namespace skg
