// kernels_route.hip -- routing: the k best experts of each token by a score
// of its router logits, optionally from the best groups, and their weights.
//
// One wave holds a token: C keys per lane, expert c * 64 + lane.  Keys are
// compared as unsigned numbers that order as the floats do, so the largest
// over the wave is a chain of integer DPP maxima, and among equal keys the
// smallest index is a second chain.  0 marks a key out of the running; every
// real key, -inf included, lies above it.
#include "device_common.h"
#include "internal.h"
#include "moe_internal.h"
#include "mx_common.h"

namespace skg {

namespace {

struct RouteArgs {
    const void *logits;
    const float *bias;
    float *weights;
    int *ids;
    int T, E;
    int k, groups, top_groups, renormalize;
    float factor;
};

__device__ __forceinline__ float load_logit(const float *p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t *p) { return bf16_to_f32(*p); }

// Order-preserving bits; NaN as -inf, -0 as +0.
__device__ __forceinline__ unsigned order_of(float v) {
    if (v != v) v = -__builtin_inff();
    const unsigned u = __float_as_uint(v + 0.0f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float sigmoid(float l) { return 1.0f / (1.0f + expf(-l)); }

// Largest / smallest over the wave's 64 lanes, the same in every lane.
__device__ __forceinline__ unsigned wave_max(unsigned v) {
    v = max(v, dpp_u32<kDppQuadSwap1>(v));
    v = max(v, dpp_u32<kDppQuadSwap2>(v));
    v = max(v, dpp_u32<kDppHalfMirror>(v));
    v = max(v, dpp_u32<kDppMirror>(v));
    // readlane's type is int: back to unsigned before comparing
    const unsigned r0 = __builtin_amdgcn_readlane(v, 0), r1 = __builtin_amdgcn_readlane(v, 16);
    const unsigned r2 = __builtin_amdgcn_readlane(v, 32), r3 = __builtin_amdgcn_readlane(v, 48);
    return max(max(r0, r1), max(r2, r3));
}
__device__ __forceinline__ unsigned wave_min(unsigned v) { return ~wave_max(~v); }

__device__ __forceinline__ float wave_max_f(float v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor(v, d, 64));
    return v;
}

// A softmax term before its division: +inf against a +inf maximum is 1, and
// a row of -inf (or a NaN) is 0 rather than NaN.
__device__ __forceinline__ float softmax_term(float l, float m) {
    if (!(l > -__builtin_inff())) return 0.0f;
    return l == m ? 1.0f : expf(l - m);
}

}  // namespace

template <typename TL, int C, bool SIGMOID>
__global__ void __launch_bounds__(256) route_kernel(RouteArgs a) {
    extern __shared__ unsigned route_lds[];  // groups > 1: E keys per wave
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t = blockIdx.x * 4 + wave;
    if (t >= a.T) return;
    const TL *l = (const TL *)a.logits + (size_t)t * a.E;

    float v[C];
    unsigned key[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int e = c * 64 + lane;
        v[c] = e < a.E ? load_logit(l + e) : -__builtin_inff();
    }
    // softmax's maximum and, where the weights keep softmax's own division,
    // its sum; a bias goes on the divided scores
    float m = 0.0f, sum = 1.0f;
    if constexpr (!SIGMOID) {
        m = v[0];
#pragma unroll
        for (int c = 1; c < C; ++c) m = fmaxf(m, v[c]);
        m = wave_max_f(m);
        if (!a.renormalize || a.bias) {
            sum = 0.0f;
#pragma unroll
            for (int c = 0; c < C; ++c) sum += softmax_term(v[c], m);
            sum = wave_sum(sum);
        }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int e = c * 64 + lane;
        float s = v[c];
        if constexpr (SIGMOID) s = sigmoid(s);
        if (a.bias && e < a.E) {
            if constexpr (!SIGMOID) s = sum > 0.0f ? softmax_term(s, m) / sum : 0.0f;
            s += v[c] == v[c] ? a.bias[e] : 0.0f;
            if (v[c] != v[c]) s = -__builtin_inff();
        }
        key[c] = e < a.E ? order_of(s) : 0u;
    }

    if (a.groups > 1) {
        // lane l works on group l / per, `per` lanes (a power of two) each
        unsigned *ks = route_lds + wave * a.E;
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (c * 64 + lane < a.E) ks[c * 64 + lane] = key[c];
        // one wave's LDS operations complete in order; only the compiler must
        // not move the reads of other lanes' keys up
        asm volatile("" ::: "memory");
        const int size = a.E / a.groups;
        int per = 1;
        while (per * 2 * a.groups <= 64) per *= 2;
        const int g = lane / per, sub = lane % per;
        unsigned b1 = 0, b2 = 0;  // the two best keys
        if (g < a.groups)
            for (int i = sub; i < size; i += per) {
                const unsigned q = ks[g * size + i];
                b2 = max(b2, min(b1, q));
                b1 = max(b1, q);
            }
        for (int d = 1; d < per; d <<= 1) {
            const unsigned o1 = __shfl_xor(b1, d, 64), o2 = __shfl_xor(b2, d, 64);
            b2 = max(max(b2, o2), min(b1, o1));
            b1 = max(b1, o1);
        }
        unsigned score = b1;
        if (SIGMOID && size > 1) {
            const float f1 = __uint_as_float((b1 & 0x80000000u) ? b1 ^ 0x80000000u : ~b1);
            const float f2 = __uint_as_float((b2 & 0x80000000u) ? b2 ^ 0x80000000u : ~b2);
            score = order_of(f1 + f2);
        }
        int rank = 0;  // groups that go before this lane's
        for (int o = 0; o < a.groups; ++o) {
            const unsigned so = __builtin_amdgcn_readlane(score, o * per);
            rank += (so > score || (so == score && o < g)) ? 1 : 0;
        }
        const unsigned long long kept = __ballot(g < a.groups && rank < a.top_groups);
        const unsigned magic = (1u << 20) / (unsigned)size + 1u;  // e / size for e < 1024
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int e = c * 64 + lane;
            const int ge = (int)(((unsigned)e * magic) >> 20);
            if (e < a.E && !((kept >> (ge * per)) & 1ull)) key[c] = 0u;
        }
    }

    int chosen = 0;  // lane j < k: the j-th choice
    for (int j = 0; j < a.k; ++j) {
        unsigned best = key[0];
#pragma unroll
        for (int c = 1; c < C; ++c) best = max(best, key[c]);
        best = wave_max(best);
        unsigned at = 0xFFFFu;
#pragma unroll
        for (int c = C - 1; c >= 0; --c)
            if (key[c] == best) at = (unsigned)(c * 64 + lane);
        at = wave_min(at);
        if (lane == j) chosen = (int)at;
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (at == (unsigned)(c * 64 + lane)) key[c] = 0u;
    }

    if (lane < a.k) {
        const float lc = load_logit(l + chosen);
        float p;
        if constexpr (SIGMOID) p = lc == lc ? sigmoid(lc) : 0.0f;
        else p = softmax_term(lc, m);
        v[0] = p;
    } else {
        v[0] = 0.0f;
    }
    if (a.renormalize) sum = wave_sum(v[0]);
    if (lane < a.k) {
        const size_t o = (size_t)t * a.k + lane;
        float w = v[0];
        if (a.renormalize || !SIGMOID) w = sum > 0.0f ? w / sum : 0.0f;
        a.weights[o] = w * a.factor;
        a.ids[o] = chosen;
    }
}

namespace {

template <typename TL, int C>
int go(const RouteArgs &a, bool sigmoid, hipStream_t stream) {
    const dim3 grid((unsigned)((a.T + 3) / 4)), block(256);
    const size_t lds = a.groups > 1 ? (size_t)a.E * 16 : 0;
    if (sigmoid)
        hipLaunchKernelGGL((route_kernel<TL, C, true>), grid, block, lds, stream, a);
    else
        hipLaunchKernelGGL((route_kernel<TL, C, false>), grid, block, lds, stream, a);
    return (int)hipGetLastError();
}

template <typename TL>
int pick(const RouteArgs &a, bool sigmoid, hipStream_t stream) {
    const int c = (a.E + 63) / 64;
    if (c <= 1) return go<TL, 1>(a, sigmoid, stream);
    if (c <= 2) return go<TL, 2>(a, sigmoid, stream);
    if (c <= 4) return go<TL, 4>(a, sigmoid, stream);
    if (c <= 6) return go<TL, 6>(a, sigmoid, stream);
    if (c <= 8) return go<TL, 8>(a, sigmoid, stream);
    return go<TL, 16>(a, sigmoid, stream);
}

}  // namespace

int launch_route(const void *logits, int dtype, const float *bias, const skinny_route_options &o,
                 float *weights, int *ids, int T, int E, hipStream_t stream) {
    const RouteArgs a{logits, bias, weights, ids, T, E, o.k, o.groups, o.top_groups,
                      o.renormalize, o.factor};
    const bool sig = o.scores == SKG_SCORE_SIGMOID;
    return dtype == SKG_DTYPE_F32 ? pick<float>(a, sig, stream) : pick<uint16_t>(a, sig, stream);
}

}  // namespace skg
