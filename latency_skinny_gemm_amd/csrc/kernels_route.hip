// kernels_route.hip -- routing: the k best experts of each token by a score
// of its router logits, optionally from the best groups, and their weights.
//
// Keys are compared as unsigned numbers that order as the floats do.  0 marks
// a key out of the running; every real key, -inf included, lies above it.
// Two kernels: sorted lists with 16 lanes to a token (k up to 8), and one
// choice at a time with a wave to a token (the rest).  Both are bound by
// vector instructions, not by memory: 16384 tokens of 384 bf16 logits take
// 8.4 us where their 14 MB would take 3; up to 512 tokens they take what a
// launch and the chain of dependent steps take, 3 to 5 us.
#include <algorithm>
#include <type_traits>

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

// ---------------------------------------------------------------- sorted lists

namespace {

constexpr int kList = 8;          // best keys a lane keeps
constexpr int kTokenLanes = 16;   // one row of DPP
constexpr int kChunk = kList * kTokenLanes;

// A key and its expert in one number, so that one maximum and one minimum
// exchange two of them and equal keys order by their index.  Keys of bf16
// logits fill the upper half of 32 bits; other keys and their index are the
// mantissa of a double in [1, 2), which a maximum of doubles passes on bit for
// bit (the vector unit does it at the rate of fp32).
__device__ __forceinline__ void pack_key(unsigned &k, unsigned order, unsigned e) {
    k = (order & 0xFFFF0000u) | (0xFFFFu - e);
}
__device__ __forceinline__ void pack_key(double &k, unsigned order, unsigned e) {
    k = __longlong_as_double(0x3FF0000000000000ll | (long long)order << 20 | (0xFFFFFu - e));
}
__device__ __forceinline__ void no_key(unsigned &k) { k = 0u; }
__device__ __forceinline__ void no_key(double &k) { k = 1.0; }
__device__ __forceinline__ int key_expert(unsigned k) { return (int)(0xFFFFu - (k & 0xFFFFu)); }
__device__ __forceinline__ int key_expert(double k) {
    return (int)(0xFFFFFu - ((unsigned)__double_as_longlong(k) & 0xFFFFFu));
}
__device__ __forceinline__ unsigned key_order(unsigned k) {
    return (k & 0x80000000u) ? k & 0xFFFF0000u : k | 0xFFFFu;
}
__device__ __forceinline__ unsigned key_order(double k) {
    return (unsigned)((unsigned long long)__double_as_longlong(k) >> 20);
}
__device__ __forceinline__ float value_of(unsigned order) {
    return __uint_as_float((order & 0x80000000u) ? order ^ 0x80000000u : ~order);
}

__device__ __forceinline__ unsigned key_max(unsigned a, unsigned b) { return max(a, b); }
__device__ __forceinline__ unsigned key_min(unsigned a, unsigned b) { return min(a, b); }
// by the instruction: the library call adds one to each operand to quiet NaN
__device__ __forceinline__ double key_max(double a, double b) {
    double r;
    asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
__device__ __forceinline__ double key_min(double a, double b) {
    double r;
    asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
template <int CTRL>
__device__ __forceinline__ unsigned key_dpp(unsigned k) { return dpp_u32<CTRL>(k); }
template <int CTRL>
__device__ __forceinline__ double key_dpp(double k) {
    const unsigned long long u = (unsigned long long)__double_as_longlong(k);
    const unsigned lo = dpp_u32<CTRL>((unsigned)u), hi = dpp_u32<CTRL>((unsigned)(u >> 32));
    return __longlong_as_double((long long)((unsigned long long)hi << 32 | lo));
}

template <typename K>
__device__ __forceinline__ void exchange(K &a, K &b) {  // the larger into a
    const K hi = key_max(a, b);
    b = key_min(a, b);
    a = hi;
}

// Eight keys, largest first: odd-even merge sort, 19 exchanges.
template <typename K>
__device__ __forceinline__ void sort8(K (&v)[kList]) {
    constexpr int at[19][2] = {{0, 1}, {2, 3}, {4, 5}, {6, 7}, {0, 2}, {1, 3}, {4, 6}, {5, 7}, {1, 2}, {5, 6},
                               {0, 4}, {1, 5}, {2, 6}, {3, 7}, {2, 4}, {3, 5}, {1, 2}, {3, 4}, {5, 6}};
#pragma unroll
    for (int i = 0; i < 19; ++i) exchange(v[at[i][0]], v[at[i][1]]);
}

// a = the eight best of the sorted lists a and b: the larger of a[i] and
// b[7 - i] is a bitonic sequence of them, which three halvings sort.
template <typename K>
__device__ __forceinline__ void merge8(K (&a)[kList], const K (&b)[kList]) {
#pragma unroll
    for (int i = 0; i < kList; ++i) a[i] = key_max(a[i], b[kList - 1 - i]);
#pragma unroll
    for (int d = 4; d > 0; d >>= 1)
#pragma unroll
        for (int i = 0; i < kList; ++i)
            if (!(i & d)) exchange(a[i], a[i + d]);
}
template <int CTRL, typename K>
__device__ __forceinline__ void merge_lanes(K (&a)[kList]) {
    K b[kList];
#pragma unroll
    for (int i = 0; i < kList; ++i) b[i] = key_dpp<CTRL>(a[i]);
    merge8(a, b);
}

template <int CTRL>
__device__ __forceinline__ float dpp_f(float v) { return __uint_as_float(dpp_u32<CTRL>(__float_as_uint(v))); }
// Sum and largest over a token's 16 lanes, the same in each.
__device__ __forceinline__ float token_sum(float v) {
    v += dpp_f<kDppQuadSwap1>(v);
    v += dpp_f<kDppQuadSwap2>(v);
    v += dpp_f<kDppHalfMirror>(v);
    return v + dpp_f<kDppMirror>(v);
}
__device__ __forceinline__ float token_max(float v) {
    v = fmaxf(v, dpp_f<kDppQuadSwap1>(v));
    v = fmaxf(v, dpp_f<kDppQuadSwap2>(v));
    v = fmaxf(v, dpp_f<kDppHalfMirror>(v));
    return fmaxf(v, dpp_f<kDppMirror>(v));
}

// A lane's eight experts of chunk c: neighbours (VEC), or 16 apart.
template <bool VEC>
__device__ __forceinline__ int list_expert(int c, int sub, int i) {
    return c * kChunk + (VEC ? sub * kList + i : i * kTokenLanes + sub);
}
// Their values; those past E, -inf (VEC: E is a multiple of 8).
template <bool VEC>
__device__ __forceinline__ void list_load(const float *l, int E, int c, int sub, float (&v)[kList]) {
    if constexpr (VEC) {
        const int e = min(c * kChunk + sub * kList, E - kList);
        const f32x4 a = *reinterpret_cast<const f32x4 *>(l + e), b = *reinterpret_cast<const f32x4 *>(l + e + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = a[i], v[i + 4] = b[i];
    } else {
#pragma unroll
        for (int i = 0; i < kList; ++i) v[i] = l[min(list_expert<false>(c, sub, i), E - 1)];
    }
}
template <bool VEC>
__device__ __forceinline__ void list_load(const uint16_t *l, int E, int c, int sub, float (&v)[kList]) {
    if constexpr (VEC) {
        bf16x8_to_f32(*reinterpret_cast<const u32x4 *>(l + min(c * kChunk + sub * kList, E - kList)), v);
    } else {
#pragma unroll
        for (int i = 0; i < kList; ++i) v[i] = bf16_to_f32(l[min(list_expert<false>(c, sub, i), E - 1)]);
    }
}

struct Softmax {
    float m, sum;
};

// The order of a score: l itself, sigmoid(l), or either probability + bias.
template <bool SIGMOID, bool BIAS>
__device__ __forceinline__ unsigned score_order(float l, float bias, const Softmax &sm) {
    float s = l;
    if constexpr (SIGMOID) s = sigmoid(l);
    if constexpr (BIAS) {
        if constexpr (!SIGMOID) s = sm.sum > 0.0f ? softmax_term(l, sm.m) / sm.sum : 0.0f;
        s = l == l ? s + bias : -__builtin_inff();
    }
    return order_of(s);
}

}  // namespace

// Sixteen lanes to a token, four tokens to a wave.  A lane sorts eight keys at
// a time and keeps the best eight it has seen; four merges with the lists of
// its neighbours then leave the token's eight best, in order, in every lane.
// One instruction serves four tokens at every step, and no step waits for the
// one before it across the wave.
// GROUPS (E / groups a multiple of 8, so that a lane's eight experts share a
// group): a first pass leaves the two best keys of every eight in LDS, from
// which the groups are ranked; the second takes the kept ones.
template <typename TL, typename K, bool SIGMOID, bool BIAS, bool VEC, bool GROUPS>
__global__ void __launch_bounds__(256) route_lists_kernel(RouteArgs a) {
    extern __shared__ unsigned route_lds[];  // GROUPS: per token E / 8 pairs of keys, 64 scores
    const int sub = threadIdx.x % kTokenLanes, local = threadIdx.x / kTokenLanes;
    const int token = blockIdx.x * (256 / kTokenLanes) + local;
    const int t = min(token, a.T - 1);  // lanes past the last token repeat it and store nothing
    const TL *l = (const TL *)a.logits + (size_t)t * a.E;
    const int chunks = (a.E + kChunk - 1) / kChunk;
    float v[kList];

    Softmax sm{0.0f, 1.0f};
    // softmax's own division is needed before a bias, or for the weights
    if (!SIGMOID && (BIAS || !a.renormalize)) {
        sm.m = -__builtin_inff();
        for (int c = 0; c < chunks; ++c) {
            list_load<VEC>(l, a.E, c, sub, v);  // values seen twice do no harm here
#pragma unroll
            for (int i = 0; i < kList; ++i) sm.m = fmaxf(sm.m, v[i]);
        }
        sm.m = token_max(sm.m);
        sm.sum = 0.0f;
        for (int c = 0; c < chunks; ++c) {
            list_load<VEC>(l, a.E, c, sub, v);
#pragma unroll
            for (int i = 0; i < kList; ++i)
                sm.sum += list_expert<VEC>(c, sub, i) < a.E ? softmax_term(v[i], sm.m) : 0.0f;
        }
        sm.sum = token_sum(sm.sum);
    }

    unsigned long long kept = ~0ull;
    unsigned magic = 0;
    if constexpr (GROUPS) {
        const int size = a.E / a.groups, blocks = a.E / kList, per = size / kList;
        magic = (1u << 20) / (unsigned)size + 1u;  // e / size for e < 1024
        unsigned *mine = route_lds + local * (2 * blocks + SKG_ROUTE_MAX_GROUPS), *score = mine + 2 * blocks;
        for (int c = 0; c < chunks; ++c) {
            const int e = c * kChunk + sub * kList;
            list_load<VEC>(l, a.E, c, sub, v);
            unsigned b1 = 0, b2 = 0;
#pragma unroll
            for (int i = 0; i < kList; ++i) {
                const float b = BIAS ? a.bias[min(e, a.E - kList) + i] : 0.0f;
                const unsigned q = score_order<SIGMOID, BIAS>(v[i], b, sm);
                b2 = max(b2, min(b1, q));
                b1 = max(b1, q);
            }
            if (e < a.E) {
                mine[2 * (e / kList)] = b1;
                mine[2 * (e / kList) + 1] = b2;
            }
        }
        // a token's lanes are one wave's, whose LDS operations complete in
        // order; only the compiler must not move the reads up
        asm volatile("" ::: "memory");
        for (int g = sub; g < a.groups; g += kTokenLanes) {
            unsigned b1 = 0, b2 = 0;
            for (int i = 0; i < per; ++i) {
                const unsigned o1 = mine[2 * (g * per + i)], o2 = mine[2 * (g * per + i) + 1];
                b2 = max(max(b2, o2), min(b1, o1));
                b1 = max(b1, o1);
            }
            score[g] = SIGMOID ? order_of(value_of(b1) + value_of(b2)) : b1;
        }
        asm volatile("" ::: "memory");
        kept = 0;
        for (int g0 = 0; g0 < a.groups; g0 += kTokenLanes) {
            const int g = g0 + sub;
            const unsigned s = g < a.groups ? score[g] : 0u;
            int rank = 0;  // groups that go before this lane's
            for (int o = 0; o < a.groups; ++o) {
                const unsigned so = score[o];
                rank += (so > s || (so == s && o < g)) ? 1 : 0;
            }
            const unsigned long long b = __ballot(g < a.groups && rank < a.top_groups);
            kept |= ((b >> (threadIdx.x & 48)) & 0xFFFFull) << g0;
        }
    }

    K best[kList];
#pragma unroll
    for (int i = 0; i < kList; ++i) no_key(best[i]);
    float next[kList];
    list_load<VEC>(l, a.E, 0, sub, next);
    for (int c = 0; c < chunks; ++c) {
#pragma unroll
        for (int i = 0; i < kList; ++i) v[i] = next[i];
        if (c + 1 < chunks) list_load<VEC>(l, a.E, c + 1, sub, next);
        bool in = true;
        if constexpr (GROUPS)
            in = (kept >> (((unsigned)min(c * kChunk + sub * kList, a.E - kList) * magic) >> 20)) & 1ull;
        K key[kList];
#pragma unroll
        for (int i = 0; i < kList; ++i) {
            const int e = list_expert<VEC>(c, sub, i);
            const float b = BIAS ? a.bias[min(e, a.E - 1)] : 0.0f;
            pack_key(key[i], score_order<SIGMOID, BIAS>(v[i], b, sm), (unsigned)e);
            if (e >= a.E || !in) no_key(key[i]);
        }
        sort8(key);
        if (c == 0) {
#pragma unroll
            for (int i = 0; i < kList; ++i) best[i] = key[i];
        } else {
            merge8(best, key);
        }
    }
    merge_lanes<kDppQuadSwap1>(best);
    merge_lanes<kDppQuadSwap2>(best);
    merge_lanes<kDppHalfMirror>(best);
    merge_lanes<kDppMirror>(best);

    K mine = best[0];  // lane j < k: the j-th choice
#pragma unroll
    for (int i = 1; i < kList; ++i)
        if (sub == i) mine = best[i];
    const bool chosen = sub < a.k;
    const int e = key_expert(mine);
    float p = 0.0f;
    if (chosen) {
        // the score that was ordered, or the logit below a bias
        const float s = BIAS ? load_logit(l + e) : value_of(key_order(mine));
        if constexpr (!SIGMOID)
            p = softmax_term(s, BIAS || !a.renormalize ? sm.m : value_of(key_order(best[0])));
        else
            p = BIAS ? (s == s ? sigmoid(s) : 0.0f) : (s > 0.0f ? s : 0.0f);
    }
    const float sum = a.renormalize ? token_sum(p) : sm.sum;
    if (chosen && token < a.T) {
        const size_t o = (size_t)t * a.k + sub;
        if (a.renormalize || !SIGMOID) p = sum > 0.0f ? p / sum : 0.0f;
        a.weights[o] = p * a.factor;
        a.ids[o] = e;
    }
}

// ---------------------------------------------------------------- choice by choice

// One wave holds a token: C keys per lane, expert c * 64 + lane.  Each choice
// is a chain of integer DPP maxima over the wave, and among equal keys the
// smallest index is a second chain.
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
            score = order_of(value_of(b1) + value_of(b2));
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

template <typename TL, typename K, bool SIGMOID, bool BIAS>
int lists(const RouteArgs &a, bool vec, hipStream_t stream) {
    constexpr int tokens = 256 / kTokenLanes;
    const dim3 grid((unsigned)((a.T + tokens - 1) / tokens)), block(256);
    if (a.groups > 1) {
        const size_t lds = (size_t)tokens * (2 * (a.E / kList) + SKG_ROUTE_MAX_GROUPS) * 4;
        hipLaunchKernelGGL((route_lists_kernel<TL, K, SIGMOID, BIAS, true, true>), grid, block, lds, stream, a);
    } else if (vec) {
        hipLaunchKernelGGL((route_lists_kernel<TL, K, SIGMOID, BIAS, true, false>), grid, block, 0, stream, a);
    } else {
        hipLaunchKernelGGL((route_lists_kernel<TL, K, SIGMOID, BIAS, false, false>), grid, block, 0, stream, a);
    }
    return (int)hipGetLastError();
}

template <typename TL>
int pick(const RouteArgs &a, bool sigmoid, hipStream_t stream) {
    // whole 16-byte vectors of logits in every row
    const bool vec = a.E % kList == 0 && ((uintptr_t)a.logits & 15) == 0;
    const bool grouped = a.groups > 1;
    // Choice by choice against lists, in us at 1, 512, 4096 and 16384 tokens:
    // 384 bf16 logits, 8 chosen       4.6 5.1 7.1 19.2    3.6 3.9 4.1  8.2
    // 256 fp32, sigmoid and bias      4.3 4.9 6.6 17.7    4.6 4.9 5.2 14.2
    // the same in 8 groups            5.4 6.2 8.4 22.5    6.7 7.2 7.7 16.2
    // 256 fp32, softmax's division    4.1 4.8 6.5 17.1    5.2 5.6 5.8 11.9
    // so lists that read the logits twice are for many tokens only.
    const bool twice = grouped || (!sigmoid && (a.bias || !a.renormalize));
    if (a.k <= kList && (!grouped || (vec && a.E / a.groups % kList == 0)) && (!twice || a.T >= 2048)) {
        if (sigmoid)
            return a.bias ? lists<TL, double, true, true>(a, vec, stream)
                          : lists<TL, double, true, false>(a, vec, stream);
        if (a.bias) return lists<TL, double, false, true>(a, vec, stream);
        // the logits themselves are the keys
        typedef typename std::conditional<sizeof(TL) == 2, unsigned, double>::type K;
        return lists<TL, K, false, false>(a, vec, stream);
    }
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
    const bool sig = o.scores == SKG_SCORE_SIGMOID, f32 = dtype == SKG_DTYPE_F32;
    // a grid has fewer than 2^32 work-items: 2^21 tokens of up to 64 lanes at a time
    constexpr int kMostTokens = 1 << 21;
    for (size_t t0 = 0; t0 < (size_t)T; t0 += kMostTokens) {
        const RouteArgs a{(const uint8_t *)logits + t0 * E * (f32 ? 4 : 2), bias, weights + t0 * o.k, ids + t0 * o.k,
                          (int)std::min<size_t>(T - t0, kMostTokens), E, o.k, o.groups, o.top_groups,
                          o.renormalize, o.factor};
        const int e = f32 ? pick<float>(a, sig, stream) : pick<uint16_t>(a, sig, stream);
        if (e != (int)hipSuccess) return e;
    }
    return (int)hipSuccess;
}

}  // namespace skg
