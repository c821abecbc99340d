// api_moe.hip -- entry points of include/skinny_moe.h: argument checks on the
// host before any HIP call, workspace, launches.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "internal.h"
#include "moe_internal.h"
#include "mx_common.h"

using namespace skg;

namespace {

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// A tensor's memory, for the overlap checks (null: none).
struct Span {
    const void *p;
    size_t bytes;
};
bool overlap(Span a, Span b) {
    if (!a.p || !b.p || !a.bytes || !b.bytes) return false;
    const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}
template <size_t N, size_t L>
bool any_overlap(const Span (&outs)[N], const Span (&ins)[L]) {
    for (size_t i = 0; i < N; ++i) {
        for (size_t j = i + 1; j < N; ++j)
            if (overlap(outs[i], outs[j])) return true;
        for (const Span &s : ins)
            if (overlap(outs[i], s)) return true;
    }
    return false;
}

bool format_ok(int f) { return f == SKG_MX_E4M3 || f == SKG_MX_E2M1; }
size_t code_bytes(int format, size_t n) { return format == SKG_MX_E4M3 ? n : n / 2; }
int status(int hip) { return hip == (int)hipSuccess ? SKG_OK : SKG_ERR_HIP; }

int check_mx(int format, int M, int K) {
    if (!format_ok(format) || M < 0 || K < 0) return SKG_ERR_INVALID_ARG;
    if (K < 32 || K % 32 != 0 || (long)M * K > kMaxBufferBytes) return SKG_ERR_UNSUPPORTED;
    return SKG_OK;
}

// Quantised rows in a workspace: codes, then padded scale rows.
size_t round256(size_t n) { return (n + 255) / 256 * 256; }
size_t linear_workspace_bytes(size_t M, int K) {
    // e4m3 codes are the larger of the two formats
    return round256(M * (size_t)mx_code_stride(SKG_MX_E4M3, K)) + round256(M * (size_t)mx_scale_stride(K));
}

int check_linear(int M, int N, int K) {
    if (M < 0 || N < 0 || K < 0) return SKG_ERR_INVALID_ARG;
    if (M > SKG_MAX_M || N >= 1 << 20 || K >= 1 << 20 || K < 32 || K % 32 != 0)
        return SKG_ERR_UNSUPPORTED;
    return SKG_OK;
}

// How a product is done: by blocks of few rows (how many; bf16 rows quantised on
// the way or by a launch before), or by tiles (0).
struct Mxfp4Way {
    int blocks;
    bool quantise_first;
};

// Time in us of the blocks that suit M rows best.  A workgroup brings its rows
// and 16 columns of weights to a CU, 16 rows and more in two row blocks of the
// matrix instruction; a CU's workgroups follow each other, from 32 steps of K on
// (16 waves) without overlap.
double rows_time(int M, int N, int K, int format, bool codes, int *blocks) {
    // a column group's blocks share an XCD: 32 CUs for every eighth group
    const int groups = (mxfp4_groups(N) + 7) / 8, cus = kNumCusMI355X / 8;
    const size_t fit = kMxRowMaxLds / mxfp4_row_lds_bytes(format, K);
    const int most = (int)std::min<size_t>(codes ? kMxRowsCodes : kMxRowsBf16, fit);
    if (most < 1) return 1e30;
    const bool alone = mxfp4_steps(K) > 32;
    const double weights = 3e-4 * K;
    const double row = !codes ? 0.07 + 4.1e-5 * K : format == SKG_MX_E4M3 ? 0.05 + 2e-5 * K : 0.05 + 0.6e-5 * K;
    const int least = (M + most - 1) / most;  // blocks
    double best = 1e30;
    for (int i = 0; i < 3; ++i) {
        const long cu = i < 2 ? i + 1 : ((long)least * groups + cus - 1) / cus;
        const int b = (int)std::min<long>(M, cu * cus / groups);
        if (b < least) continue;
        const int r = (M + b - 1) / b;
        const double us = (alone ? cu : 1) * 1.5 + cu * (weights + row * r + (r > 16 ? 1.3 : 0.0));
        if (us < best) {
            best = us;
            *blocks = (M + r - 1) / r;
        }
    }
    return best;
}

// Fitted to the ways of 784 products, M = 2-512, N = 256-16384, K = 2048-7168, both
// formats.  Of those the way taken is within 1 % of the best of some twenty in the
// mean, over 15 % slower at 25, and nowhere more than 4 % slower than the tiles.
Mxfp4Way mxfp4_way(int M, int N, int K, int format, bool codes) {
    Mxfp4Way way{0, false};
    double best = mxfp4_tile_time(M, N, K, format);
    int blocks = 0;
    double us = rows_time(M, N, K, format, codes, &blocks);
    if (us < best) {
        best = us;
        way = {blocks, false};
    }
    if (!codes) {
        us = rows_time(M, N, K, format, true, &blocks) + 2.3;  // the launch before
        if (us < best) way = {blocks, true};
    }
    return way;
}

int check_moe(int T, int k, int H, int I, int E) {
    if (T < 0 || k < 1 || H < 1 || I < 1 || E < 1) return SKG_ERR_INVALID_ARG;
    if (H % 32 != 0 || I % 32 != 0 || H >= 1 << 20 || I >= 1 << 19 || E > SKG_ROUTE_MAX_E ||
        k > SKG_ROUTE_MAX_K)
        return SKG_ERR_UNSUPPORTED;
    const long P = (long)T * k, wide = H > I ? H : I;
    const int f = SKG_MX_E4M3;  // the wider codes: a row map spans less than 2 GiB
    if (P > kMaxBufferBytes || (long)T * mx_code_stride(f, H) > kMaxBufferBytes ||
        P * mx_code_stride(f, I) > kMaxBufferBytes || P * wide * 4 >= 1L << 40)
        return SKG_ERR_UNSUPPORTED;
    return SKG_OK;
}

size_t floats_of(size_t bytes) { return (bytes + 3) / 4; }

}  // namespace

extern "C" int skinny_quant_mx(const void *x, void *q, void *e8m0, int format, int M, int K,
                               hipStream_t stream) {
    const int rc = check_mx(format, M, K);
    if (rc != SKG_OK) return rc;
    if (M == 0) return SKG_OK;
    if (!x || !q || !e8m0) return SKG_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(q, 16)) return SKG_ERR_ALIGNMENT;
    const size_t n = (size_t)M * K;
    const Span outs[] = {{q, code_bytes(format, n)}, {e8m0, n / 32}}, ins[] = {{x, n * 2}};
    if (any_overlap(outs, ins)) return SKG_ERR_INVALID_ARG;
    return status(launch_quant_mx(x, q, e8m0, format, M, K, false, stream));
}

extern "C" int skinny_dequant_mx(const void *q, const void *e8m0, int format, void *out, int M,
                                 int K, hipStream_t stream) {
    const int rc = check_mx(format, M, K);
    if (rc != SKG_OK) return rc;
    if (M == 0) return SKG_OK;
    if (!q || !e8m0 || !out) return SKG_ERR_INVALID_ARG;
    if (!aligned(out, 16) || !aligned(q, 16)) return SKG_ERR_ALIGNMENT;
    const size_t n = (size_t)M * K;
    const Span outs[] = {{out, n * 2}}, ins[] = {{q, code_bytes(format, n)}, {e8m0, n / 32}};
    if (any_overlap(outs, ins)) return SKG_ERR_INVALID_ARG;
    return status(launch_dequant_mx(q, e8m0, format, out, M, K, stream));
}

extern "C" int skinny_rmsnorm(const void *x, const void *residual, const void *weight, float eps,
                              int out_format, const float *scale, void *y, void *e8m0,
                              void *residual_out, int M, int K, hipStream_t stream) {
    if (M < 0 || K < 0 || !(eps >= 0.0f) || out_format < SKG_NORM_BF16 || out_format > SKG_NORM_MX)
        return SKG_ERR_INVALID_ARG;
    if (K < 8 || K % (out_format == SKG_NORM_MX ? 32 : 8) != 0 || K > 65536 ||
        (long)M * K >= 1L << 40)
        return SKG_ERR_UNSUPPORTED;
    if (M == 0) return SKG_OK;
    if (!x || !weight || !y || (residual == nullptr) != (residual_out == nullptr) ||
        (scale != nullptr) != (out_format == SKG_NORM_E4M3) ||
        (e8m0 != nullptr) != (out_format == SKG_NORM_MX))
        return SKG_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(y, 16) ||
        !aligned(residual_out, 16) || !aligned(scale, 4))
        return SKG_ERR_ALIGNMENT;
    const size_t n = (size_t)M * K;
    const Span outs[] = {{y, out_format == SKG_NORM_BF16 ? 2 * n : n}, {e8m0, n / 32},
                         {residual_out, 2 * n}};
    // residual_out may be exactly x or residual: every element is read by the
    // lane that writes it, before it writes it
    const Span ins[] = {{x == residual_out ? nullptr : x, 2 * n},
                        {residual == residual_out ? nullptr : residual, 2 * n},
                        {weight, (size_t)K * 2},
                        {scale, 4}};
    if (any_overlap(outs, ins)) return SKG_ERR_INVALID_ARG;
    const Span y_out[] = {outs[0], outs[1]}, whole[] = {{x, 2 * n}, {residual, 2 * n}};
    if (any_overlap(y_out, whole)) return SKG_ERR_INVALID_ARG;
    return status(launch_rmsnorm(x, residual, weight, eps, out_format, scale, y, e8m0,
                                 residual_out, M, K, stream));
}

extern "C" int skinny_route(const void *logits, int dtype, const float *bias,
                            const skinny_route_options *o, float *weights, int *ids, int T, int E,
                            hipStream_t stream) {
    if (!o || T < 0 || E < 1 || o->k < 1 || o->groups < 1 || o->top_groups < 1)
        return SKG_ERR_INVALID_ARG;
    if (dtype != SKG_DTYPE_F32 && dtype != SKG_DTYPE_BF16) return SKG_ERR_INVALID_ARG;
    if (o->scores != SKG_SCORE_SOFTMAX && o->scores != SKG_SCORE_SIGMOID)
        return SKG_ERR_INVALID_ARG;
    if (E > SKG_ROUTE_MAX_E || o->k > SKG_ROUTE_MAX_K || o->groups > SKG_ROUTE_MAX_GROUPS ||
        E % o->groups != 0 || o->top_groups > o->groups ||
        o->k > o->top_groups * (E / o->groups))
        return SKG_ERR_UNSUPPORTED;
    if (T == 0) return SKG_OK;
    if (!logits || !weights || !ids) return SKG_ERR_INVALID_ARG;
    const uintptr_t la = dtype == SKG_DTYPE_F32 ? 4 : 2;
    if (!aligned(logits, la) || !aligned(bias, 4) || !aligned(weights, 4) || !aligned(ids, 4))
        return SKG_ERR_ALIGNMENT;
    const size_t n = (size_t)T * o->k * 4;
    const Span outs[] = {{weights, n}, {ids, n}},
               ins[] = {{logits, (size_t)T * E * la}, {bias, (size_t)E * 4}};
    if (any_overlap(outs, ins)) return SKG_ERR_INVALID_ARG;
    return status(launch_route(logits, dtype, bias, *o, weights, ids, T, E, stream));
}

extern "C" size_t skinny_mxfp4_packed_bytes(int E, int N, int K) {
    if (E < 1 || E > 65535 || N < 1 || K < 32 || K % 32 != 0 || N >= 1 << 20 || K >= 1 << 20)
        return 0;
    return mxfp4_packed_bytes(E, N, K);
}

extern "C" int skinny_mxfp4_pack(const void *q, const void *e8m0, void *packed, int E, int N,
                                 int K, hipStream_t stream) {
    if (E < 1 || N < 1 || K < 1) return SKG_ERR_INVALID_ARG;
    const size_t bytes = skinny_mxfp4_packed_bytes(E, N, K);
    if (bytes == 0) return SKG_ERR_UNSUPPORTED;
    if (!q || !e8m0 || !packed) return SKG_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(packed, 16)) return SKG_ERR_ALIGNMENT;
    const size_t n = (size_t)E * N * K;
    const Span outs[] = {{packed, bytes}}, ins[] = {{q, n / 2}, {e8m0, n / 32}};
    if (any_overlap(outs, ins)) return SKG_ERR_INVALID_ARG;
    return status(launch_mxfp4_pack(q, e8m0, packed, E, N, K, stream));
}

extern "C" int skinny_gemm_mxfp4(const void *x, const void *x_e8m0, int x_format,
                                 const void *packed, const void *bias, void *out, int out_dtype,
                                 int M, int N, int K, hipStream_t stream) {
    if (!format_ok(x_format) || (out_dtype != SKG_DTYPE_BF16 && out_dtype != SKG_DTYPE_F32))
        return SKG_ERR_INVALID_ARG;
    int rc = check_linear(M, N, K);
    if (rc != SKG_OK) return rc;
    if (M == 0 || N == 0) return SKG_OK;
    if (!x || !packed || !out) return SKG_ERR_INVALID_ARG;
    const bool f32 = out_dtype == SKG_DTYPE_F32;
    if (!aligned(x, 16) || !aligned(packed, 16) || !aligned(bias, 2) || !aligned(out, f32 ? 4 : 2))
        return SKG_ERR_ALIGNMENT;
    const size_t n = (size_t)M * K;
    const Span outs[] = {{out, (size_t)M * N * (f32 ? 4 : 2)}};
    const Span ins[] = {{x, x_e8m0 ? code_bytes(x_format, n) : 2 * n},
                        {x_e8m0, n / 32},
                        {packed, mxfp4_packed_bytes(1, N, K)},
                        {bias, (size_t)N * 2}};
    if (any_overlap(outs, ins)) return SKG_ERR_INVALID_ARG;
    Mxfp4Args a{(const uint8_t *)x, (int)code_bytes(x_format, K), (const uint8_t *)x_e8m0, K / 32, x_format,
                (const uint8_t *)packed, (const uint16_t *)bias, out, f32 ? 1 : 0, M, N, K};
    const Mxfp4Way way = mxfp4_way(M, N, K, x_format, x_e8m0 != nullptr);
    if (way.blocks && !way.quantise_first) return status(launch_mxfp4_rows(a, way.blocks, stream));
    float *ws = nullptr;
    unsigned *tk = nullptr;
    rc = acquire(stream, floats_of(linear_workspace_bytes((size_t)M, K)), 0, &ws, &tk);
    if (rc != SKG_OK) return rc;
    uint8_t *codes = (uint8_t *)ws, *scales = codes + round256((size_t)M * mx_code_stride(x_format, K));
    int e;
    if (x_e8m0) {
        e = launch_pad_scales(x_e8m0, scales, M, K, stream);
    } else {
        e = launch_quant_mx(x, codes, scales, x_format, M, K, true, stream);
        a.x = codes;
        a.xs = mx_code_stride(x_format, K);
    }
    if (e != (int)hipSuccess) return SKG_ERR_HIP;
    a.xe = scales;
    a.es = mx_scale_stride(K);
    return status(way.blocks ? launch_mxfp4_rows(a, way.blocks, stream) : launch_mxfp4(a, stream));
}

extern "C" int skinny_moe_mxfp4(const void *x, const int *ids, const float *weights,
                                const void *w13, const void *w2, void *out, int x_format, int T,
                                int k, int H, int I, int E, hipStream_t stream) {
    if (!format_ok(x_format)) return SKG_ERR_INVALID_ARG;
    int rc = check_moe(T, k, H, I, E);
    if (rc != SKG_OK) return rc;
    if (T == 0) return SKG_OK;
    if (!x || !ids || !weights || !w13 || !w2 || !out) return SKG_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(w13, 16) || !aligned(w2, 16) || !aligned(out, 16) ||
        !aligned(ids, 4) || !aligned(weights, 4))
        return SKG_ERR_ALIGNMENT;
    const size_t n = (size_t)T * H * 2, p = (size_t)T * k * 4;
    const Span outs[] = {{out, n}};
    const Span ins[] = {{x, n}, {ids, p}, {weights, p}, {w13, mxfp4_packed_bytes(E, 2 * I, H)},
                        {w2, mxfp4_packed_bytes(E, H, I)}};
    if (any_overlap(outs, ins)) return SKG_ERR_INVALID_ARG;
    float *ws = nullptr;
    unsigned *tk = nullptr;
    rc = acquire(stream, floats_of(moe_workspace_bytes(T, k, H, I, E, x_format)), 0, &ws, &tk);
    if (rc != SKG_OK) return rc;
    const MoeArgs a{(const uint16_t *)x, ids, weights, (const uint8_t *)w13, (const uint8_t *)w2,
                    (uint16_t *)out, x_format, T, k, H, I, E};
    return status(launch_moe(a, ws, stream));
}

// For the tests: the way a product takes (its blocks of rows, 0 for tiles, with
// their rows, whether they are quantised before, and the tile), and the experts'.
extern "C" int skg_mxfp4_way(int M, int N, int K, int format, int codes, int *rows, int *first, int *tile) {
    const Mxfp4Way way = mxfp4_way(M, N, K, format, codes != 0);
    *rows = way.blocks ? (M + way.blocks - 1) / way.blocks : 0;
    *first = way.quantise_first;
    *tile = dense_tile(M, N, format);
    return way.blocks;
}
extern "C" int skg_moe_way(int T, int k, int H, int I, int E, int format) {
    MoeArgs a{};
    a.fmt = format;
    a.T = T;
    a.k = k;
    a.H = H;
    a.I = I;
    a.E = E;
    return moe_way(a);
}

extern "C" int skinny_moe_reserve(int max_M, int max_K, int max_T, int k, int H, int I, int E,
                                  hipStream_t stream) {
    int rc = check_linear(max_M, 0, max_K ? max_K : 32);
    if (rc != SKG_OK) return rc;
    if (max_K < 0 || max_T < 0) return SKG_ERR_INVALID_ARG;
    size_t bytes = max_K ? linear_workspace_bytes((size_t)max_M, max_K) : 0;
    if (max_T > 0) {
        rc = check_moe(max_T, k, H, I, E);
        if (rc != SKG_OK) return rc;
        // e4m3 codes are the larger of the two formats
        const size_t moe = moe_workspace_bytes(max_T, k, H, I, E, SKG_MX_E4M3);
        bytes = moe > bytes ? moe : bytes;
    }
    if (bytes == 0) return SKG_OK;
    float *ws = nullptr;
    unsigned *tk = nullptr;
    return acquire(stream, floats_of(bytes), 0, &ws, &tk);
}
