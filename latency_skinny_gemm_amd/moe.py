"""Binding of the operators around the small-M products of a
mixture-of-experts decode step (include/skinny_moe.h): norm, routing,
microscaling and the MXFP4 products.

As for the products: argument marshalling only, tensors contiguous on one
device, work on `stream` or the device's current stream, SkinnyGemmError for
what the library refuses, no fallback.

    n = rmsnorm(x, g, residual=r)                 # n.y, n.residual
    logits = gemm_bf16_f32(n.y, w_router)
    weights, ids = route(logits, k)
    out = moe_mxfp4(n.y, ids, weights, w13, w2)   # w13, w2 = mxfp4_pack(...)
"""
import ctypes
import math
from collections import namedtuple

import torch

import latency_skinny_gemm_amd as _c

__all__ = ["MX_E4M3", "MX_E2M1", "NormOut", "MxfpWeights", "rmsnorm", "route", "quant_mx",
           "dequant_mx", "mxfp4_pack", "gemm_mxfp4", "moe_mxfp4", "reserve_moe"]

# mirrors of include/skinny_moe.h
MX_E4M3 = 0
MX_E2M1 = 4
NORM_BF16 = 0
NORM_E4M3 = 1
NORM_MX = 2
SCORE_SOFTMAX = 0
SCORE_SIGMOID = 1

_FORMATS = {"e4m3": MX_E4M3, "e2m1": MX_E2M1}
_NORMS = {"bf16": NORM_BF16, "e4m3": NORM_E4M3, "mx": NORM_MX}
_SCORES = {"softmax": SCORE_SOFTMAX, "sigmoid": SCORE_SIGMOID}

NormOut = namedtuple("NormOut", "y e8m0 residual")


class RouteOptions(ctypes.Structure):
    _fields_ = [("scores", ctypes.c_int), ("k", ctypes.c_int), ("groups", ctypes.c_int),
                ("top_groups", ctypes.c_int), ("renormalize", ctypes.c_int),
                ("factor", ctypes.c_float)]


class MxfpWeights:
    """MXFP4 weights [E, N, K] (or [N, K]: E is None) in the products' layout."""

    __slots__ = ("packed", "E", "N", "K")

    def __init__(self, packed, E, N, K):
        self.packed, self.E, self.N, self.K = packed, E, N, K

    def __repr__(self):
        return f"MxfpWeights(E={self.E}, N={self.N}, K={self.K}, device={self.packed.device})"


def declare(L):
    """Sets the argument types of skinny_moe.h's entry points."""
    P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    for name, args in (
            ("skinny_quant_mx", [P, P, P, I, I, I, P]),
            ("skinny_dequant_mx", [P, P, I, P, I, I, P]),
            ("skinny_rmsnorm", [P, P, P, F, I, P, P, P, P, I, I, P]),
            ("skinny_route", [P, I, P, ctypes.POINTER(RouteOptions), P, P, I, I, P]),
            ("skinny_mxfp4_pack", [P, P, P, I, I, I, P]),
            ("skinny_gemm_mxfp4", [P, P, I, P, P, P, I, I, I, I, P]),
            ("skinny_moe_mxfp4", [P, P, P, P, P, P, I, I, I, I, I, I, P]),
            ("skinny_moe_reserve", [I, I, I, I, I, I, I, P])):
        f = getattr(L, name)
        f.argtypes, f.restype = args, I
    L.skinny_mxfp4_packed_bytes.argtypes = [I, I, I]
    L.skinny_mxfp4_packed_bytes.restype = ctypes.c_size_t


def _tensor(name, t, dtypes, shape=None):
    if (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in dtypes and t.is_contiguous()
            and (shape is None or t.shape == shape)):
        return
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    raise ValueError(f"{name} must be contiguous (the library takes no strides)")


def _same_device(x, *ts):
    """x's device; the others (None entries skipped) must be on it."""
    i = x.get_device()
    for t in ts:
        if t is not None and t.get_device() != i:
            raise ValueError(f"all tensors must be on one device, got {x.device} and {t.device}")
    return x.device


def _choice(name, value, table):
    if value not in table:
        raise ValueError(f"{name} must be one of {', '.join(map(repr, table))}, got {value!r}")
    return table[value]


_BF16 = (torch.bfloat16,)
_F32 = (torch.float32,)
_U8 = (torch.uint8,)
_E8M0 = (torch.uint8, torch.float8_e8m0fnu)
_E4M3 = (torch.float8_e4m3fn, torch.uint8)


def _codes(name, q, e8m0, fmt):
    """Checks MX codes and scales; returns (rows shape, K)."""
    _tensor(name, q, _U8 if fmt == MX_E2M1 else _E4M3)
    if q.dim() < 1:
        raise ValueError(f"{name} must have a row dimension")
    K = q.shape[-1] * (2 if fmt == MX_E2M1 else 1)
    lead = q.shape[:-1]
    _tensor(name + "'s e8m0", e8m0, _E8M0, (*lead, K // 32))
    return lead, K


def _count(n):
    """n, refused past 31 bits: ctypes would pass its low half on."""
    if n >> 31:
        _c._check(_c.ERR_UNSUPPORTED, f"a size of {n}")
    return n


def _rows(lead):
    return _count(math.prod(lead))


def quant_mx(x, format="e4m3", stream=None):
    """MX codes of bf16 x [..., K]: (float8_e4m3fn [..., K] or packed e2m1
    uint8 [..., K/2], e8m0 uint8 [..., K/32])."""
    fmt = _choice("format", format, _FORMATS)
    _tensor("x", x, _BF16)
    if x.dim() < 1 or x.shape[-1] % 32:
        raise ValueError("x must be [..., K] with K a multiple of 32")
    lead, K = x.shape[:-1], x.shape[-1]
    if fmt == MX_E4M3:
        q = _c._empty_like(x, torch.float8_e4m3fn, stream)
    else:
        q = _c._empty((*lead, K // 2), torch.uint8, x.device, stream)
    e = _c._empty((*lead, K // 32), torch.uint8, x.device, stream)
    M = _rows(lead)
    rc = _c._launch(x.device, stream, _c._load().skinny_quant_mx, x.data_ptr(), q.data_ptr(),
                    e.data_ptr(), fmt, M, K)
    if rc:
        _c._check(rc, f"skinny_quant_mx(M={M}, K={K}, {format})")
    return q, e


def dequant_mx(q, e8m0, stream=None):
    """The bf16 values of MX codes as quant_mx and rmsnorm(out_format="mx")
    return them: float8_e4m3fn codes, or packed e2m1 in uint8."""
    fmt = MX_E2M1 if q.dtype == torch.uint8 else MX_E4M3
    lead, K = _codes("q", q, e8m0, fmt)
    out = _c._empty((*lead, K), torch.bfloat16, q.device, stream)
    M = _rows(lead)
    rc = _c._launch(_same_device(q, e8m0), stream, _c._load().skinny_dequant_mx, q.data_ptr(),
                    e8m0.data_ptr(), fmt, out.data_ptr(), M, K)
    if rc:
        _c._check(rc, f"skinny_dequant_mx(M={M}, K={K})")
    return out


def rmsnorm(x, weight, residual=None, eps=1e-6, out_format="bf16", scale=None, residual_out=None,
            stream=None):
    """Residual addition and root-mean-square norm of x [..., K].

    s = x + residual in fp32; y = s / sqrt(mean(s^2) + eps) * weight.
    out_format "bf16"; "e4m3": codes of y / scale (a one-element fp32 tensor),
    for gemm_fp8(sx=scale); "mx": e4m3 codes with e8m0 scales, for
    gemm_fp8(xe=...) and gemm_mxfp4(xe=...).  Returns NormOut(y, e8m0,
    residual): e8m0 None unless "mx"; residual = bf16(s), None without one
    given.  residual_out may be residual or x itself (updated in place)."""
    fmt = _choice("out_format", out_format, _NORMS)
    _tensor("x", x, _BF16)
    if x.dim() < 1:
        raise ValueError("x must be [..., K]")
    K, dev = x.shape[-1], x.device
    _tensor("weight", weight, _BF16, (K,))
    if (scale is not None) != (fmt == NORM_E4M3):
        raise ValueError('scale goes with out_format "e4m3", and only with it')
    if scale is not None:
        _c._scalar_f32("scale", scale)
    if residual is not None:
        _tensor("residual", residual, _BF16, tuple(x.shape))
        if residual_out is None:
            residual_out = _c._empty_like(x, torch.bfloat16, stream)
        else:
            _tensor("residual_out", residual_out, _BF16, tuple(x.shape))
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    if fmt == NORM_MX and K % 32:
        raise ValueError("MX output needs K a multiple of 32")
    y = _c._empty_like(x, torch.bfloat16 if fmt == NORM_BF16 else torch.float8_e4m3fn, stream)
    e = _c._empty((*x.shape[:-1], K // 32), torch.uint8, dev, stream) if fmt == NORM_MX else None
    M = _rows(x.shape[:-1])
    p = _c._addr
    rc = _c._launch(_same_device(x, weight, residual, scale, residual_out), stream,
                    _c._load().skinny_rmsnorm, x.data_ptr(), p(residual), weight.data_ptr(), eps,
                    fmt, p(scale), y.data_ptr(), p(e), p(residual_out), M, K)
    if rc:
        _c._check(rc, f"skinny_rmsnorm(M={M}, K={K}, {out_format})")
    return NormOut(y, e, residual_out)


def route(logits, k, scores="softmax", bias=None, groups=1, top_groups=1, renormalize=True,
          factor=1.0, stream=None):
    """(weights fp32 [T, k], ids int32 [T, k]) of router logits [T, E] (fp32 or
    bf16): the k best experts by softmax or sigmoid scores plus bias (fp32
    [E]), from the top_groups best of `groups` groups; see skinny_route."""
    sc = _choice("scores", scores, _SCORES)
    _tensor("logits", logits, (torch.float32, torch.bfloat16))
    if logits.dim() != 2:
        raise ValueError("logits must be [T, E]")
    T, E = logits.shape
    _count(max(T, k, groups, top_groups))
    if bias is not None:
        _tensor("bias", bias, _F32, (E,))
    o = RouteOptions(sc, k, groups, top_groups, 1 if renormalize else 0, factor)
    w = _c._empty((T, max(k, 0)), torch.float32, logits.device, stream)
    ids = _c._empty((T, max(k, 0)), torch.int32, logits.device, stream)
    rc = _c._launch(_same_device(logits, bias), stream, _c._load().skinny_route,
                    logits.data_ptr(), _c.DTYPE_F32 if logits.dtype == torch.float32
                    else _c.DTYPE_BF16, _c._addr(bias), ctypes.byref(o), w.data_ptr(),
                    ids.data_ptr(), T, E)
    if rc:
        _c._check(rc, f"skinny_route(T={T}, E={E}, k={k}, groups={groups}/{top_groups})")
    return w, ids


def mxfp4_pack(q, e8m0, stream=None):
    """MXFP4 weights (packed e2m1 uint8 [N, K/2] or [E, N, K/2], e8m0 [..,
    K/32]), laid out once for gemm_mxfp4 or moe_mxfp4."""
    lead, K = _codes("q", q, e8m0, MX_E2M1)
    if len(lead) not in (1, 2):
        raise ValueError("q must be [N, K/2] or [E, N, K/2]")
    E, N = (None, lead[0]) if len(lead) == 1 else lead
    _count(max(lead))
    L = _c._load()
    n = L.skinny_mxfp4_packed_bytes(E or 1, N, K)
    if n == 0:
        _c._check(_c.ERR_UNSUPPORTED, f"skinny_mxfp4_pack(E={E}, N={N}, K={K})")
    packed = _c._empty((n,), torch.uint8, q.device, stream)
    rc = _c._launch(_same_device(q, e8m0), stream, L.skinny_mxfp4_pack, q.data_ptr(),
                    e8m0.data_ptr(), packed.data_ptr(), E or 1, N, K)
    _c._check(rc, f"skinny_mxfp4_pack(E={E}, N={N}, K={K})")
    return MxfpWeights(packed, E, N, K)


def gemm_mxfp4(x, w, xe=None, x_format="e4m3", bias=None, out_dtype=torch.bfloat16, out=None,
               stream=None):
    """out[M, N] = x @ W^T (+ bias bf16 [N]) with w = mxfp4_pack(...).  x: bf16
    [M, K], quantised in the call to x_format, or (xe given) MX codes of
    x_format: float8_e4m3fn [M, K] or packed e2m1 uint8 [M, K/2]."""
    fmt = _choice("x_format", x_format, _FORMATS)
    if not isinstance(w, MxfpWeights) or w.E is not None:
        raise TypeError("w must be mxfp4_pack of one [N, K] weight")
    if x.dim() != 2:
        raise ValueError("x must be [M, K]")
    if xe is None:
        _tensor("x", x, _BF16)
        K = x.shape[1]
    else:
        _, K = _codes("x", x, xe, fmt)
    M, N = _count(x.shape[0]), w.N
    if K != w.K:
        raise ValueError(f"x has K={K}, w has K={w.K}")
    if bias is not None:
        _tensor("bias", bias, _BF16, (N,))
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("out_dtype must be torch.bfloat16 or torch.float32")
    if out is None:
        out = _c._empty((M, N), out_dtype, x.device, stream)
    else:
        _tensor("out", out, (out_dtype,), (M, N))
    rc = _c._launch(_same_device(x, w.packed, xe, bias, out), stream,
                    _c._load().skinny_gemm_mxfp4, x.data_ptr(), _c._addr(xe), fmt,
                    w.packed.data_ptr(), _c._addr(bias), out.data_ptr(),
                    _c.DTYPE_F32 if out_dtype == torch.float32 else _c.DTYPE_BF16, M, N, K)
    if rc:
        _c._check(rc, f"skinny_gemm_mxfp4(M={M}, N={N}, K={K}, {x_format})")
    return out


def moe_mxfp4(x, ids, weights, w13, w2, x_format="e4m3", out=None, stream=None):
    """The routed experts' feed-forward, bf16 [T, H]: sum over a token's
    choices of weights[t, j] * W2 . q(silu(g) * u), (g, u) = W13 . q(x[t]).
    ids int32 and weights fp32 [T, k] (as route returns them; ids outside
    [0, E) are skipped); w13 = mxfp4_pack of [E, 2I, H], w2 of [E, H, I]."""
    fmt = _choice("x_format", x_format, _FORMATS)
    _tensor("x", x, _BF16)
    if x.dim() != 2:
        raise ValueError("x must be [T, H]")
    _tensor("ids", ids, (torch.int32,))
    if ids.dim() != 2 or ids.shape[0] != x.shape[0]:
        raise ValueError("ids must be [T, k]")
    _tensor("weights", weights, _F32, tuple(ids.shape))
    for name, w in (("w13", w13), ("w2", w2)):
        if not isinstance(w, MxfpWeights) or w.E is None:
            raise TypeError(f"{name} must be mxfp4_pack of [E, N, K] weights")
    (T, H), k, I, E = x.shape, ids.shape[1], w2.K, w2.E
    _count(max(T, k))
    if w13.E != E or w13.N != 2 * I or w13.K != H or w2.N != H:
        raise ValueError(f"w13 must be [E, 2I, H] and w2 [E, H, I] with H={H}, got {w13} and {w2}")
    if out is None:
        out = _c._empty((T, H), torch.bfloat16, x.device, stream)
    else:
        _tensor("out", out, _BF16, (T, H))
    rc = _c._launch(_same_device(x, ids, weights, w13.packed, w2.packed, out), stream,
                    _c._load().skinny_moe_mxfp4, x.data_ptr(), ids.data_ptr(), weights.data_ptr(),
                    w13.packed.data_ptr(), w2.packed.data_ptr(), out.data_ptr(), fmt, T, k, H, I, E)
    if rc:
        _c._check(rc, f"skinny_moe_mxfp4(T={T}, k={k}, H={H}, I={I}, E={E}, {x_format})")
    return out


def reserve_moe(max_M=0, max_K=0, max_T=0, k=1, H=32, I=32, E=1, stream=None):
    """Reserves workspace for `stream` (else the current stream): gemm_mxfp4
    calls with x up to [max_M, max_K] and moe_mxfp4 calls of up to max_T tokens
    with these sizes.  Before graph capture."""
    s = torch.cuda.current_stream() if stream is None else stream
    with torch.cuda.device(s.device):
        _c._check(_c._load().skinny_moe_reserve(max_M, max_K, max_T, k, H, I, E,
                                                ctypes.c_void_p(s.cuda_stream)),
                  "skinny_moe_reserve")
