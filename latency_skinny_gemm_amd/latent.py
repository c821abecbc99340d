"""Binding of latent attention (include/skinny_latent.h): norm, rotation and
append to a paged cache, attention over it in the absorbed form, attention of
prompts over expanded keys and values, and the products per head between them.

As for the products: argument marshalling only, device tensors of one device,
work on `stream` or the device's current stream, SkinnyGemmError for what the
library refuses, no fallback.  Tensors are contiguous except where strides are
mentioned.  The contents of table, kv_lens and q_starts (int32) stay on the
device; see skinny_latent_batch for what they mean.

One decode step, q [T, H, 192] and kv [T, 576] from the projections:

    ql = torch.empty(T, H, 576, dtype=torch.bfloat16, device=q.device)
    latent_append(kv, cache, table, kv_lens, rotations, weight=g,
                  q_rope=q[..., 128:], q_rope_out=ql[..., 512:])
    heads_gemm(q[..., :128], wk, out=ql[..., :512])        # wk [H, 512, 128]
    o = latent_attention(ql, cache, table, kv_lens, scale)
    y = heads_gemm(o, wv)                                  # wv [H, 128, 512]
"""
import ctypes
from collections import namedtuple

import torch

import latency_skinny_gemm_amd as _c
from .moe import _BF16, _F32, _choice, _count, _same_device, _tensor

__all__ = ["LatentOut", "latent_append", "latent_attention", "latent_attention_expanded",
           "heads_gemm", "reserve_latent"]

# mirrors of include/skinny_latent.h
LATENT, ROPE, ROW = 512, 64, 576
NOPE, V = 128, 128
ROPE_PAIRS = 0
ROPE_HALVES = 1

_STYLES = {"pairs": ROPE_PAIRS, "halves": ROPE_HALVES}
_I32 = (torch.int32,)
_BF = torch.bfloat16
_CACHE = (torch.bfloat16, torch.float8_e4m3fn)

LatentOut = namedtuple("LatentOut", "latent q_rope")


class LatentBatch(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("kv_lens", ctypes.c_void_p), ("q_starts", ctypes.c_void_p),
                ("B", ctypes.c_int), ("T", ctypes.c_int), ("table_width", ctypes.c_int),
                ("page_size", ctypes.c_int), ("pages", ctypes.c_int)]


def declare(L):
    """Sets the argument types of skinny_latent.h's entry points."""
    P, I, F, N = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_long
    B = ctypes.POINTER(LatentBatch)
    for name, args in (
            ("skinny_latent_append", [B, P, N, P, F, P, I, I, P, I, P, P, P, N, N, P, N, N, I, P]),
            ("skinny_latent_attention", [B, P, P, I, P, F, P, I, P]),
            ("skinny_latent_attention_expanded", [P, P, P, N, P, P, P, F, I, I, I, I, I, P]),
            ("skinny_heads_gemm", [P, N, N, P, P, N, N, I, I, I, I, P]),
            ("skinny_latent_reserve", [I, P])):
        f = getattr(L, name)
        f.argtypes, f.restype = args, I


def _refuse(name, t, shape):
    """Raises for what _rows and _heads did not take."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if t.dim() != len(shape) or any(s is not None and s != n for s, n in zip(shape, t.shape)):
        raise ValueError(f"{name} must be {['any' if s is None else s for s in shape]}, got {list(t.shape)}")
    raise ValueError(f"{name} must be dense in its last dimension")


def _rows(name, t, rows, n):
    """The stride of bf16 t [rows, n] (rows None: any number) from row to row; the
    last dimension is dense."""
    if isinstance(t, torch.Tensor) and t.dtype is _BF and t.is_cuda and t.dim() == 2:
        r, c = t.shape
        if c == n and (rows is None or r == rows):
            s, one = t.stride()
            if one == 1:
                return s if r > 1 else n  # torch may give one row any stride
    _refuse(name, t, (rows, n))


def _heads(name, t, T, H, n):
    """The strides of bf16 t [T, H, n] (T, H None: any number) from token to token and
    from head to head; the last dimension is dense."""
    if isinstance(t, torch.Tensor) and t.dtype is _BF and t.is_cuda and t.dim() == 3:
        r, h, c = t.shape
        if c == n and (T is None or r == T) and (H is None or h == H):
            s, sh, one = t.stride()
            if one == 1 or n == 1:
                if h == 1:
                    sh = n
                return (s if r > 1 else max(n, sh * h)), sh
    _refuse(name, t, (T, H, n))


def _batch(cache, table, kv_lens, q_starts, T):
    if not (cache.dtype in _CACHE and cache.is_cuda and cache.dim() == 3 and cache.is_contiguous()):
        _tensor("cache", cache, _CACHE)
    pages, page, row = cache.shape if cache.dim() == 3 else (0, 0, 0)
    if row != ROW:
        raise ValueError(f"cache must be [pages, page_size, {ROW}], got {list(cache.shape)}")
    _tensor("table", table, _I32)
    if table.dim() != 2:
        raise ValueError("table must be [B, table_width]")
    B, W = table.shape
    _tensor("kv_lens", kv_lens, _I32, (B,))
    if q_starts is not None:
        _tensor("q_starts", q_starts, _I32, (B + 1,))
    elif T != B:
        raise ValueError(f"without q_starts every sequence has one new token, got {T} for {B} sequences")
    _count(B | T | W | page | pages)  # one of 32 bits or more shows in the union
    return LatentBatch(table.data_ptr(), kv_lens.data_ptr(), None if q_starts is None else q_starts.data_ptr(),
                       B, T, W, page, pages)


def _cache_scale(cache, scale):
    if (scale is not None) != (cache.dtype == torch.float8_e4m3fn):
        raise ValueError("scale goes with a float8_e4m3fn cache, and only with it")
    if scale is not None:
        _c._scalar_f32("scale", scale)
    return _c.DTYPE_FP8 if scale is not None else _c.DTYPE_BF16


def latent_append(kv, cache, table, kv_lens, rotations, q_starts=None, weight=None, eps=1e-6,
                  rope="pairs", scale=None, q_rope=None, q_rope_out=None, latent=False, stream=None):
    """Norm (weight bf16 [512]; None: none) and rotation of new tokens' kv bf16
    [T, 576] into cache [pages, page_size, 576] (bf16, or float8_e4m3fn with
    scale), and the rotation of the queries' q_rope bf16 [T, H, 64].

    kv, q_rope and q_rope_out may have strides (the last dimension dense);
    q_rope_out may be q_rope.  rotations: fp32 [rows, 64], 32 cosines and 32 sines
    a row.  rope: "pairs" or "halves".  Returns LatentOut(latent, q_rope): latent
    = the rows in bf16 [T, 576] if asked for, q_rope the rotated queries if given."""
    style = _choice("rope", rope, _STYLES)
    kv_stride = _rows("kv", kv, None, ROW)
    T = kv.shape[0]
    batch = _batch(cache, table, kv_lens, q_starts, T)
    dtype = _cache_scale(cache, scale)
    _tensor("rotations", rotations, _F32)
    if rotations.dim() != 2 or rotations.shape[1] != ROPE:
        raise ValueError(f"rotations must be [rows, {ROPE}]")
    if weight is not None:
        _tensor("weight", weight, _BF16, (LATENT,))
    H = qt = qh = ot = oh = 0
    qp = op = None
    if q_rope is not None:
        qt, qh = _heads("q_rope", q_rope, T, None, ROPE)
        H = q_rope.shape[1]
        if q_rope_out is None:
            q_rope_out = _c._empty((T, H, ROPE), torch.bfloat16, kv.device, stream)
            ot, oh = H * ROPE, ROPE
        else:
            ot, oh = _heads("q_rope_out", q_rope_out, T, H, ROPE)
        if T == 0:
            H = 0  # torch gives an empty tensor no address
        if H:
            qp, op = q_rope.data_ptr(), q_rope_out.data_ptr()
    elif q_rope_out is not None:
        raise ValueError("q_rope_out needs a q_rope")
    out = _c._empty((T, ROW), torch.bfloat16, kv.device, stream) if latent else None
    p = _c._addr
    rc = _c._launch(_same_device(kv, cache, table, kv_lens, q_starts, rotations, weight, scale, q_rope, q_rope_out),
                    stream, _c._load().skinny_latent_append, batch, kv.data_ptr(), kv_stride, p(weight), eps,
                    rotations.data_ptr(), _count(rotations.shape[0]), style, cache.data_ptr(), dtype, p(scale),
                    p(out), qp, qt, qh, op, ot, oh, H)
    if rc:
        _c._check(rc, f"skinny_latent_append(T={T}, H={H}, {cache.dtype}, {rope})")
    return LatentOut(out, q_rope_out)


def latent_attention(q, cache, table, kv_lens, softmax_scale, q_starts=None, scale=None, out=None,
                     stream=None):
    """Attention in the absorbed form, bf16 [T, H, 512]: q bf16 [T, H, 576] over the
    cache rows (bf16, or float8_e4m3fn with scale) of each token's sequence up to
    its own.  One new token a sequence, or q_starts[b] .. q_starts[b + 1] - 1.
    Outputs of tokens behind the last sequence are left as they were.  A table no
    wider than the longest sequence needs is fastest."""
    _tensor("q", q, _BF16)
    if q.dim() != 3 or q.shape[2] != ROW:
        raise ValueError(f"q must be [T, H, {ROW}], got {list(q.shape)}")
    T, H = q.shape[:2]
    batch = _batch(cache, table, kv_lens, q_starts, T)
    dtype = _cache_scale(cache, scale)
    if out is None:
        out = _c._empty((T, H, LATENT), torch.bfloat16, q.device, stream)
    else:
        _tensor("out", out, _BF16, (T, H, LATENT))
    rc = _c._launch(_same_device(q, cache, table, kv_lens, q_starts, scale, out), stream,
                    _c._load().skinny_latent_attention, batch, q.data_ptr(), cache.data_ptr(), dtype,
                    _c._addr(scale), softmax_scale, out.data_ptr(), _count(H))
    if rc:
        _c._check(rc, f"skinny_latent_attention(T={T}, B={table.shape[0]}, H={H}, {cache.dtype})")
    return out


def latent_attention_expanded(q, kv, k_rope, q_starts, softmax_scale, kv_starts=None, causal=True,
                              out=None, stream=None):
    """Attention of prompts in the expanded form, bf16 [T, H, 128]: q bf16 [T, H,
    192], kv bf16 [S, H, 256] (128 key values of the head's own, 128 values),
    k_rope bf16 [S, 64] (rows may have a stride).  Sequence b: tokens q_starts[b] ..
    q_starts[b + 1] - 1 and keys kv_starts[b] .. (None: the same as q_starts)."""
    _tensor("q", q, _BF16)
    _tensor("kv", kv, _BF16)
    if q.dim() != 3 or q.shape[2] != NOPE + ROPE:
        raise ValueError(f"q must be [T, H, {NOPE + ROPE}], got {list(q.shape)}")
    T, H = q.shape[:2]
    if kv.dim() != 3 or tuple(kv.shape[1:]) != (H, NOPE + V):
        raise ValueError(f"kv must be [S, {H}, {NOPE + V}], got {list(kv.shape)}")
    S = kv.shape[0]
    rs = _rows("k_rope", k_rope, S, ROPE)
    _tensor("q_starts", q_starts, _I32)
    if q_starts.dim() != 1 or q_starts.shape[0] < 1:
        raise ValueError("q_starts must be [B + 1]")
    if kv_starts is None:
        kv_starts = q_starts
    else:
        _tensor("kv_starts", kv_starts, _I32, tuple(q_starts.shape))
    if out is None:
        out = _c._empty((T, H, V), torch.bfloat16, q.device, stream)
    else:
        _tensor("out", out, _BF16, (T, H, V))
    B = q_starts.shape[0] - 1
    _count(B | T | S | H)
    rc = _c._launch(_same_device(q, kv, k_rope, q_starts, kv_starts, out), stream,
                    _c._load().skinny_latent_attention_expanded, q.data_ptr(), kv.data_ptr(), k_rope.data_ptr(), rs,
                    q_starts.data_ptr(), kv_starts.data_ptr(), out.data_ptr(), softmax_scale, 1 if causal else 0,
                    B, T, S, H)
    if rc:
        _c._check(rc, f"skinny_latent_attention_expanded(T={T}, S={S}, B={B}, H={H})")
    return out


def heads_gemm(x, W, out=None, stream=None):
    """out[t, h] = W[h] @ x[t, h], bf16 [T, H, N]: x bf16 [T, H, K], W bf16 [H, N,
    K]; x and out may have strides (the last dimension dense)."""
    _tensor("W", W, _BF16)
    if W.dim() != 3:
        raise ValueError("W must be [H, N, K]")
    H, N, K = W.shape
    xs = _heads("x", x, None, H, K)
    T = x.shape[0]
    _count(T | H | N | K)
    if out is None:
        out = _c._empty((T, H, N), torch.bfloat16, x.device, stream)
        os = (H * N, N)
    else:
        os = _heads("out", out, T, H, N)
    rc = _c._launch(_same_device(x, W, out), stream, _c._load().skinny_heads_gemm, x.data_ptr(), *xs, W.data_ptr(),
                    out.data_ptr(), *os, T, H, N, K)
    if rc:
        _c._check(rc, f"skinny_heads_gemm(T={T}, H={H}, N={N}, K={K})")
    return out


def reserve_latent(H, stream=None):
    """Reserves workspace for `stream` (else the current stream): latent_attention
    calls of H heads, any batch and lengths, and latent_attention_expanded calls.
    Before graph capture."""
    _count(H)
    s = torch.cuda.current_stream() if stream is None else stream
    with torch.cuda.device(s.device):
        _c._check(_c._load().skinny_latent_reserve(H, ctypes.c_void_p(s.cuda_stream)), "skinny_latent_reserve")
