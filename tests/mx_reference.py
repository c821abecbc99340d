"""Plain implementations of the operators of skinny_moe.h on the CPU, in 64
bits (test infrastructure).  MX codes are made with exact integer and fp64
arithmetic, apart from the kernels' bit tricks."""
import math

import numpy as np
import torch

E4M3_LARGEST, E2M1_LARGEST = 448.0, 6.0
E2M1_VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _e4m3_values():
    v = [(m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
         for e in range(16) for m in range(8)]
    v[-1] = math.nan
    return np.array(v)


E4M3_VALUES = _e4m3_values()


def values(fmt):
    """The value of each non-negative code (the sign is the next bit)."""
    return E4M3_VALUES if fmt == "e4m3" else E2M1_VALUES


def _nearest(q, table):
    """Codes of the values of `table` (ascending) nearest to |q| <= table[-1], ties to the even code."""
    a = np.abs(q)
    hi = np.clip(np.searchsorted(table, a), 1, len(table) - 1)
    lo = hi - 1
    dl, dh = a - table[lo], table[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return code | (np.signbit(q).astype(np.int64) * (128 if len(table) > 8 else 8))


def quantise(v, fmt):
    """fp64 [..., K] -> (codes int64 [..., K], e int64 [..., K/32])."""
    b = np.asarray(v, dtype=np.float64).reshape(*v.shape[:-1], -1, 32)
    largest = E4M3_LARGEST if fmt == "e4m3" else E2M1_LARGEST
    amax = np.abs(b).max(-1)
    bad = ~np.isfinite(amax)
    safe = np.where(bad | (amax == 0), largest, amax)
    m, p = np.frexp(safe / largest)  # safe / largest = m * 2^p, 0.5 <= m < 1
    e = np.clip(np.where(m == 0.5, p - 1, p) + 127, 0, 254)
    e = np.where(bad, 255, np.where(amax == 0, 127, e)).astype(np.int64)
    with np.errstate(invalid="ignore"):
        q = np.where(bad[..., None], 0.0, np.ldexp(b, (127 - np.minimum(e, 254))[..., None]))
    table = values(fmt)
    return _nearest(q, table[:-1] if fmt == "e4m3" else table).reshape(v.shape), e


def dequantise(codes, e, fmt):
    table = values(fmt)
    n = len(table)
    v = table[codes % n] * np.where(codes // n % 2 == 1, -1.0, 1.0)
    v = v.reshape(*codes.shape[:-1], -1, 32)
    with np.errstate(over="ignore"):
        v = np.where((e == 255)[..., None], np.nan, np.ldexp(v, (e - 127)[..., None]))
    return v.reshape(codes.shape)


def rounded(v, fmt):
    """v with its values replaced by those of their MX codes."""
    return dequantise(*quantise(v, fmt), fmt)


def pack_bytes(codes, fmt):
    """Codes as the library stores them, uint8."""
    if fmt == "e4m3":
        return codes.astype(np.uint8)
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack_bytes(b, fmt):
    if fmt == "e4m3":
        return b.astype(np.int64)
    return np.stack([b & 15, b >> 4], -1).reshape(*b.shape[:-1], -1).astype(np.int64)


def f64(t):
    return t.detach().cpu().double().numpy()


def norm(x, r, w, eps):
    s = f64(x) if r is None else f64(x) + f64(r)
    with np.errstate(invalid="ignore", divide="ignore"):
        return s, s / np.sqrt((s * s).mean(-1, keepdims=True) + eps) * f64(w)


def route(l, k, scores, bias, groups, top_groups, renormalize, factor):
    """(keys [T, E], experts of kept groups [T, E], ids [T, k], weights [T, k])."""
    l = np.where(np.isnan(l), -np.inf, np.asarray(l, dtype=np.float64))
    T, E = l.shape
    with np.errstate(invalid="ignore", over="ignore"):
        if scores == "sigmoid":
            p = 1.0 / (1.0 + np.exp(-l))
        else:
            m = l.max(-1, keepdims=True)
            t = np.where(l == -np.inf, 0.0, np.where(l == m, 1.0, np.exp(l - m)))
            total = t.sum(-1, keepdims=True)
            p = np.where(total > 0, t / np.where(total > 0, total, 1.0), 0.0)
    key = l if scores == "softmax" and bias is None else p + (0.0 if bias is None else bias)
    size = E // groups
    kept = np.ones((T, E), dtype=bool)
    if groups > 1:
        per = key.reshape(T, groups, size)
        best = np.sort(per, -1)[..., ::-1]
        value = best[..., 0] if scores == "softmax" or size == 1 else best[..., 0] + best[..., 1]
        first = np.argsort(-value, -1, kind="stable")[:, :top_groups]
        kept = np.zeros((T, groups), dtype=bool)
        np.put_along_axis(kept, first, True, 1)
        kept = np.repeat(kept, size, 1)
    ids = np.empty((T, k), dtype=np.int64)
    for t in range(T):
        ok = np.nonzero(kept[t])[0]
        ids[t] = ok[np.argsort(-key[t, ok], kind="stable")[:k]]
    w = np.take_along_axis(p, ids, 1)
    if renormalize:
        total = w.sum(-1, keepdims=True)
        w = np.where(total > 0, w / np.where(total > 0, total, 1.0), 0.0)
    return key, kept, ids, w * factor


def _undecided(v, fmt, near):
    """Hidden values whose code, or whose block's scale, lies within `near` of
    its value of the next one: (slice, the values it would then stand for)."""
    largest, table = (E4M3_LARGEST, E4M3_VALUES[:-1]) if fmt == "e4m3" else (E2M1_LARGEST, E2M1_VALUES)
    codes, e = quantise(v, fmt)
    scaled = np.ldexp(np.abs(v), 127 - np.repeat(e, 32))
    mids = (table[1:] + table[:-1]) / 2
    k = np.clip(np.searchsorted(mids, scaled), 0, len(mids) - 1)
    k = np.where((k > 0) & (np.abs(scaled - mids[k - 1]) < np.abs(scaled - mids[k])), k - 1, k)
    for i in np.nonzero(np.abs(scaled - mids[k]) <= near * scaled)[0]:
        here = codes[i] % len(values(fmt))
        other = np.ldexp(table[k[i] + 1 if here == k[i] else k[i]], int(e[i // 32]) - 127)
        yield slice(i, i + 1), np.copysign([other], v[i])
    top = np.repeat(np.abs(v).reshape(-1, 32).max(-1), 32)
    for f in (1 - near, 1 + near):
        o = quantise(top * f, fmt)[1]
        for b in np.nonzero((o != e) & (top[::32] > 0))[0]:
            at = slice(32 * b, 32 * b + 32)
            q = np.clip(np.ldexp(v[at], 127 - int(o[b])), -largest, largest)
            yield at, dequantise(_nearest(q, table), o[b:b + 1], fmt)


def experts(x, ids, weights, w13, w2, fmt, either=None):
    """x [T, H], w13 [E, 2I, H], w2 [E, H, I] fp64 values.  either: a list that
    takes (t, change of out[t]) for the hidden values and scales that lie within
    2^-13 of a tie, where the precision of the products' sums decides."""
    xq = rounded(x, fmt)
    out = np.zeros_like(xq)
    for t in range(x.shape[0]):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if not 0 <= e < w13.shape[0]:
                continue
            g, u = np.split(w13[e] @ xq[t], 2)
            v = g / (1.0 + np.exp(-g)) * u
            h = rounded(v, fmt)
            out[t] += weights[t, j] * (w2[e] @ h)
            if either is not None:
                either += [(t, weights[t, j] * (w2[e][:, at] @ (alt - h[at])))
                           for at, alt in _undecided(v, fmt, 2.0 ** -13)]
    return out


def bf16(v):
    return torch.from_numpy(np.asarray(v, dtype=np.float32)).to(torch.bfloat16)
