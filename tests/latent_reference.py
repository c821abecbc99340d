"""Plain implementations of latent attention in 64 bits on the CPU, one sequence
and one row at a time, and the bounds that the tests allow around them.

Bounds, derived from the parts:
- A weight is rounded to bf16 before the second product: at most 2^-8 of it.  Its
  exponent is off by the first product's fp32 sum and by the fp32 rounding of
  exp2's argument: an error of `d` moves a weight by d of it.  The sum of weights
  moves likewise.  So the output moves by at most (2^-8 + 2 d + n 2^-24) sum_p
  w_p |v_p|, n the number of keys, and its own rounding adds 2^-8 |out|.
- The first product adds up k terms in fp32, whatever the order: at most
  k 2^-24 sum |q_i k_i|; the argument of exp2 is rounded at most twice: 2^-23 of
  the largest score.
- A product of K terms: K 2^-24 sum |w x|, and 2^-8 of the output.
"""
import torch

L, R, ROW = 512, 64, 576
NOPE, V = 128, 128


def nearest(x, bits, low):
    """fp64 x to the nearest number of `bits` fraction bits (ties to even), binades below 2^low as subnormals."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** low))) - bits)
    y = torch.round(x / step) * step
    return torch.where(torch.isfinite(x), y, x)


def to_bf16(x):
    return nearest(x, 7, -126).float().bfloat16()


def to_e4m3(x):
    """Codes (float8_e4m3fn) of fp64 x, clamped to +-448; NaN stays."""
    return nearest(x, 3, -6).clamp(-448.0, 448.0).float().to(torch.float8_e4m3fn)


def rotate(x, row, style):
    """x [.., 64] (fp64) by row [.., 64]: 32 cosines, 32 sines."""
    c, s = row.double().chunk(2, -1)
    a, b = (x[..., 0::2], x[..., 1::2]) if style == "pairs" else (x[..., :32], x[..., 32:])
    y = torch.empty_like(x)
    if style == "pairs":
        y[..., 0::2], y[..., 1::2] = a * c - b * s, a * s + b * c
    else:
        y[..., :32], y[..., 32:] = a * c - b * s, a * s + b * c
    return y


def sequences(starts, B, T):
    """(first, n) of each sequence's tokens."""
    if starts is None:
        return [(b, 1) for b in range(B)]
    s = [min(max(v, 0), T) for v in starts]
    return [(s[b], max(s[b + 1] - s[b], 0)) for b in range(B)]


def append(kv, weight, eps, rotations, style, cache, scale, table, lens, starts, q):
    """(cache, latent [T, 576] fp64, q fp64): cache as its type, updated in a copy; rows of no token are NaN."""
    T = kv.shape[0]
    B, W = table.shape
    pages, page = cache.shape[:2]
    cache = cache.clone()
    latent = torch.full((T, ROW), float("nan"), dtype=torch.float64)
    qo = None if q is None else torch.full(q.shape, float("nan"), dtype=torch.float64)
    for b, (first, n) in enumerate(sequences(starts, B, T)):
        length = min(max(int(lens[b]), 0), W * page)
        for j in range(n):
            t, at = first + j, length - n + j
            x = kv[t].double()
            c = x[:L]
            if weight is not None:
                c = c * (1.0 / torch.sqrt((c * c).mean() + eps) * weight.double())
            row = torch.cat((c, rotate(x[L:], rotations[max(at, 0)], style)))
            latent[t] = row
            if q is not None:
                qo[t] = rotate(q[t].double(), rotations[max(at, 0)], style)
            if at < 0:
                continue
            p = int(table[b, at // page])
            if 0 <= p < pages:
                if scale is None:
                    cache[p, at % page] = to_bf16(row)
                else:
                    cache.view(torch.uint8)[p, at % page] = to_e4m3(row / float(scale)).view(torch.uint8)
    return cache, latent, qo


def softmax_rows(q, keys, values, seen, scale):
    """One sequence: q [n, H, d], keys [m, H or 1, d], values [m, H or 1, e], seen [n, m] bool.  (out, bound) [n, H, e]."""
    n, H, d = q.shape
    out = torch.zeros(n, H, values.shape[-1], dtype=torch.float64)
    bound = torch.full_like(out, 1e-30)  # rows without keys are zeros
    for j in range(n):
        at = seen[j].nonzero()[:, 0]
        if not len(at):
            continue
        for h in range(H):
            k, v = keys[at, h % keys.shape[1]], values[at, h % values.shape[1]]
            s = (k @ q[j, h]) * scale
            w = torch.softmax(s, 0)
            out[j, h] = w @ v
            off = scale * d * 2.0 ** -24 * float((k.abs() @ q[j, h].abs()).max()) + 2.0 ** -22 * float(s.abs().max())
            bound[j, h] = (1.02 * 2.0 ** -8 + 2 * off + len(at) * 2.0 ** -24) * (w @ v.abs()) + 1.01 * 2.0 ** -8 * out[j, h].abs() + 1e-30
    return out, bound


def attention(q, cache, scale, table, lens, starts, softmax_scale):
    """(out, bound) fp64 [T, H, 512]; NaN where no sequence has the token."""
    T, H = q.shape[:2]
    B, W = table.shape
    pages, page = cache.shape[:2]
    out = torch.full((T, H, L), float("nan"), dtype=torch.float64)
    bound = torch.full_like(out, float("nan"))
    for b, (first, n) in enumerate(sequences(starts, B, T)):
        m = min(max(int(lens[b]), 0), W * page)
        rows = torch.zeros(m, ROW, dtype=torch.float64)
        held = torch.zeros(m, dtype=torch.bool)
        for p in range((m + page - 1) // page):
            e = int(table[b, p])
            k = min(page, m - p * page)
            if 0 <= e < pages:
                rows[p * page:p * page + k] = cache[e, :k].double() * (1.0 if scale is None else float(scale))
                held[p * page:p * page + k] = True
        seen = held[None] & (torch.arange(m)[None] <= torch.arange(m - n, m)[:, None])
        out[first:first + n], bound[first:first + n] = softmax_rows(q[first:first + n].double(), rows[:, None], rows[:, None, :L], seen, softmax_scale)
    return out, bound


def expanded(q, kv, k_rope, q_starts, kv_starts, softmax_scale, causal):
    T, H = q.shape[:2]
    S, B = kv.shape[0], len(q_starts) - 1
    out = torch.full((T, H, V), float("nan"), dtype=torch.float64)
    bound = torch.full_like(out, float("nan"))
    for (first, n), (k0, m) in zip(sequences(q_starts, B, T), sequences(kv_starts, B, S)):
        x = kv[k0:k0 + m].double()
        keys = torch.cat((x[..., :NOPE], k_rope[k0:k0 + m].double()[:, None].expand(-1, H, -1)), -1)
        seen = torch.ones(n, m, dtype=torch.bool)
        if causal:
            seen = torch.arange(m)[None] <= torch.arange(m - n, m)[:, None]
        out[first:first + n], bound[first:first + n] = softmax_rows(q[first:first + n].double(), keys, x[..., NOPE:], seen, softmax_scale)
    return out, bound


def heads(x, w):
    x, w = x.double(), w.double()
    out = torch.einsum("thk,hnk->thn", x, w)
    mag = torch.einsum("thk,hnk->thn", x.abs(), w.abs())
    return out, x.shape[-1] * 2.0 ** -24 * mag + 1.01 * 2.0 ** -8 * out.abs() + 1e-30


def rotation_rows(n, device="cpu"):
    angle = torch.arange(n).double()[:, None] * 10000.0 ** (-torch.arange(0, R, 2).double() / R)
    return torch.cat((angle.cos(), angle.sin()), -1).float().to(device)


def check(got, ref, bound):
    """Worst error over its bound where the reference has a value."""
    got = got.cpu().double()
    there = ~torch.isnan(ref)
    assert torch.isfinite(got[there]).all(), "not finite"
    over = (got - ref).abs()[there] / bound[there]
    worst = float(over.max()) if over.numel() else 0.0
    assert worst <= 1.0, f"error {worst:.3g} times its bound"
    return worst
