"""Attention with keys and values from one shared latent vector a token, and
what stands around it in a decode or prompt step, as measured cases: the norm,
rotation and append to a paged cache (latent_append), attention over that cache
in the absorbed form (latent_attention; single tokens and chunks of new tokens),
attention of a prompt over expanded keys and values (latent_attention_expanded),
and the per-head products that lead into and out of the absorbed form
(heads_gemm).

`own` false: elementary torch operations in fp32.  `own` true: the library's
entry points.

A token's cache row has 576 values: a latent of 512 (normed), of which all
heads' keys and values are linear functions, and a rotated key of 64 that the
heads share.  In the absorbed form a head's query is 576 wide and its output
512; in the expanded form they are 128 + 64 and 128.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
L, R, D = 512, 64, 576  # latent, rotated part, cache row
NOPE, V = 128, 128      # expanded: a head's own key part and value
PAGE = 64
EPS = 1e-6
SCALE = 0.0625          # of e4m3 caches
SOFTMAX = (NOPE + R) ** -0.5


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decode token of a model with 128 heads: the smallest call, latency
        dict(name="append-1", op="append", B=1, T=1, prev=200, H=128, cache="bf16", rope="pairs", latent=False),
        # prompts of several requests on a rank with 16 heads, 8-bit cache; the latents are expanded next
        dict(name="append-8192-e4m3", op="append", B=7, T=8192, prev=0, H=16, cache="e4m3", rope="halves", latent=True),
        # one request's next token: latency
        dict(name="decode-1", op="attend", B=1, T=1, len=4000, H=128, cache="bf16"),
        # a decode batch of ragged lengths on a rank with 16 heads, 8-bit cache: cache bandwidth
        dict(name="decode-32-e4m3", op="attend", B=32, T=32, len=24000, H=16, cache="e4m3"),
        # a large decode batch with all heads: cache bandwidth and matrix rate together
        dict(name="decode-128", op="attend", B=128, T=128, len=6000, H=128, cache="bf16"),
        # drafted tokens and short chunks of ragged requests
        dict(name="chunk-12-e4m3", op="attend", B=12, T=150, len=9000, H=20, cache="e4m3"),
        # chunks of two prompts over a long cache: matrix rate
        dict(name="chunk-2", op="attend", B=2, T=512, len=8192, H=128, cache="bf16"),
        # short ragged prompts on a rank with 16 heads
        dict(name="prompt-3", op="prompt", B=3, T=337, prev=0, H=16),
        # a long prompt with all heads: the largest
        dict(name="prompt-4096", op="prompt", B=1, T=4096, prev=0, H=128),
        # a prompt's next chunk over what came before
        dict(name="prompt-chunk-500", op="prompt", B=1, T=500, prev=7600, H=32),
        # one token's queries into the latent space: weights once, latency
        dict(name="heads-1", op="heads", T=1, H=128, N=512, K=128, xs=192),
        # the outputs of a prompt's latents back to the heads' values
        dict(name="heads-2048", op="heads", T=2048, H=128, N=128, K=512, xs=512),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    return rng.choice((8, 16, 16, 32, 64, 128, 128, rng.randint(1, 128)))


def draw(rng):
    op = rng.choice(("append", "decode", "chunk", "prompt", "heads"))
    if op == "append":
        B = _log(rng, 1, 200)
        T = B if rng.random() < 0.4 else _log(rng, B, 8192)
        return dict(op=op, B=B, T=T, prev=rng.randint(0, 300), H=_heads(rng) if T < 3000 else _log(rng, 1, 32),
                    cache=rng.choice(("bf16", "e4m3")), rope=rng.choice(("pairs", "halves")), latent=rng.random() < 0.4)
    if op == "decode":
        H = _heads(rng)
        n = _log(rng, 64, 24000)
        B = _log(rng, 1, max(2, min(160, 768000 // n)))
        return dict(op="attend", B=B, T=B, len=n, H=H, cache=rng.choice(("bf16", "e4m3")))
    if op == "chunk":
        H, B = _heads(rng), _log(rng, 1, 12)
        T = _log(rng, B + 1, 1200)
        q = _most(T, B)
        return dict(op="attend", B=B, T=T, len=_log(rng, q, max(q + 1, min(16000, 500000000 // (B * q * H)))), H=H,
                    cache=rng.choice(("bf16", "e4m3")))
    if op == "prompt":
        B, H = _log(rng, 1, 6), _heads(rng)
        T = _log(rng, max(B, 16), 4000)
        q = _most(T, B)
        room = 1500000000 // (B * q * H)
        return dict(op=op, B=B, T=T, prev=0 if rng.random() < 0.5 or room < q + 16 else _log(rng, 16, min(8000, room - q)), H=H)
    N, K = rng.choice(((512, 128), (128, 512), (32 * rng.randint(1, 16), 32 * rng.randint(1, 16))))
    return dict(op=op, T=_log(rng, 1, 2048), H=_heads(rng), N=N, K=K, xs=K + rng.choice((0, 64)))


def _most(T, B):
    """The most new tokens that a sequence has."""
    return int(np.max(_lengths(T, B)))


def _lengths(T, B):
    """T new tokens over B sequences, unequal: every one has at least one."""
    w = 1.0 + 2.0 * ((np.arange(B) * 7) % 5)
    edges = B + np.floor(np.cumsum(w) / w.sum() * (T - B) + 1e-9)
    starts = np.concatenate([[0], edges - B + np.arange(1, B + 1)]).astype(np.int64)
    return np.diff(starts)


def _totals(case):
    """What each sequence has in the cache, its new tokens among it."""
    B, q = case["B"], _lengths(case["T"], case["B"])
    if case["op"] != "attend":
        return q + (case["prev"] if case["op"] == "prompt" else (case["prev"] * (1 + np.arange(B) % 3)) // 3)
    # spread from a quarter to the whole
    return np.maximum(q, (case["len"] * (1 + (np.arange(B) * 5) % 7 / 2) / 4 if B > 1 else np.array([case["len"]])).astype(np.int64))


def _pairs(case):
    """(query token, key) pairs that the causal rule leaves."""
    q, n = _lengths(case["T"], case["B"]), _totals(case)
    return int(np.sum(q * (n - q) + q * (q + 1) // 2))


def work(case):
    c = case
    if c["op"] == "append":
        # the latents and shared keys in, cache rows out, the new latents out, rotation rows; the queries' rotated part in and out
        row = D * (2 if c["cache"] == "bf16" else 1) + (2 * D if c["latent"] else 0)
        return {"bytes": c["T"] * (2 * D + row + 4 * R + 4 * c["H"] * R) + 2 * L, "flops": c["T"] * (4 * L + 3 * (1 + c["H"]) * R)}
    if c["op"] == "attend":
        n = int(_totals(c).sum())
        return {"bytes": n * D * (2 if c["cache"] == "bf16" else 1) + 2 * c["T"] * c["H"] * (D + L), "flops": 2 * _pairs(c) * c["H"] * (D + L)}
    if c["op"] == "prompt":
        S = int(_totals(c).sum())
        return {"bytes": 2 * (c["T"] * c["H"] * (NOPE + R + V) + S * (c["H"] * (NOPE + V) + R)), "flops": 2 * _pairs(c) * c["H"] * (NOPE + R + V)}
    T, H, N, K = c["T"], c["H"], c["N"], c["K"]
    return {"bytes": 2 * H * (T * K + N * K + T * N), "flops": 2 * T * H * N * K}


# ---------------------------------------------------------------- inputs

def _int(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.int32).to(DEV)


def _starts(a):
    return _int(np.concatenate([[0], np.cumsum(a)]))


def _codes(v):
    """What an e4m3 cache holds of v."""
    return (v * (1.0 / SCALE)).clamp(-448.0, 448.0).to(E4M3)


def _paged(g, case, s):
    """A cache whose pages lie in any order, some unused, and the table."""
    total = _totals(case)
    W, B = int(-(-np.max(total) // PAGE)), case["B"]
    pages = B * W + 5
    s["table"] = torch.randperm(pages, generator=g, device=DEV)[:B * W].view(B, W).to(torch.int32)
    v = torch.randn(pages, PAGE, D, generator=g, device=DEV, dtype=torch.bfloat16)
    s["cache"] = v if case["cache"] == "bf16" else _codes(v.float())
    s["scale"] = torch.full((1,), SCALE, device=DEV) if case["cache"] == "e4m3" else None
    s["kv_lens"] = _int(total)
    q = _lengths(case["T"], B)
    s["q_starts"] = None if case["T"] == B else _starts(q)
    s["most"] = int(q.max())


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    s = dict(case)
    if case["op"] == "append":
        T, H = case["T"], case["H"]
        _paged(g, case, s)
        # the projection's output for the step: the queries' latents (not used here), the latents and the shared key
        s["kv"] = (randn(T, 1536 + D) * torch.exp(0.3 * randn(1536 + D))).bfloat16()[:, 1536:]
        s["weight"] = (1 + 0.2 * randn(L)).bfloat16()
        s["q"] = randn(T, H, NOPE + R).bfloat16()[:, :, NOPE:]
        angle = torch.arange(s["table"].shape[1] * PAGE, device=DEV).double()[:, None] * 10000.0 ** (-torch.arange(0, R, 2, device=DEV).double() / R)
        s["rotations"] = torch.cat((angle.cos(), angle.sin()), -1).float()
    elif case["op"] == "attend":
        _paged(g, case, s)
        s["q"] = (1.2 * randn(case["T"], case["H"], D)).bfloat16()
    elif case["op"] == "prompt":
        T, H, total = case["T"], case["H"], _totals(case)
        S = int(total.sum())
        s["q"] = (1.5 * randn(T, H, NOPE + R)).bfloat16()
        s["kv"] = torch.randn(S, H, NOPE + V, generator=g, device=DEV, dtype=torch.bfloat16)
        s["k_rope"] = randn(S, D).bfloat16()[:, L:]
        s["q_starts"], s["kv_starts"] = _starts(_lengths(T, case["B"])), _starts(total)
        s["most"], s["most_kv"] = _most(T, case["B"]), int(total.max())
    else:
        T, H, N, K = case["T"], case["H"], case["N"], case["K"]
        s["x"] = randn(T, H, case["xs"]).bfloat16()[:, :, :K]
        s["w"] = (randn(H, N, K) / math.sqrt(K)).bfloat16()
    return s


# ---------------------------------------------------------------- passes

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import latency_skinny_gemm_amd as skg
    if s["op"] == "append":
        a = skg.latent_append(s["kv"], s["cache"], s["table"], s["kv_lens"], s["rotations"], q_starts=s["q_starts"], weight=s["weight"],
                              eps=EPS, rope=s["rope"], scale=s["scale"], q_rope=s["q"], latent=s["latent"])
        return {"cache": s["cache"], "q": a.q_rope, "latent": a.latent}
    if s["op"] == "attend":
        return skg.latent_attention(s["q"], s["cache"], s["table"], s["kv_lens"], SOFTMAX, q_starts=s["q_starts"], scale=s["scale"])
    if s["op"] == "prompt":
        return skg.latent_attention_expanded(s["q"], s["kv"], s["k_rope"], s["q_starts"], SOFTMAX, kv_starts=s["kv_starts"])
    return skg.heads_gemm(s["x"], s["w"])


def _places(s, T):
    """Each new token's sequence and its place among that sequence's new tokens."""
    t = torch.arange(T, device=DEV)
    if s["q_starts"] is None:
        return t, torch.zeros_like(t)
    b = torch.searchsorted(s["q_starts"][1:], t.int(), right=True)
    return b, t - s["q_starts"][b]


def _rotate(x, c, sn, rope):
    """x [.., 64] in fp32, its pairs turned by the angles of c and sn [.., 32]."""
    a, b = (x[..., 0::2], x[..., 1::2]) if rope == "pairs" else x.chunk(2, -1)
    u, v = a * c - b * sn, a * sn + b * c
    return torch.stack((u, v), -1).flatten(-2) if rope == "pairs" else torch.cat((u, v), -1)


def _softmax(scores, ok):
    """Weights over the keys that `ok` leaves; a row without any has none."""
    scores.masked_fill_(~ok, -math.inf)
    m = scores.amax(-1, keepdim=True)
    p = torch.exp(scores.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)))
    n = p.sum(-1, keepdim=True)
    return p.div_(torch.where(n == 0, torch.ones_like(n), n))


def _run_plain(s):
    T = s["T"]
    if s["op"] == "heads":
        return torch.matmul(s["x"].float().transpose(0, 1), s["w"].float().transpose(1, 2)).transpose(0, 1).bfloat16()
    b, j = _places(s, T)
    n_new = torch.ones_like(b) if s["q_starts"] is None else (s["q_starts"].diff()[b])
    if s["op"] == "append":
        at = s["kv_lens"][b].long() - n_new + j
        x = s["kv"].float()
        c = x[:, :L]
        c = c / torch.sqrt((c * c).mean(-1, keepdim=True) + EPS) * s["weight"].float()
        cos, sin = s["rotations"][at].chunk(2, -1)
        row = torch.cat((c, _rotate(x[:, L:], cos, sin, s["rope"])), -1)
        page = s["table"][b, at // PAGE].long()
        if s["scale"] is None:
            s["cache"][page, at % PAGE] = row.bfloat16()
        else:
            s["cache"].view(torch.uint8)[page, at % PAGE] = (row / s["scale"]).clamp(-448.0, 448.0).to(E4M3).view(torch.uint8)
        q = _rotate(s["q"].float(), cos[:, None], sin[:, None], s["rope"]).bfloat16()
        return {"cache": s["cache"], "q": q, "latent": row.bfloat16() if s["latent"] else None}
    B, H, most = s["B"], s["H"], s["most"]
    q = s["q"].new_zeros(B, most, H, s["q"].shape[-1], dtype=torch.float32)
    q[b, j] = s["q"].float()
    new = n_new.new_zeros(B).index_copy(0, b, n_new)
    if s["op"] == "attend":
        rows = s["cache"].view(torch.uint8)[s["table"].long()].view(s["cache"].dtype).flatten(1, 2).float()
        if s["scale"] is not None:
            rows = rows * s["scale"]
        last = (s["kv_lens"] - new)[:, None] + torch.arange(most, device=DEV)
        ok = torch.arange(rows.shape[1], device=DEV) <= last[..., None]
        scores = torch.matmul(q.flatten(1, 2), rows.transpose(1, 2)).mul_(SOFTMAX)
        p = _softmax(scores.unflatten(1, (most, H)), ok[:, :, None])
        out = torch.matmul(p.flatten(1, 2), rows[..., :L]).unflatten(1, (most, H))
        return out[b, j].bfloat16()
    n = s["kv_starts"].diff().long()
    t = torch.arange(s["kv"].shape[0], device=DEV)
    kb = torch.searchsorted(s["kv_starts"][1:], t.int(), right=True)
    kj = t - s["kv_starts"][kb]
    k = q.new_zeros(B, s["most_kv"], H, NOPE + R + V)
    k[kb, kj] = torch.cat((s["kv"][..., :NOPE], s["k_rope"][:, None].expand(-1, H, -1), s["kv"][..., NOPE:]), -1).float()
    k = k.transpose(1, 2).contiguous()
    last = (n - new)[:, None] + torch.arange(most, device=DEV)
    ok = torch.arange(s["most_kv"], device=DEV) <= last[..., None]
    scores = torch.matmul(q.transpose(1, 2), k[..., :NOPE + R].transpose(2, 3)).mul_(SOFTMAX)
    out = torch.matmul(_softmax(scores, ok[:, None]), k[..., NOPE + R:]).transpose(1, 2)
    return out[b, j].bfloat16()


# ---------------------------------------------------------------- in 64 bits

def _attend64(q, k, v, before):
    """q [n, H, d], k [m, H or 1, d], v [m, H or 1, e]: token i sees keys 0 .. before + i."""
    out = torch.empty(*q.shape[:2], v.shape[-1], dtype=torch.float64, device=DEV)
    keys = torch.arange(k.shape[0], device=DEV)
    for h in range(q.shape[1]):
        kh, vh = k[:, h % k.shape[1]], v[:, h % v.shape[1]]
        for i in range(0, q.shape[0], 1024):
            z = (q[i:i + 1024, h] @ kh.t()) * SOFTMAX
            hidden = keys[None] > before + torch.arange(i, min(i + 1024, q.shape[0]), device=DEV)[:, None]
            out[i:i + 1024, h] = torch.softmax(z.masked_fill(hidden, -math.inf), -1) @ vh
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "heads":
        return torch.stack([s["x"][:, h].double() @ s["w"][h].double().t() for h in range(case["H"])], 1)
    q_new, total = _lengths(case["T"], case["B"]).tolist(), _totals(case).tolist()
    if case["op"] == "append":
        table, t0 = s["table"].cpu().numpy(), 0
        cache = s["cache"].double()
        q, latent = torch.empty_like(s["q"], dtype=torch.float64), torch.empty(case["T"], D, dtype=torch.float64, device=DEV)
        for b, (m, n) in enumerate(zip(q_new, total)):
            at = np.arange(n - m, n)
            x = s["kv"][t0:t0 + m].double()
            z = torch.complex(*s["rotations"][torch.from_numpy(at).to(DEV)].double().chunk(2, -1))

            def turned(y, z):
                pairs = y.unflatten(-1, (-1, 2)) if case["rope"] == "pairs" else y.unflatten(-1, (2, -1)).transpose(-1, -2)
                w = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z)
                return (w if case["rope"] == "pairs" else w.transpose(-1, -2)).flatten(-2)

            c = x[:, :L] * torch.rsqrt(x[:, :L].square().mean(-1, keepdim=True) + EPS) * s["weight"].double()
            row = torch.cat((c, turned(x[:, L:], z)), -1)
            q[t0:t0 + m], latent[t0:t0 + m] = turned(s["q"][t0:t0 + m].double(), z[:, None]), row
            if case["cache"] == "e4m3":
                row = row / s["scale"].double()
                step = torch.exp2(torch.floor(torch.log2(row.abs().clamp(min=2.0 ** -6))) - 3)
                row = (torch.round(row / step) * step).clamp(-448.0, 448.0)
            cache[torch.from_numpy(table[b, at // PAGE]).long().to(DEV), torch.from_numpy(at % PAGE).to(DEV)] = row
            t0 += m
        return {"cache": cache, "q": q, "latent": latent if case["latent"] else None}
    out, t0, s0 = [], 0, 0
    for b, (m, n) in enumerate(zip(q_new, total)):
        q = s["q"][t0:t0 + m].double()
        if case["op"] == "attend":
            pages = s["cache"].view(torch.uint8)[s["table"][b].long()].view(s["cache"].dtype)
            rows = pages.flatten(0, 1)[:n].double()
            if case["cache"] == "e4m3":
                rows = rows * s["scale"].double()
            if m == 1:  # all heads at once: they share the keys
                p = torch.softmax(q[0] @ rows.t() * SOFTMAX, -1)
                out.append((p @ rows[:, :L])[None])
            else:
                out.append(_attend64(q, rows[:, None], rows[:, None, :L], n - m))
        else:
            kv = s["kv"][s0:s0 + n].double()
            shared = s["k_rope"][s0:s0 + n].double()[:, None].expand(-1, case["H"], -1)
            out.append(_attend64(q, torch.cat((kv[..., :NOPE], shared), -1), kv[..., NOPE:], n - m))
        t0, s0 = t0 + m, s0 + n
    return torch.cat(out)
