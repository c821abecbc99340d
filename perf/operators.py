"""The operators around the small-M products of a mixture-of-experts decode
step, as measured cases: root-mean-square norm with the residual's addition
and 8-bit outputs (rmsnorm), routing to experts (route), microscaled
quantisation (quant_mx, dequant_mx) and product (gemm_mxfp4), and the routed
experts' feed-forward in MXFP4 (moe_mxfp4).

`own` false: elementary torch operations in fp32.  `own` true: the library's
entry points.

Microscaling, everywhere below: 32 consecutive values of a row share one
power of two 2^(e - 127) (byte e), the smallest with
amax <= largest code * 2^(e - 127); largest code 448 (e4m3) or 6 (e2m1).
e is clamped to [0, 254]; an all-zero block takes e = 127.  Codes are the
nearest, ties to even.  Two e2m1 codes share a byte, the even index low.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
EPS = 1e-6
# e2m1 magnitudes by code
FP4 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decode token entering a per-tensor FP8 linear: the smallest call, latency
        dict(name="norm-1-e4m3", op="norm", M=1, K=7168, out="e4m3", residual=True),
        # a long prompt entering an MX linear: HBM bound
        dict(name="norm-8192-mx", op="norm", M=8192, K=7168, out="mx", residual=True),
        # one decode token over 256 experts in 8 groups, balanced by a bias
        dict(name="route-1", op="route", T=1, E=256, k=8, scores="sigmoid", bias=True, groups=8,
             top_groups=4, renorm=True, dtype="f32"),
        # a long prompt over 384 experts, softmax of bf16 logits
        dict(name="route-16384", op="route", T=16384, E=384, k=8, scores="softmax", bias=False,
             groups=1, top_groups=1, renorm=True, dtype="bf16"),
        # activations of a decode batch to MX e4m3
        dict(name="quant-64-e4m3", op="quant", M=64, K=2880, fmt="e4m3"),
        # a weight matrix to MXFP4
        dict(name="quant-4096-e2m1", op="quant", M=4096, K=7168, fmt="e2m1"),
        # one decode token through a 4-bit linear: weight bandwidth and latency
        dict(name="linear-1", op="linear", M=1, N=2112, K=7168, fmt="e4m3", bias=False),
        # a ragged batch through a ragged linear
        dict(name="linear-37", op="linear", M=37, N=1111, K=2880, fmt="e4m3", bias=True),
        # the largest batch the library's products take, 4-bit activations
        dict(name="linear-512", op="linear", M=512, N=4096, K=7168, fmt="e2m1", bias=False),
        # one decode token through its experts
        dict(name="experts-1", op="experts", T=1, H=2880, I=2880, E=128, k=4, fmt="e4m3", absent=0.0),
        # a decode batch on a rank that holds half of the experts chosen, 4-bit activations
        dict(name="experts-40", op="experts", T=40, H=4096, I=1408, E=64, k=8, fmt="e2m1", absent=0.5),
        # a prompt
        dict(name="experts-2048", op="experts", T=2048, H=2880, I=2880, E=128, k=4, fmt="e4m3", absent=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _odd32(rng, lo, hi):
    """An odd multiple of 32 between lo and hi, even over the logarithm."""
    return min(max(_log(rng, lo, hi) // 32 | 1, 3), (hi // 32 - 1) | 1) * 32


def draw(rng):
    op = rng.choice(("norm", "route", "quant", "linear", "experts"))
    if op == "norm":
        return dict(op=op, M=_log(rng, 1, 7000), K=_odd32(rng, 512, 8192),
                    out=rng.choice(("bf16", "e4m3", "mx")), residual=rng.random() < 0.75)
    if op == "route":
        groups = rng.choice((1, 1, 4, 8))
        E = groups * rng.randint(max(1, 16 // groups), 384 // groups)
        top_groups = rng.randint(1, groups)
        scores = rng.choice(("softmax", "sigmoid"))
        return dict(op=op, T=_log(rng, 1, 16384), E=E, k=rng.randint(1, min(10, top_groups * (E // groups))),
                    scores=scores, bias=scores == "sigmoid" and rng.random() < 0.7, groups=groups,
                    top_groups=top_groups, renorm=rng.random() < 0.7, dtype=rng.choice(("f32", "bf16")))
    if op == "quant":
        return dict(op=op, M=_log(rng, 1, 3500), K=_odd32(rng, 512, 8192), fmt=rng.choice(("e4m3", "e2m1")))
    if op == "linear":
        return dict(op=op, M=_log(rng, 1, 512), N=_log(rng, 64, 4000), K=_odd32(rng, 1024, 7168),
                    fmt=rng.choice(("e4m3", "e2m1")), bias=rng.random() < 0.5)
    return dict(op=op, T=_log(rng, 1, 2048), H=_odd32(rng, 1024, 2880), I=_odd32(rng, 256, 2880),
                E=rng.randint(8, 128), k=rng.randint(1, 4), fmt=rng.choice(("e4m3", "e2m1")),
                absent=rng.choice((0.0, 0.0, 0.5)))


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["M"] * c["K"]
        # x, the gains and the output (its values in bf16, its codes in 8 bits); the residual in and out
        return {"bytes": n * (2 + (1 if c["out"] == "e4m3" else 2)) + (4 * n if c["residual"] else 0) + 2 * c["K"],
                "flops": 6 * n}
    if c["op"] == "route":
        return {"bytes": c["T"] * (c["E"] * (4 if c["dtype"] == "f32" else 2) + 8 * c["k"]) + (4 * c["E"] if c["bias"] else 0),
                "flops": 4 * c["T"] * c["E"]}
    if c["op"] == "quant":
        return {"bytes": 4 * c["M"] * c["K"], "flops": 3 * c["M"] * c["K"]}  # bf16 in, the values in bf16 out
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": N * K * 17 / 32 + 2 * M * K + 2 * M * N + (2 * N if c["bias"] else 0), "flops": 2 * M * N * K}
    T, H, I, E, k = c["T"], c["H"], c["I"], c["E"], c["k"]
    here = 1 - c["absent"]
    touched = E * (1 - (1 - k * here / E) ** T)  # experts that at least one token chose, expected
    return {"bytes": touched * 3 * H * I * 17 / 32 + 4 * T * H + 8 * T * k, "flops": 6 * T * k * here * H * I}


# ---------------------------------------------------------------- inputs

def _mx_exponent(amax, fmt):
    """The biased exponent byte (int32) of blocks whose largest magnitudes are amax (fp32)."""
    m, p = torch.frexp(amax)  # amax = m * 2^p, 0.5 <= m < 1
    top, emax = (0.875, 9) if fmt == "e4m3" else (0.75, 3)  # 448 = 0.875 * 2^9, 6 = 0.75 * 2^3
    e = (p - emax + (m > top) + 127).clamp(0, 254)
    return torch.where(amax > 0, e, torch.full_like(e, 127))


def _fp4_code(v):
    """e2m1 codes (uint8) of v, nearest with ties to the even code."""
    a = v.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return code | (torch.signbit(v).to(torch.uint8) << 3)


def _mx_codes(v, fmt):
    """fp32 [..., K] -> (e4m3 [..., K] or packed uint8 [..., K/2], e uint8 [..., K/32])."""
    b = v.unflatten(-1, (-1, 32))
    e = _mx_exponent(b.abs().amax(-1), fmt)
    q = torch.ldexp(b, (127 - e).unsqueeze(-1)).flatten(-2)
    if fmt == "e4m3":
        return q.to(E4M3), e.to(torch.uint8)
    c = _fp4_code(q)
    return c[..., 0::2] | (c[..., 1::2] << 4), e.to(torch.uint8)


def _mx_values(codes, e, dtype=torch.float32):
    """What MX codes stand for."""
    if codes.dtype == torch.uint8:
        table = torch.tensor(FP4 + tuple(-v for v in FP4), dtype=dtype, device=codes.device)
        v = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1).flatten(-2)
    else:
        v = codes.to(dtype)
    return torch.ldexp(v.unflatten(-1, (-1, 32)), (e.to(torch.int32) - 127).unsqueeze(-1)).flatten(-2)


def _mx_round(v, fmt):
    """v with its values replaced by what their MX codes stand for, in v's type."""
    return _mx_values(*_mx_codes(v.float(), fmt), dtype=v.dtype)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _weights4(g, n, k, experts=None):
    """N(0, 1/k) weights in MXFP4; several experts one after another, so that the fp32 values stay small."""
    parts = [_mx_codes(_randn(g, n, k) / math.sqrt(k), "e2m1") for _ in range(experts or 1)]
    if experts is None:
        return parts[0]
    return torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = dict(case)
    if case["op"] == "norm":
        M, K = case["M"], case["K"]
        # a residual stream has a few channels far above the others
        channels = torch.exp(0.5 * _randn(g, K))
        s["x"] = (_randn(g, M, K) * channels).bfloat16()
        s["r"] = (2 * _randn(g, M, K) * channels).bfloat16() if case["residual"] else None
        s["g"] = (1 + 0.2 * _randn(g, K)).bfloat16()
        s["scale"] = torch.full((1,), 6.0 / 448.0, device=DEV)
    elif case["op"] == "route":
        T, E = case["T"], case["E"]
        l = 1.5 * _randn(g, T, E) + 0.5 * _randn(g, E)
        s["l"] = l if case["dtype"] == "f32" else l.bfloat16()
        s["b"] = 0.05 * _randn(g, E) if case["bias"] else None
    elif case["op"] == "quant":
        s["x"] = (_randn(g, case["M"], case["K"]) * torch.exp(0.5 * _randn(g, case["K"]))).bfloat16()
    elif case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        s["x"] = _randn(g, M, K).bfloat16()
        s["w"] = _weights4(g, N, K)
        s["b"] = (0.3 * _randn(g, N)).bfloat16() if case["bias"] else None
        if own:  # the handle that a program keeps of its weight
            import latency_skinny_gemm_amd as skg
            s["w4"] = skg.mxfp4_pack(*s["w"])
    else:
        T, H, I, E, k = case["T"], case["H"], case["I"], case["E"], case["k"]
        s["x"] = _randn(g, T, H).bfloat16()
        top = (_randn(g, T, E) + 0.5 * _randn(g, E)).topk(k, -1)  # some experts are chosen more often
        s["weights"] = torch.softmax(top.values, -1)
        away = torch.rand(T, k, generator=g, device=DEV) < case["absent"]  # experts of other ranks
        s["ids"] = torch.where(away, torch.full_like(top.indices, -1), top.indices).int()
        s["w13"] = _weights4(g, 2 * I, H, E)
        s["w2"] = _weights4(g, H, I, E)
        if own:
            import latency_skinny_gemm_amd as skg
            s["w13_4"], s["w2_4"] = skg.mxfp4_pack(*s["w13"]), skg.mxfp4_pack(*s["w2"])
    return s


# ---------------------------------------------------------------- passes

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import latency_skinny_gemm_amd as skg
    if s["op"] == "norm":
        n = skg.rmsnorm(s["x"], s["g"], residual=s["r"], eps=EPS, out_format=s["out"],
                        scale=s["scale"] if s["out"] == "e4m3" else None)
        y = skg.dequant_mx(n.y, n.e8m0) if s["out"] == "mx" else n.y
        return {"y": y, "residual": n.residual}
    if s["op"] == "route":
        w, ids = skg.route(s["l"], s["k"], scores=s["scores"], bias=s["b"], groups=s["groups"],
                           top_groups=s["top_groups"], renormalize=s["renorm"])
        return {"weights": w, "ids": ids}
    if s["op"] == "quant":
        return skg.dequant_mx(*skg.quant_mx(s["x"], s["fmt"]))
    if s["op"] == "linear":
        return skg.gemm_mxfp4(s["x"], s["w4"], x_format=s["fmt"], bias=s["b"])
    return skg.moe_mxfp4(s["x"], s["ids"], s["weights"], s["w13_4"], s["w2_4"], x_format=s["fmt"])


def _norm(s, dtype):
    t = s["x"].to(dtype)
    if s["r"] is not None:
        t = t + s["r"].to(dtype)
    y = t / torch.sqrt((t * t).mean(-1, keepdim=True) + EPS) * s["g"].to(dtype)
    return t if s["r"] is not None else None, y


def _run_plain(s):
    if s["op"] == "norm":
        t, y = _norm(s, torch.float32)
        if s["out"] == "e4m3":
            y = (y * (1.0 / s["scale"])).clamp(-448.0, 448.0).to(E4M3)
        else:
            y = (y if s["out"] == "bf16" else _mx_round(y, "e4m3")).bfloat16()
        return {"y": y, "residual": None if t is None else t.bfloat16()}
    if s["op"] == "route":
        return _route_plain(s)
    if s["op"] == "quant":
        return _mx_round(s["x"].float(), s["fmt"]).bfloat16()
    if s["op"] == "linear":
        out = _mx_round(s["x"].float(), s["fmt"]) @ _mx_values(*s["w"]).t()
        return (out if s["b"] is None else out + s["b"].float()).bfloat16()
    return _experts_plain(s)


def _first(key, n):
    """Indices of the n largest of each row, equal ones in the order of their index."""
    return torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :n]


def _route_plain(s):
    l = s["l"].float()
    if s["scores"] == "softmax":
        p = torch.exp(l - l.amax(-1, keepdim=True))
        score, key = p / p.sum(-1, keepdim=True), l
    else:
        score = 1.0 / (1.0 + torch.exp(-l))
        key = score if s["b"] is None else score + s["b"]
    if s["groups"] > 1:
        per = key.unflatten(-1, (s["groups"], -1))
        best = torch.sort(per, dim=-1, descending=True).values
        best = best[..., 0] if s["scores"] == "softmax" else best[..., :2].sum(-1)
        kept = torch.zeros_like(best, dtype=torch.bool).scatter(-1, _first(best, s["top_groups"]), True)
        key = torch.where(kept.unsqueeze(-1), per, torch.full_like(per, -math.inf)).flatten(-2)
    ids = _first(key, s["k"])
    w = score.gather(-1, ids)
    if s["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return {"weights": w, "ids": ids.int()}


def _swiglu(h):
    g, u = h.chunk(2, -1)
    return g / (1.0 + torch.exp(-g)) * u


def _experts_plain(s):
    """Few pairs: every pair gathers its expert's weights.  Many: the pairs of an expert side by side, one product over experts."""
    T, k, E = s["T"], s["k"], s["E"]
    x = _mx_round(s["x"].float(), s["fmt"])
    ids, w = s["ids"].long().flatten(), s["weights"].flatten()
    here = ids >= 0
    if T * k <= 32:
        e = ids.clamp(min=0)
        rows = x.repeat_interleave(k, 0)
        h = (_mx_values(s["w13"][0][e], s["w13"][1][e]) * rows.unsqueeze(1)).sum(-1)
        h = _mx_round(_swiglu(h), s["fmt"])
        y = (_mx_values(s["w2"][0][e], s["w2"][1][e]) * h.unsqueeze(1)).sum(-1)
        y = torch.where(here.unsqueeze(-1), y, torch.zeros_like(y))
    else:
        slot = torch.where(here, ids, torch.full_like(ids, E))
        order = torch.sort(slot, stable=True).indices
        count = torch.bincount(slot, minlength=E + 1)
        start = torch.cumsum(count, 0) - count
        at = torch.empty_like(ids)
        at[order] = torch.arange(T * k, device=ids.device) - start[slot[order]]
        most = max(1, int(count[:E].max()))
        e, at, pair = slot[here], at[here], torch.arange(T * k, device=ids.device)[here]
        rows = x.new_zeros(E, most, x.shape[1])
        rows[e, at] = x[pair // k]
        h = torch.bmm(rows, _mx_values(*s["w13"]).transpose(1, 2).contiguous())
        h = _mx_round(_swiglu(h), s["fmt"])
        h = torch.bmm(h, _mx_values(*s["w2"]).transpose(1, 2).contiguous())
        y = x.new_zeros(T * k, x.shape[1])
        y[pair] = h[e, at]
    return (y * w.unsqueeze(-1)).unflatten(0, (T, k)).sum(1).bfloat16()


# ---------------------------------------------------------------- in 64 bits

def _exact_value(codes, e):
    """MX codes in 64 bits, decoded from their bits."""
    if codes.dtype == torch.uint8:
        c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()
        sign, exp, man = c >> 3, (c >> 1) & 3, (c & 1).double()
        v = torch.where(exp > 0, (1 + man / 2) * torch.exp2(exp.double() - 1), man / 2)
    else:
        c = codes.view(torch.uint8).int()
        sign, exp, man = c >> 7, (c >> 3) & 15, (c & 7).double()
        v = torch.where(exp > 0, (1 + man / 8) * torch.exp2(exp.double() - 7), man / 8 * 2.0 ** -6)
    v = torch.where(sign > 0, -v, v)
    return (v.unflatten(-1, (-1, 32)) * torch.exp2(e.double() - 127).unsqueeze(-1)).flatten(-2)


def _exact_round(v, fmt):
    """64-bit v to the nearest MX value: the quotient by the step of its binade, rounded to an even whole number."""
    b = v.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    largest, low, bits = (448.0, -6, 3) if fmt == "e4m3" else (6.0, 0, 1)
    e = torch.ceil(torch.log2(torch.where(amax > 0, amax, torch.full_like(amax, largest)) / largest))
    e = torch.where(torch.exp2(e - 1) * largest >= amax, e - 1, e)  # log2 rounded up past a power of two
    e = torch.where(torch.exp2(e) * largest < amax, e + 1, e)
    e = torch.where(amax > 0, e.clamp(-127, 127), torch.zeros_like(e))
    q = b / torch.exp2(e)
    binade = torch.floor(torch.log2(q.abs().clamp(min=2.0 ** low)))
    step = torch.exp2(binade - bits)
    return (torch.round(q / step) * step * torch.exp2(e)).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        t, y = _norm(s, torch.float64)
        if case["out"] == "e4m3":
            y = y / s["scale"].double()
            binade = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
            step = torch.exp2(binade - 3)
            y = (torch.round(y / step) * step).clamp(-448.0, 448.0)
        elif case["out"] == "mx":
            y = _exact_round(y, "e4m3")
        return {"y": y, "residual": t}
    if case["op"] == "route":
        l = s["l"].double()
        score = torch.softmax(l, -1) if case["scores"] == "softmax" else torch.sigmoid(l)
        key = score if s["b"] is None else score + s["b"].double()
        if case["groups"] > 1:
            per = key.unflatten(-1, (case["groups"], -1))
            n = 1 if case["scores"] == "softmax" else min(2, per.shape[-1])
            best = per.topk(n, -1).values.sum(-1)
            out = best < best.topk(case["top_groups"], -1).values[..., -1:]
            key = per.masked_fill(out.unsqueeze(-1), -math.inf).flatten(-2)
        w = score.gather(-1, torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :case["k"]])
        return {"weights": w / w.sum(-1, keepdim=True) if case["renorm"] else w, "ids": None}
    if case["op"] == "quant":
        return _exact_round(s["x"].double(), case["fmt"])
    if case["op"] == "linear":
        out = _exact_round(s["x"].double(), case["fmt"]) @ _exact_value(*s["w"]).t()
        return out if s["b"] is None else out + s["b"].double()
    x = _exact_round(s["x"].double(), case["fmt"])
    y = torch.zeros_like(x)
    for e in range(case["E"]):
        t, j = (s["ids"] == e).nonzero(as_tuple=True)
        g, u = (x[t] @ _exact_value(s["w13"][0][e], s["w13"][1][e]).t()).chunk(2, -1)
        h = _exact_round(g * torch.sigmoid(g) * u, case["fmt"])
        y.index_add_(0, t, (h @ _exact_value(s["w2"][0][e], s["w2"][1][e]).t()) * s["weights"][t, j].double().unsqueeze(-1))
    return y
