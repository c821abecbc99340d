"""The operators of skinny_moe.h on the GPU against plain implementations in
64 bits (tests/mx_reference.py), through the Python binding.

Tolerances, derived:
- MX codes of bf16 values are decided exactly on both sides: bit for bit.
- rmsnorm: the fp32 chain (one addition, a sum of K squares in a tree of at
  most K / 64 / 8 + 10 sequential additions a lane, sqrt, divide, two
  products) stays within 2^-16 of the value for the K used here; the output's
  rounding adds half a step of its type.  Codes may differ by one step where
  the value lies within 2^-16 of a tie, or its block's largest within 2^-16 of
  the range's end (then by the step of the doubled scale).
- route: fp32 scores are within 2^-20 of the exact ones, so the keys of the
  chosen experts must match the exact best keys, place by place, within 2^-19
  (+ 2^-19 of the key); weights within 2^-18 of the exact weight.
- products: small integers are exact (bit for bit); otherwise the library's
  own bound, |err| <= 2^-7 |ref| + 1e-3 sqrt(K) rms(ref).
- experts: the product's bound does not apply twice over, so from the parts:
  the output's rounding 2^-8 |ref| at most; and the hidden codes that flip
  because the products' sums differ from the exact ones: the instruction keeps
  about 2^-14 of its largest term, so fewer than one code in 100 lies that near a
  tie; a flip moves a value by at most 2^-2 (e2m1) of it, so the sum by about
  sqrt(1/100) * 2^-2 * rms = 0.025 rms; twice that is allowed.
  That is a bound on many flips; a single one of a value far above the rest, or
  of a block's scale, is accounted for itself: the reference has both codes
  where a value lies within 2^-13 of a tie.
"""
import importlib.util
import math
import os

import numpy as np
import pytest
import torch

from tests import mx_reference as ref
from workloads import inputs as gen

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
FORMATS = ("e4m3", "e2m1")


@pytest.fixture(scope="module")
def skg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import latency_skinny_gemm_amd as m
    m.lib()
    return m


def _randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def _np(t):
    """Codes and scales as uint8 numpy."""
    return t.cpu().view(torch.uint8).numpy()


# ------------------------------------------------------------ MX codes

@pytest.mark.parametrize("fmt", FORMATS)
def test_quant_every_bf16_code(skg, fmt):
    """Every bf16 bit pattern, finite ones in blocks of like size and of mixed size."""
    bits = np.arange(65536, dtype=np.uint16)
    same = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).reshape(-1, 64)
    finite = same.reshape(-1)[torch.isfinite(same.reshape(-1))]
    mixed = finite[torch.randperm(len(finite), generator=torch.Generator().manual_seed(1))]
    for x in (same, mixed[:len(finite) // 64 * 64].reshape(-1, 64)):
        q, e = skg.quant_mx(x.to(DEV), fmt)
        codes, er = ref.quantise(ref.f64(x), fmt)
        assert np.array_equal(_np(e), er)
        ok = np.repeat(er != 255, 32, -1)
        got = ref.unpack_bytes(_np(q), fmt)
        assert np.array_equal(got[ok], codes[ok])
        back = skg.dequant_mx(q, e)
        want = torch.from_numpy(ref.dequantise(codes, er, fmt)).float().bfloat16()
        want[torch.from_numpy(~ok)] = math.nan
        assert torch.equal(torch.isnan(back.cpu()), torch.isnan(want))
        fine = ~torch.isnan(want)
        assert torch.equal(back.cpu()[fine], want[fine])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("shape", [(1, 32), (3, 32), (1, 2880), (5, 160), (2, 3, 96), (257, 544)])
def test_quant_shapes_and_round_trip(skg, fmt, shape):
    x = (_randn(sum(shape), *shape) * torch.exp2(torch.randint(-9, 9, shape).float())).bfloat16()
    q, e = skg.quant_mx(x.to(DEV), fmt)
    codes, er = ref.quantise(ref.f64(x), fmt)
    assert np.array_equal(_np(e), er) and np.array_equal(ref.unpack_bytes(_np(q), fmt), codes)
    back = skg.dequant_mx(q, e)
    assert back.shape == x.shape
    assert np.array_equal(ref.f64(back), ref.dequantise(codes, er, fmt))
    # values that codes stand for come back as the same codes' values
    again = skg.dequant_mx(*skg.quant_mx(back, fmt))
    assert torch.equal(again, back)


def test_dequant_every_scale(skg):
    e = torch.arange(256, dtype=torch.uint8).reshape(256, 1)
    for fmt, q in (("e4m3", torch.arange(32, dtype=torch.uint8).repeat(256, 1) * 4),
                   ("e2m1", (torch.arange(16, dtype=torch.uint8) * 17).repeat(256, 1))):
        qd = q.to(DEV)
        out = skg.dequant_mx(qd.view(torch.float8_e4m3fn) if fmt == "e4m3" else qd, e.to(DEV))
        want = torch.from_numpy(ref.dequantise(ref.unpack_bytes(q.numpy(), fmt), e.numpy().astype(np.int64), fmt))
        want = want.to(torch.bfloat16)
        nan = torch.isnan(want)
        assert torch.equal(torch.isnan(out.cpu()), nan)
        assert torch.equal(out.cpu()[~nan], want[~nan])


# ------------------------------------------------------------ norm

NORM_SIZES = [(1, 32), (3, 96), (5, 1024), (2, 1056), (1, 7168), (67, 2880), (3, 8224), (2, 16384),
              (2, 16416), (1, 65536), (1026, 4160)]


def _norm_close(skg, out, y, fmt, scale):
    """out (device) against exact y, by the bounds above."""
    slack = 2.0 ** -16 * np.abs(y)
    if fmt == "bf16":
        step = np.exp2(np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -126))) - 7)
        assert np.all(np.abs(ref.f64(out.y) - y) <= step / 2 + slack)
        return
    if fmt == "e4m3":
        got = ref.dequantise(_np(out.y).astype(np.int64), np.full((*y.shape[:-1], y.shape[-1] // 32), 127), "e4m3")
        t = np.clip(y / scale, -448, 448)
        step = np.exp2(np.floor(np.log2(np.maximum(np.abs(t), 2.0 ** -6))) - 3)
        assert np.all(np.abs(got - t) <= step / 2 + 2.0 ** -15 * np.abs(t))
        return
    codes, e = ref.quantise(y, "e4m3")
    ge = _np(out.e8m0).astype(np.int64)
    assert np.abs(ge - e).max() <= 1
    near = np.abs(np.log2(np.abs(y).reshape(*e.shape, 32).max(-1) / 448.0) % 1.0 - 0.5) > 0.5 - 2.0 ** -14
    assert np.all((ge == e) | near)
    got = ref.dequantise(_np(out.y).astype(np.int64), ge, "e4m3")
    f = np.exp2(np.repeat(ge, 32, -1) - 127.0)
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(y / f), 2.0 ** -6))) - 3) * f
    assert np.all(np.abs(got - y) <= step / 2 + 2.0 ** -15 * np.abs(y))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "mx"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("M,K", NORM_SIZES)
def test_rmsnorm(skg, M, K, residual, fmt):
    x, w = _randn(K, M, K).bfloat16(), (1 + 0.3 * _randn(K + 1, K)).bfloat16()
    r = (3 * _randn(K + 2, M, K)).bfloat16() if residual else None
    scale = 0.0123 if fmt == "e4m3" else None
    out = skg.rmsnorm(x.to(DEV), w.to(DEV), residual=None if r is None else r.to(DEV), eps=1e-5,
                      out_format=fmt, scale=None if scale is None else torch.tensor([scale], device=DEV))
    s, y = ref.norm(x, r, w, 1e-5)
    _norm_close(skg, out, y, fmt, None if scale is None else float(np.float32(scale)))
    if r is None:
        assert out.residual is None
    else:  # bf16 of the fp32 sum
        assert torch.equal(out.residual.cpu(), (x.float() + r.float()).bfloat16())
    assert (out.e8m0 is None) == (fmt != "mx")


@pytest.mark.parametrize("K", [8, 24, 1016, 1032, 16392])
def test_rmsnorm_lengths_off_the_vector(skg, K):
    x, w = _randn(K, 6, K).bfloat16(), _randn(K + 1, K).bfloat16()
    out = skg.rmsnorm(x.to(DEV), w.to(DEV))
    _norm_close(skg, out, ref.norm(x, None, w, 1e-6)[1], "bf16", None)


def test_rmsnorm_in_place_and_leading_dimensions(skg):
    x, r, w = _randn(1, 2, 3, 320).bfloat16(), _randn(2, 2, 3, 320).bfloat16(), _randn(3, 320).bfloat16()
    want = skg.rmsnorm(x.to(DEV), w.to(DEV), residual=r.to(DEV))
    for into_x in (False, True):
        xd, rd = x.to(DEV), r.to(DEV)
        got = skg.rmsnorm(xd, w.to(DEV), residual=rd, residual_out=xd if into_x else rd)
        assert got.residual is (xd if into_x else rd)
        assert torch.equal(got.y, want.y) and torch.equal(got.residual, want.residual)
    # rows longer than the registers hold are read twice: in place all the same
    x, r, w = _randn(4, 2, 20000).bfloat16(), _randn(5, 2, 20000).bfloat16(), _randn(6, 20000).bfloat16()
    want = skg.rmsnorm(x.to(DEV), w.to(DEV), residual=r.to(DEV))
    rd = r.to(DEV)
    got = skg.rmsnorm(x.to(DEV), w.to(DEV), residual=rd, residual_out=rd)
    assert torch.equal(got.y, want.y) and torch.equal(rd, want.residual)


def test_rmsnorm_zero_infinite_and_nan_rows(skg):
    x = _randn(7, 5, 64).bfloat16()
    x[0] = 0
    x[1, 5] = math.inf
    x[2, 40] = math.nan
    w = torch.ones(64, dtype=torch.bfloat16)
    out = skg.rmsnorm(x.to(DEV), w.to(DEV)).y.cpu()
    assert torch.all(out[0] == 0)
    assert math.isnan(out[1, 5]) and torch.all(out[1, :5] == 0)
    assert torch.all(torch.isnan(out[2]))
    assert torch.all(torch.isfinite(out[3:]))
    m = skg.rmsnorm(x.to(DEV), w.to(DEV), out_format="mx")
    assert _np(m.e8m0)[0].tolist() == [127, 127] and np.all(_np(m.y)[0] == 0)
    assert _np(m.e8m0)[1].tolist() == [255, 127] and _np(m.e8m0)[2].tolist() == [255, 255]
    z = skg.rmsnorm(x[:1].to(DEV), w.to(DEV), eps=0.0).y  # 0 / 0
    assert torch.all(torch.isnan(z))


def test_rmsnorm_feeds_the_fp8_products(skg):
    """The 8-bit outputs are operands of gemm_fp8: per tensor and MX."""
    M, K, N = 5, 512, 48
    x, w = _randn(1, M, K).bfloat16(), torch.ones(K, dtype=torch.bfloat16)
    wq, we = gen.quantise_mx(_randn(2, N, K))
    m = skg.rmsnorm(x.to(DEV), w.to(DEV), out_format="mx")
    out = skg.gemm_fp8(m.y, wq.to(DEV), xe=m.e8m0, we=we.to(DEV))
    want = ref.f64(skg.dequant_mx(m.y, m.e8m0)) @ ref.dequantise(gen.bits8(wq).astype(np.int64), we.numpy().astype(np.int64), "e4m3").T
    _product_close(out, want, K)
    s = torch.tensor([0.01], device=DEV)
    t = skg.rmsnorm(x.to(DEV), w.to(DEV), out_format="e4m3", scale=s)
    sw = torch.tensor([1.0], device=DEV)
    out = skg.gemm_fp8(t.y, wq.to(DEV), sx=s, sw=sw)
    want = ref.f64(t.y.float()) * float(np.float32(0.01)) @ ref.f64(wq.float()).T
    _product_close(out, want, K)


# ------------------------------------------------------------ routing

def _check_route(skg, l, k, dtype=torch.float32, bias=None, **o):
    ld = l.to(dtype)
    b = None if bias is None else bias.float()
    w, ids = skg.route(ld.to(DEV), k, bias=None if b is None else b.to(DEV), **o)
    w, ids = w.cpu().double().numpy(), ids.cpu().numpy().astype(np.int64)
    args = dict(scores="softmax", groups=1, top_groups=1, renormalize=True, factor=1.0)
    args.update(o)
    key, kept, best, _ = ref.route(ref.f64(ld), k, args["scores"], None if b is None else ref.f64(b), args["groups"],
                                   args["top_groups"], args["renormalize"], args["factor"])
    T, E = key.shape
    assert ids.min() >= 0 and ids.max() < E
    rows = np.arange(T)[:, None]
    assert all(len(set(r)) == k for r in ids.tolist())
    got, want = key[rows, ids], key[rows, best]
    same_groups = kept[rows, ids].all(-1)
    with np.errstate(invalid="ignore"):
        close = (got == want) | (np.abs(got - want) <= 2.0 ** -19 * (1 + np.abs(want)))
    if args["groups"] == 1:
        assert same_groups.all() and close.all()
    else:  # groups nearly equal may change places: exact scores decide which rows count
        assert (same_groups & close.all(-1)).mean() > 0.99
    # weights of the experts the kernel chose
    p = _scores(ref.f64(ld), args["scores"])[rows, ids]
    if args["renormalize"]:
        tot = p.sum(-1, keepdims=True)
        p = np.where(tot > 0, p / np.where(tot > 0, tot, 1), 0)
    p = p * np.float64(np.float32(args["factor"]))
    assert np.all(np.abs(w - p) <= 2.0 ** -18 * np.abs(p) + 2.0 ** -126)
    return w, ids


def _scores(l, scores):
    l = np.where(np.isnan(l), -np.inf, l)
    with np.errstate(invalid="ignore", over="ignore"):
        if scores == "sigmoid":
            return 1 / (1 + np.exp(-l))
        m = l.max(-1, keepdims=True)
        t = np.where(l == -np.inf, 0.0, np.where(l == m, 1.0, np.exp(l - m)))
        s = t.sum(-1, keepdims=True)
        return np.where(s > 0, t / np.where(s > 0, s, 1), 0.0)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 8), (5, 60, 4), (3, 64, 64), (7, 65, 1), (130, 384, 8),
                                   (2, 1024, 64), (9, 513, 10), (4, 129, 6), (16, 8, 8), (33, 1000, 8),
                                   (17, 136, 3), (2, 1023, 7), (2051, 72, 5)])
def test_route(skg, T, E, k, dtype, scores):
    l = 2 * _randn(T * E, T, E)
    for renorm in (True, False):
        _check_route(skg, l, k, dtype, scores=scores, renormalize=renorm, factor=1.0 if renorm else 2.5)
    _check_route(skg, l, k, dtype, scores=scores, bias=0.1 * _randn(E, E))


@pytest.mark.parametrize("scores,bias", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
@pytest.mark.parametrize("E,groups,top,k", [(256, 8, 4, 8), (60, 4, 2, 6), (64, 64, 8, 8), (48, 16, 16, 5),
                                            (1024, 2, 1, 20), (96, 3, 1, 32), (160, 8, 3, 6), (1000, 40, 7, 64),
                                            (128, 16, 5, 8), (512, 64, 9, 8), (1024, 2, 1, 8), (384, 16, 16, 1)])
def test_route_groups(skg, E, groups, top, k, scores, bias):
    for T in (200, 2100):
        _check_route(skg, 2 * _randn(E + k + T, T, E), k, scores=scores, groups=groups, top_groups=top,
                     bias=0.1 * _randn(E, E) if bias else None)


def test_route_logits_off_16_bytes(skg):
    for dtype in (torch.float32, torch.bfloat16):
        l = (2 * _randn(4, 5 * 64 + 1)).to(dtype).to(DEV)
        for o in (dict(), dict(groups=4, top_groups=2, scores="sigmoid"), dict(renormalize=False)):
            off = skg.route(l[1:].reshape(5, 64), 6, **o)
            on = skg.route(l[1:].clone().reshape(5, 64), 6, **o)
            assert torch.equal(off[1], on[1])
            assert torch.allclose(off[0], on[0], rtol=2.0 ** -18, atol=0)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("k", [5, 9])
def test_route_ties_go_to_the_lowest_index(skg, scores, k):
    T, E = 50, 200
    l = torch.randint(0, 3, (T, E), generator=torch.Generator().manual_seed(5)).float()
    _, ids = skg.route(l.to(DEV), k, scores=scores)
    want = torch.sort(l, dim=-1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(ids.cpu().long(), want)
    # all equal: experts 0..k-1; equal groups: the first ones; -0 equals 0
    z = torch.zeros(2, 64)
    z[1, ::2] = -0.0
    _, ids = skg.route(z.to(DEV), 5, scores=scores)
    assert ids.cpu().tolist() == [[0, 1, 2, 3, 4]] * 2
    _, ids = skg.route(z.to(DEV), k, scores=scores, groups=8, top_groups=2)
    assert ids.cpu().tolist() == [list(range(k))] * 2


def test_route_masked_and_non_finite_logits(skg):
    inf = math.inf
    l = torch.tensor([[-inf] * 6,                        # nothing left
                      [-inf, 1.0, -inf, 2.0, -inf, -inf],  # fewer than k left
                      [math.nan, 0.0, 1.0, math.nan, -1.0, -2.0],
                      [inf, 0.0, inf, 1.0, 2.0, 3.0],
                      [-3.3895313892515355e38] * 6,       # the type's lowest value
                      [3e38, -3e38, 0.0, 0.0, 0.0, 0.0]])
    w, ids = skg.route(l.to(DEV), 3)
    w, ids = w.cpu(), ids.cpu()
    assert ids.tolist() == [[0, 1, 2], [3, 1, 0], [2, 1, 4], [0, 2, 5], [0, 1, 2], [0, 2, 3]]
    assert w[0].tolist() == [0, 0, 0]
    assert w[1, 2] == 0 and abs(w[1, :2].sum() - 1) < 1e-6
    assert torch.all(torch.isfinite(w))
    assert w[3].tolist() == [0.5, 0.5, 0.0]
    assert torch.allclose(w[4], torch.full((3,), 1 / 3))
    assert w[5].tolist() == [1, 0, 0]
    for renorm in (True, False):
        w, ids = skg.route(l.to(DEV), 3, scores="sigmoid", renormalize=renorm)
        assert torch.all(torch.isfinite(w))
        assert w[0].tolist() == [0, 0, 0] and ids[0].tolist() == [0, 1, 2]
        assert ids.cpu()[2].tolist() == [2, 1, 4]
        w, _ = skg.route(l.to(DEV), 3, renormalize=renorm)
        assert torch.all(torch.isfinite(w)) and w[0].tolist() == [0, 0, 0]
    # a masked expert of a kept group goes before any expert of a dropped one
    g = torch.tensor([[5.0, -inf, 1.0, 1.0]])
    _, ids = skg.route(g.to(DEV), 2, groups=2, top_groups=1)
    assert ids.tolist() == [[0, 1]]


def test_route_refuses(skg):
    l = torch.zeros(2, 16, device=DEV)
    for bad in (dict(k=17), dict(k=0), dict(k=2, groups=3), dict(k=9, groups=4, top_groups=2)):
        with pytest.raises(skg.SkinnyGemmError):
            skg.route(l, **bad)
    for bad in (dict(k=2, scores="tanh"), dict(k=2, bias=torch.zeros(15, device=DEV))):
        with pytest.raises(ValueError):
            skg.route(l, **bad)
    with pytest.raises(ValueError):
        skg.route(l.t(), 2)
    w, ids = skg.route(l[:0], 3)
    assert w.shape == ids.shape == (0, 3)


# ------------------------------------------------------------ product

def _product_close(out, want, K):
    got = ref.f64(out)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    fine = np.isfinite(want)
    rms = math.sqrt(np.mean(want[fine] ** 2)) if fine.any() else 0.0
    err = np.abs(got[fine] - want[fine])
    bound = 2.0 ** -7 * np.abs(want[fine]) + 1e-3 * math.sqrt(K) * rms
    assert np.all(err <= bound), f"worst {np.max(err - bound)}"


def _weight(seed, N, K, E=None):
    """(codes bytes, e8m0, values) of N(0, 1/K) weights."""
    shape = (N, K) if E is None else (E, N, K)
    v = _randn(seed, *shape).double().numpy() / math.sqrt(K)
    c, e = ref.quantise(v, "e2m1")
    return (torch.from_numpy(ref.pack_bytes(c, "e2m1")), torch.from_numpy(e.astype(np.uint8)),
            ref.dequantise(c, e, "e2m1"))


GEMM_SIZES = [(1, 1, 32), (1, 16, 128), (2, 15, 64), (3, 17, 96), (15, 33, 160), (16, 64, 512), (17, 100, 544),
              (1, 2112, 7168), (5, 576, 7168), (16, 1111, 2880), (32, 48, 1024), (33, 128, 2880), (64, 65, 320),
              (65, 256, 2016), (128, 130, 640), (129, 96, 1024), (200, 31, 5984), (512, 272, 288), (512, 16, 32),
              # every tile of the products above 32 rows, and K past the 8192 whose scales a tile holds at once
              (21, 40, 352), (40, 33, 8480), (512, 600, 96), (500, 1100, 160), (512, 2100, 544), (490, 2180, 8736),
              # few rows: several rounds of loads, and rows too long for them
              (2, 33, 30016), (16, 40, 6368), (20, 24, 4640), (30, 50, 4320), (16, 40, 9248), (31, 20, 9248),
              (512, 400, 8480)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", GEMM_SIZES)
def test_gemm_mxfp4(skg, M, N, K, fmt):
    x = _randn(M + N, M, K).bfloat16()
    q, e, w = _weight(K, N, K)
    b = (0.3 * _randn(1, N)).bfloat16()
    h = skg.mxfp4_pack(q.to(DEV), e.to(DEV))
    want = ref.rounded(ref.f64(x), fmt) @ w.T
    out = skg.gemm_mxfp4(x.to(DEV), h, x_format=fmt)
    _product_close(out, want, K)
    _product_close(skg.gemm_mxfp4(x.to(DEV), h, x_format=fmt, bias=b.to(DEV)), want + ref.f64(b), K)
    f32 = skg.gemm_mxfp4(x.to(DEV), h, x_format=fmt, out_dtype=torch.float32)
    assert torch.equal(f32.bfloat16(), out)  # one rounding
    xq, xe = skg.quant_mx(x.to(DEV), fmt)
    codes = skg.gemm_mxfp4(xq, h, xe=xe, x_format=fmt)
    if M > 16:  # may take another kernel, with another order of its sums
        _product_close(codes, want, K)
    else:
        assert torch.equal(codes, out)  # codes or bf16: the same bits
    assert torch.equal(skg.gemm_mxfp4(x.to(DEV), h, x_format=fmt), out)  # the same bits again


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [(1, 40, 96), (4, 1, 32), (16, 100, 2880), (37, 33, 544), (130, 80, 1056)])
def test_gemm_mxfp4_small_integers_exact(skg, M, N, K, fmt):
    """Integers that both formats hold: every product and sum is exact in fp32."""
    g = torch.Generator().manual_seed(M * N)
    x = torch.randint(-2, 3, (M, K), generator=g).double()
    x[:, ::32] = 6.0  # so that every block's scale is one
    w = torch.randint(-3, 4, (N, K), generator=g).double()
    w[:, ::32] = 6.0
    x[:, ::32] *= 448 / 6 if fmt == "e4m3" else 1
    c, e = ref.quantise(w.numpy(), "e2m1")
    h = skg.mxfp4_pack(torch.from_numpy(ref.pack_bytes(c, "e2m1")).to(DEV), torch.from_numpy(e.astype(np.uint8)).to(DEV))
    b = torch.randint(-4, 5, (N,), generator=g).double()
    out = skg.gemm_mxfp4(x.bfloat16().to(DEV), h, x_format=fmt, bias=b.bfloat16().to(DEV), out_dtype=torch.float32)
    assert np.array_equal(ref.f64(out), (x @ w.T + b).numpy())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,K", [(3, 96), (18, 544), (70, 288)])
def test_gemm_mxfp4_nan_stays_in_its_row(skg, M, K, fmt):
    """A NaN or infinity in one row of x, a NaN scale in one row of W: that
    row or column is NaN and no other value changes (K ends inside a step, so
    the next row's values lie right after this one's)."""
    N = 35
    x = _randn(1, M, K).bfloat16()
    q, e, _ = _weight(2, N, K)
    clean = skg.gemm_mxfp4(x.to(DEV), skg.mxfp4_pack(q.to(DEV), e.to(DEV)), x_format=fmt).cpu()
    x2, e2 = x.clone(), e.clone()
    x2[1, 0] = math.nan
    x2[2, K - 1] = math.inf
    e2[20, 0] = 255
    out = skg.gemm_mxfp4(x2.to(DEV), skg.mxfp4_pack(q.to(DEV), e2.to(DEV)), x_format=fmt).cpu()
    bad = torch.zeros(M, N, dtype=torch.bool)
    bad[1:3] = True
    bad[:, 20] = True
    assert torch.equal(torch.isnan(out), bad)
    assert torch.equal(out[~bad], clean[~bad])


@pytest.mark.parametrize("fmt", FORMATS)
def test_gemm_mxfp4_wide_scales(skg, fmt):
    """Scales far from one: exact powers of two pass through the product."""
    M, N, K = 4, 20, 160
    x = _randn(3, M, K).bfloat16()
    q, e, w = _weight(4, N, K)
    h = skg.mxfp4_pack(q.to(DEV), e.to(DEV))
    base = skg.gemm_mxfp4(x.to(DEV), h, x_format=fmt, out_dtype=torch.float32)
    for p in (-60, -20, 20, 60):
        hp = skg.mxfp4_pack(q.to(DEV), (e.int() - p).to(torch.uint8).to(DEV))
        xp = (x.double() * 2.0 ** p).bfloat16()
        assert torch.equal(skg.gemm_mxfp4(xp.to(DEV), hp, x_format=fmt, out_dtype=torch.float32), base)


def test_gemm_mxfp4_refuses(skg):
    q, e, _ = _weight(1, 16, 64)
    h = skg.mxfp4_pack(q.to(DEV), e.to(DEV))
    x = torch.zeros(2, 64, dtype=torch.bfloat16, device=DEV)
    for bad in (lambda: skg.gemm_mxfp4(x[:, :32].contiguous(), h), lambda: skg.gemm_mxfp4(x.t(), h),
                lambda: skg.gemm_mxfp4(x, h, bias=torch.zeros(15, dtype=torch.bfloat16, device=DEV)),
                lambda: skg.gemm_mxfp4(x, h, x_format="e5m2"),
                lambda: skg.moe_mxfp4(x, torch.zeros(3, 1, dtype=torch.int32, device=DEV), x, h, h)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: skg.gemm_mxfp4(x.float(), h), lambda: skg.gemm_mxfp4(x, h.packed),
                lambda: skg.gemm_mxfp4(x, h, out_dtype=torch.float16)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(skg.SkinnyGemmError):
        skg.gemm_mxfp4(torch.zeros(513, 64, dtype=torch.bfloat16, device=DEV), h)
    assert skg.gemm_mxfp4(x[:0], h).shape == (0, 16)


# ------------------------------------------------------------ experts

class Experts:
    """Random codes and scales, their values about N(0, 1/K) in size."""

    def __init__(self, skg, E, H, I, seed=0):
        self.w13, self.v13 = self._make(skg, seed + 1, E, 2 * I, H)
        self.w2, self.v2 = self._make(skg, seed + 2, E, H, I)

    @staticmethod
    def _make(skg, seed, E, N, K):
        g = torch.Generator().manual_seed(seed)
        c = torch.randint(0, 16, (E, N, K), generator=g, dtype=torch.uint8).numpy()
        mid = 127 - round(math.log2(2.9 * math.sqrt(K)))
        e = torch.randint(mid - 1, mid + 2, (E, N, K // 32), generator=g, dtype=torch.uint8).numpy()
        packed = skg.mxfp4_pack(torch.from_numpy(ref.pack_bytes(c, "e2m1")).to(DEV), torch.from_numpy(e).to(DEV))
        return packed, ref.dequantise(c.astype(np.int64), e.astype(np.int64), "e2m1")


def _choices(seed, T, k, E):
    g = torch.Generator().manual_seed(seed)
    ids = torch.rand(T, E, generator=g).argsort(-1)[:, :k].int()
    w = torch.rand(T, k, generator=g) + 0.1
    return ids, w / w.sum(-1, keepdim=True)


def _check_experts(skg, m, x, ids, w, fmt):
    out = skg.moe_mxfp4(x.to(DEV), ids.to(DEV), w.to(DEV), m.w13, m.w2, x_format=fmt)
    either = []
    want = ref.experts(ref.f64(x), ids.numpy(), ref.f64(w), m.v13, m.v2, fmt, either)
    got = ref.f64(out)
    for t, change in either:  # where the sums' last bits decide: whichever was taken
        if np.linalg.norm(got[t] - want[t] - change) < np.linalg.norm(got[t] - want[t]):
            want[t] += change
    rms = math.sqrt(np.mean(want ** 2)) if want.size else 0.0
    assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 0.05 * rms)
    # most values are far closer than the worst allowed
    if rms:
        assert np.linalg.norm(got - want) <= 0.01 * np.linalg.norm(want)
    again = skg.moe_mxfp4(x.to(DEV), ids.to(DEV), w.to(DEV), m.w13, m.w2, x_format=fmt)
    assert torch.equal(again, out)  # no order of arrival in the bits
    return out


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,k,E,H,I", [(1, 1, 1, 32, 32), (1, 4, 8, 96, 160), (2, 2, 3, 160, 96), (3, 8, 8, 544, 32),
                                       (17, 4, 16, 256, 288), (40, 1, 5, 128, 64), (200, 3, 7, 96, 96),
                                       (1, 4, 6, 2880, 1440), (9, 2, 130, 64, 64), (70, 64, 64, 64, 32),
                                       # enough bytes to be sorted: tiles of 16, 32 and 64 rows
                                       (64, 4, 64, 448, 448), (200, 4, 40, 288, 224), (300, 4, 8, 160, 224),
                                       (600, 8, 12, 96, 96), (500, 64, 64, 64, 32), (80, 2, 2, 8480, 64),
                                       # enough of them for tiles of 96 rows, one or more to an expert
                                       (2500, 2, 100, 32, 1024), (896, 8, 32, 32, 1024),
                                       # unsorted, rows of several rounds of loads
                                       (1, 8, 8, 96, 4128), (1, 2, 2, 8480, 64)])
def test_experts(skg, T, k, E, H, I, fmt):
    m = Experts(skg, E, H, I)
    ids, w = _choices(T, T, k, E)
    _check_experts(skg, m, _randn(T + H, T, H).bfloat16(), ids, w, fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 5, 64, 2000])
def test_experts_skewed_and_absent(skg, T, fmt):
    """Every token on one expert; the same expert twice in a token; ids
    outside [0, E) skipped; a token, then every token, with none left."""
    E, k, H, I = 6, 4, 96, 64
    m = Experts(skg, E, H, I)
    x = _randn(T, T, H).bfloat16()
    _, w = _choices(1, T, k, E)
    ids = torch.full((T, k), 3, dtype=torch.int32)
    _check_experts(skg, m, x, ids, w, fmt)
    ids, w = _choices(2, T, k, E)
    ids[:, 1] = -1
    ids[::2, 3] = E
    ids[0] = torch.tensor([-5, E, E + 100, -2147483648], dtype=torch.int32)
    out = _check_experts(skg, m, x, ids, w, fmt)
    assert torch.all(out[0] == 0)
    out = skg.moe_mxfp4(x.to(DEV), torch.full_like(ids, -1).to(DEV), w.to(DEV), m.w13, m.w2, x_format=fmt)
    assert torch.all(out == 0)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,E,H,I", [(1, 6, 96, 64), (5, 6, 96, 64), (2000, 6, 96, 64), (72, 72, 480, 480)])
def test_experts_weights_of_absent_choices_do_not_count(skg, T, E, H, I, fmt):
    """The weight of a choice whose id lies outside [0, E) may be anything: with
    NaN and infinities there, the same bits as with zeros, in calls that each
    pair takes for itself and in sorted ones; zeros where a token has none left."""
    k = 4
    m = Experts(skg, E, H, I)
    x = _randn(T, T, H).bfloat16()
    ids, w = _choices(3, T, k, E)
    ids[:, 1] = -1
    ids[::2, 3] = E
    ids[0] = -1
    away = (ids < 0) | (ids >= E)
    zeros = skg.moe_mxfp4(x.to(DEV), ids.to(DEV), torch.where(away, 0.0, w).to(DEV), m.w13, m.w2, x_format=fmt)
    for bad in (math.nan, math.inf, -math.inf):
        got = skg.moe_mxfp4(x.to(DEV), ids.to(DEV), torch.where(away, bad, w).to(DEV), m.w13, m.w2, x_format=fmt)
        assert torch.isfinite(got).all() and torch.equal(got, zeros)
        assert torch.all(got[0] == 0)


@pytest.mark.parametrize("T", [3, 90, 3000])
def test_experts_row_does_not_depend_on_its_neighbours(skg, T):
    """Other tokens' values and choices (their number the same): the same bits,
    whatever the others hold, NaN too."""
    E, k, H, I = 5, 2, 160, 96
    m = Experts(skg, E, H, I)
    x = _randn(9, T, H).bfloat16()
    ids, w = _choices(9, T, k, E)
    keep = torch.arange(T) % 3 == 0
    one = skg.moe_mxfp4(x.to(DEV), ids.to(DEV), w.to(DEV), m.w13, m.w2).cpu()
    x2, (ids2, w2) = _randn(10, T, H).bfloat16(), _choices(11, T, k, E)
    x2[keep], ids2[keep], w2[keep] = x[keep], ids[keep], w[keep]
    x2[1] = math.nan
    two = skg.moe_mxfp4(x2.to(DEV), ids2.to(DEV), w2.to(DEV), m.w13, m.w2).cpu()
    assert torch.equal(one[keep], two[keep])
    assert torch.isnan(two[1]).all() and torch.isfinite(two[torch.arange(T) != 1]).all()


# ------------------------------------------------------------ streams, graphs, the whole layer

def _layer(skg, x, r, g, wr, m):
    n = skg.rmsnorm(x, g, residual=r)
    w, ids = skg.route(skg.gemm_bf16_f32(n.y, wr), 4)
    return skg.moe_mxfp4(n.y, ids, w, m.w13, m.w2), n.residual


def test_layer_in_a_graph_and_on_another_stream(skg):
    E, H, I, T = 8, 256, 96, 6
    m = Experts(skg, E, H, I)
    x, r = _randn(1, T, H).bfloat16().to(DEV), _randn(2, T, H).bfloat16().to(DEV)
    g, wr = torch.ones(H, dtype=torch.bfloat16, device=DEV), (_randn(3, E, H) / 16).bfloat16().to(DEV)
    want = [t.clone() for t in _layer(skg, x, r, g, wr, m)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _layer(skg, x, r, g, wr, m)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # captured: workspace reserved before, every replay checked after new inputs
    cap = torch.cuda.Stream()
    skg.reserve(16, 64, 0, 64, stream=cap)
    skg.reserve_moe(max_T=T, k=4, H=H, I=I, E=E, stream=cap)
    graph = torch.cuda.CUDAGraph()
    cap.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(cap):
        with torch.cuda.graph(graph, stream=cap):
            out = _layer(skg, x, r, g, wr, m)
    for i in range(4):
        x.copy_(_randn(10 + i, T, H).bfloat16())
        want = [t.clone() for t in _layer(skg, x, r, g, wr, m)]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i


def test_example_block(skg, monkeypatch):
    """examples/moe_layer.py: the projection and the residual, then the experts
    on the block's own normed rows and choices, against 64 bits; and its graph
    against its steps."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_layer.py")
    spec = importlib.util.spec_from_file_location("moe_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    made, pack = [], skg.mxfp4_pack

    def record(q, e):
        made.append(ref.dequantise(ref.unpack_bytes(_np(q), "e2m1"), _np(e).astype(np.int64), "e2m1"))
        return pack(q, e)

    monkeypatch.setattr(skg, "mxfp4_pack", record)
    torch.manual_seed(3)
    T, H = 11, 320
    block = mod.MoeBlock(H, 96, 8, 2)
    wo, v13, v2 = made
    a, r = _randn(1, T, H).bfloat16(), _randn(2, T, H).bfloat16()
    out, residual = block.forward(a.to(DEV), r.to(DEV))
    xq = ref.rounded(ref.f64(a), "e4m3")
    o = xq @ wo.T
    s = o + ref.f64(r)
    # bf16 of the product, fp32 sums with products cut 2^-13 below their group's largest, bf16 of the sum
    bound = 2.0 ** -8 * (np.abs(o) + 1.01 * np.abs(s)) + 2.0 ** -12 * (np.abs(xq) @ np.abs(wo).T)
    assert np.all(np.abs(ref.f64(residual) - s) <= bound)
    n = skg.rmsnorm(skg.gemm_mxfp4(a.to(DEV), block.wo), block.gain, residual=r.to(DEV))
    assert torch.equal(n.residual, residual)
    w, ids = skg.route(skg.gemm_bf16_f32(n.y, block.router), 2)
    want = ref.experts(ref.f64(n.y), ids.cpu().numpy(), ref.f64(w), v13, v2, "e4m3")
    assert np.linalg.norm(ref.f64(out) - want) <= 0.01 * np.linalg.norm(want)
    ad, rd = a.to(DEV), r.to(DEV)
    graph, again = block.capture(ad, rd)
    for i in range(4):
        ad.copy_(_randn(20 + i, T, H).bfloat16())
        step = block.forward(ad, rd)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(step, again)), i


def test_capture_needs_reserved_workspace(skg):
    q, e, _ = _weight(1, 4096, 64)
    h = skg.mxfp4_pack(q.to(DEV), e.to(DEV))
    x = torch.zeros(512, 64, dtype=torch.bfloat16, device=DEV)  # rows that are quantised first
    out = torch.empty(512, 4096, dtype=torch.bfloat16, device=DEV)
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            with pytest.raises(skg.SkinnyGemmError) as err:
                skg.gemm_mxfp4(x, h, out=out)
    assert err.value.status == skg.ERR_WORKSPACE
