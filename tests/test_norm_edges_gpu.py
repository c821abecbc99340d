"""rmsnorm where fp32 ends and next to ties, against 64 bits.

Derived:
- A value is fp32's where the formula's value is: finite ones within 2^-16 (the
  norm's own bound, see tests/test_moe_gpu.py) and half a step of the output's
  type, infinite ones infinite (e4m3: clamped to +-448), 0 / 0 NaN.
- Near a tie between two codes: with integer rows the sum of squares is exact,
  and the factor, two fp32 numbers, is within 2^-44 of its value; so is a value
  before its one rounding.  The code is that of the exact value wherever that
  lies 2^-40 of itself or more from a tie.
"""
import math

import numpy as np
import pytest
import torch

from tests import mx_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
# a wave a row; a workgroup; two vectors a lane; rows that are read twice
LENGTHS = [64, 1024, 8224, 16416]


@pytest.fixture(scope="module")
def skg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import latency_skinny_gemm_amd as m
    m.lib()
    return m


def _randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def _codes(t):
    return t.cpu().view(torch.uint8).numpy().astype(np.int64)


def _e4m3(codes):
    """Values of e4m3 codes."""
    return np.where(codes >= 128, -1.0, 1.0) * ref.E4M3_VALUES[codes % 128]


def _norm64(x, w, eps):
    return ref.norm(x, None, w, eps)[1]


# ------------------------------------------------------------ past fp32's range

@pytest.mark.parametrize("K", LENGTHS)
@pytest.mark.parametrize("scale", [0.0, 1e-45, 1e-39, 1e-37, 1e-30, -1e-39, 1e30, 3e38, math.inf, math.nan])
def test_e4m3_with_a_scale_at_the_end_of_the_range(skg, K, scale):
    x, w = _randn(K, 3, K).bfloat16(), (1 + 0.3 * _randn(K + 1, K)).bfloat16()
    x[:, 7] = 0
    s = torch.tensor([scale])
    out = skg.rmsnorm(x.to(DEV), w.to(DEV), out_format="e4m3", scale=s.to(DEV))
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        want = np.clip(_norm64(x, w, 1e-6) / float(s[0].double()), -448, 448)
    got = _e4m3(_codes(out.y))
    assert np.array_equal(np.isnan(got), np.isnan(want))
    fine = ~np.isnan(want)
    # 448, -448 or (as codes) 0, all of them
    assert np.array_equal(got[fine], _e4m3(ref._nearest(want[fine], ref.E4M3_VALUES[:-1])))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "mx"])
@pytest.mark.parametrize("K", LENGTHS)
def test_infinite_weights_and_products(skg, K, fmt):
    x, w = _randn(K, 3, K).bfloat16(), (1 + 0.3 * _randn(K + 1, K)).bfloat16()
    x[2, 3] = 0
    w2 = w.clone()
    w2[3], w2[5], w2[38] = math.inf, -math.inf, 3e38
    x[:, 38] = 4.0  # times 3e38: past the range
    clean = skg.rmsnorm(x.to(DEV), w.to(DEV), out_format=fmt,
                        scale=torch.tensor([0.01], device=DEV) if fmt == "e4m3" else None)
    out = skg.rmsnorm(x.to(DEV), w2.to(DEV), out_format=fmt,
                      scale=torch.tensor([0.01], device=DEV) if fmt == "e4m3" else None)
    sign = np.sign(ref.f64(x))
    want = {3: sign[:, 3], 5: -sign[:, 5], 38: sign[:, 38]}
    if fmt == "mx":
        e = _codes(out.e8m0)
        assert np.all(e[:, :2] == 255)
        assert np.array_equal(_codes(out.y)[:, 64:], _codes(clean.y)[:, 64:])
        return
    got = ref.f64(out.y) if fmt == "bf16" else _e4m3(_codes(out.y))
    same = ref.f64(clean.y) if fmt == "bf16" else _e4m3(_codes(clean.y))
    for i, s in want.items():
        top = math.inf if fmt == "bf16" else 448.0
        assert np.array_equal(got[s != 0, i], s[s != 0] * top)
        assert np.all(np.isnan(got[s == 0, i]))
    others = np.setdiff1d(np.arange(K), list(want))
    assert np.array_equal(got[:, others], same[:, others])


def test_e4m3_zero_infinite_and_nan_rows_and_lengths_off_the_block(skg):
    """Static codes take any multiple of 8; a NaN stays in its row, an infinity
    makes the others 0."""
    s = torch.tensor([0.01], device=DEV)
    for K in (8, 24, 1016, 1032, 8200, 16392):
        x, w = _randn(K, 5, K).bfloat16(), (1 + 0.3 * _randn(K + 1, K)).bfloat16()
        x[0], x[1, 5], x[2, 3] = 0, -math.inf, math.nan
        got = _e4m3(_codes(skg.rmsnorm(x.to(DEV), w.to(DEV), out_format="e4m3", scale=s).y))
        assert np.all(got[0] == 0) and np.isnan(got[2]).all()
        assert np.isnan(got[1, 5]) and np.all(np.delete(got[1], 5) == 0)
        t = np.clip(_norm64(x[3:], w, 1e-6) / float(np.float32(0.01)), -448, 448)
        step = np.exp2(np.floor(np.log2(np.maximum(np.abs(t), 2.0 ** -6))) - 3)
        assert np.all(np.abs(got[3:] - t) <= step / 2 + 2.0 ** -15 * np.abs(t))


# ------------------------------------------------------------ next to ties

def _integers(seed, K):
    g = np.random.default_rng(seed)
    x = g.integers(-200, 201, K).astype(np.float64)
    x[x == 0] = 1.0
    w = torch.from_numpy(1 + 0.3 * g.standard_normal(K)).bfloat16()
    return x, w, int(g.integers(0, K)), g.uniform(0.2, 1.0)


def _one_number(x, w, m, scale=None):
    """The chain with the factor in one fp32 number and every step rounded."""
    f = np.float32
    c = f(1 / np.sqrt(m))
    if scale is not None:
        c = f(c * f(1 / f(scale)))
    return (f(x) * c) * ref.f64(w).astype(f)


def _away(q):
    """Distance of |q| from the nearest tie between e4m3 values, over |q|."""
    mids = (ref.E4M3_VALUES[1:127] + ref.E4M3_VALUES[:126]) / 2
    a = np.abs(q)
    k = np.clip(np.searchsorted(mids, a), 1, len(mids) - 1)
    return np.minimum(np.abs(a - mids[k]), np.abs(a - mids[k - 1])) / np.maximum(a, 2.0 ** -10)


@pytest.mark.parametrize("K", [64, 512])
def test_e4m3_codes_next_to_ties(skg, K):
    """The scale puts one value of each row next to a tie."""
    table, other = ref.E4M3_VALUES[:-1], 0
    for seed in range(48):
        x, w, j, u = _integers(seed, K)
        m = (x * x).sum() / K + float(np.float32(1e-5))
        y = x / np.sqrt(m) * ref.f64(w)
        lo = int(np.searchsorted(table, 240.0 * u))
        scale = np.float32(abs(y[j]) / ((table[lo] + table[lo + 1]) / 2))
        q = np.clip(y / np.float64(scale), -448, 448)
        want = ref._nearest(q, table)
        one = ref._nearest(np.clip(_one_number(x, w, m, scale).astype(np.float64), -448, 448), table)
        sure = _away(q) > 2.0 ** -40
        other += int((one != want)[sure].sum())
        out = skg.rmsnorm(torch.from_numpy(x)[None].bfloat16().to(DEV), w.to(DEV), eps=1e-5, out_format="e4m3",
                          scale=torch.tensor([scale], device=DEV))
        got = _codes(out.y)[0]
        assert np.array_equal(got[sure], want[sure]), seed
    assert other >= 5  # one fp32 number does not do


@pytest.mark.parametrize("K", [64, 512])
def test_mx_codes_next_to_ties(skg, K):
    """eps puts one value of each row next to a tie."""
    table, other = ref.E4M3_VALUES[:-1], 0
    mids = (table[1:] + table[:-1]) / 2
    for seed in range(48):
        x, w, j, _ = _integers(100 + seed, K)
        wf = ref.f64(w)
        y0 = x / np.sqrt((x * x).sum() / K) * wf
        f = 2.0 ** (int(ref.quantise(y0[None], "e4m3")[1][0, j // 32]) - 127)
        t = mids[max(int(np.searchsorted(mids, abs(y0[j]) / f)) - 1, 0)] * f
        eps = np.float32(max((x[j] * wf[j] / t) ** 2 - (x * x).sum() / K, 0.0))
        m = (x * x).sum() / K + np.float64(eps)
        y = x / np.sqrt(m) * wf
        want, e = ref.quantise(y[None], "e4m3")
        one = ref.quantise(_one_number(x, w, m).astype(np.float64)[None], "e4m3")[0]
        sure = _away(np.ldexp(y, 127 - np.repeat(e[0], 32))) > 2.0 ** -40
        other += int((one != want)[0, sure].sum())
        out = skg.rmsnorm(torch.from_numpy(x)[None].bfloat16().to(DEV), w.to(DEV), eps=float(eps), out_format="mx")
        assert np.array_equal(_codes(out.e8m0), e), seed
        assert np.array_equal(_codes(out.y)[0, sure], want[0, sure]), seed
    assert other >= 5


# ------------------------------------------------------------ squares past fp32's range

@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "mx"])
@pytest.mark.parametrize("K", LENGTHS)
@pytest.mark.parametrize("residual", [False, True])
def test_rows_whose_squares_leave_fp32(skg, K, residual, fmt):
    """eps 0: rows down to bf16's subnormals and up to its largest values have
    the norm of their shape, whatever their size."""
    powers = [-131, -126, -110, -70, -63, -50, -34, 0, 59, 61, 63, 64, 90, 125]
    size = torch.exp2(torch.tensor(powers, dtype=torch.float64))[:, None]
    x = (_randn(K, len(powers), K).clamp(-3, 3).double() * size).bfloat16()
    r = (0.5 * _randn(K + 2, len(powers), K).clamp(-1, 1).double() * size).bfloat16() if residual else None
    w = (1 + 0.3 * _randn(K + 1, K)).bfloat16()
    scale = torch.tensor([0.0123], device=DEV) if fmt == "e4m3" else None
    out = skg.rmsnorm(x.to(DEV), w.to(DEV), residual=None if r is None else r.to(DEV), eps=0.0, out_format=fmt, scale=scale)
    y = ref.norm(x, r, w, 0.0)[1]
    if residual:
        assert torch.equal(out.residual.cpu(), (x.float() + r.float()).bfloat16())
    if fmt == "mx":
        e = _codes(out.e8m0)
        want_e = ref.quantise(y, "e4m3")[1]
        near = np.abs(np.log2(np.abs(y).reshape(*want_e.shape, 32).max(-1) / 448.0) % 1.0 - 0.5) > 0.5 - 2.0 ** -14
        assert np.all((e == want_e) | (near & (np.abs(e - want_e) <= 1)))
        f = np.exp2(np.repeat(e, 32, -1) - 127.0)
        got, t = _e4m3(_codes(out.y)), y / f
    elif fmt == "e4m3":
        got, t = _e4m3(_codes(out.y)), np.clip(y / float(np.float32(0.0123)), -448, 448)
    else:
        step = np.exp2(np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -126))) - 7)
        assert np.all(np.abs(ref.f64(out.y) - y) <= step / 2 + 2.0 ** -16 * np.abs(y))
        return
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(t), 2.0 ** -6))) - 3)
    assert np.all(np.abs(got - t) <= step / 2 + 2.0 ** -15 * np.abs(t))


def test_a_row_of_zeros_and_one_infinite_stay_as_the_formula_has_them(skg):
    for K in LENGTHS:
        x = torch.zeros(3, K, dtype=torch.bfloat16)
        x[1, 5], x[2, 6] = math.inf, math.nan
        y = skg.rmsnorm(x.to(DEV), torch.ones(K, dtype=torch.bfloat16, device=DEV), eps=0.0).y.cpu()
        assert torch.isnan(y[0]).all() and torch.isnan(y[1, 5]) and torch.isnan(y[2]).all()
        assert torch.all(y[1, :5] == 0) and torch.all(y[1, 6:] == 0)


# ------------------------------------------------------------ more rows than one grid holds

@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "mx"])
def test_more_rows_than_a_grid_holds(skg, fmt):
    """2^26 rows of a wave each are 2^32 work-items: the same 2^20 rows over and
    over, with the same result over and over."""
    K, times = 32, 64
    x, w = _randn(1, 1 << 20, K).bfloat16().to(DEV), (1 + 0.3 * _randn(2, K)).bfloat16().to(DEV)
    r = (2 * _randn(3, 1 << 20, K)).bfloat16().to(DEV)
    o = dict(out_format=fmt, scale=torch.tensor([0.01], device=DEV) if fmt == "e4m3" else None)
    one = skg.rmsnorm(x, w, residual=r, **o)
    many = skg.rmsnorm(torch.cat([x.repeat(times, 1), x[:3]]), w, residual=torch.cat([r.repeat(times, 1), r[:3]]), **o)
    for a, b in zip(many, one):
        if b is None:
            assert a is None
            continue
        a, b = a.view(torch.uint8), b.view(torch.uint8)
        assert torch.equal(a[-3:], b[:3])
        for i in range(times):
            assert torch.equal(a[i << 20:(i + 1) << 20], b), i
