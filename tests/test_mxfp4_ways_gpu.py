"""Every way of the MXFP4 products and of the experts (mxfp4_sizes.py): exact sums,
and NaN and infinities that stay in their rows and columns.

The inputs are those of test_mxfp4_sums_gpu.py: every product is a multiple of 2^-10
(e2m1: 2^-2) and the sum of their magnitudes below 2^14 (2^22), so that any order
of adding them up in fp32 is exact, with an integer bias too."""
import math

import numpy as np
import pytest
import torch

from tests import mxfp4_sizes as sizes
from tests.test_mxfp4_sums_gpu import _rows, _weights

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


def _made(skg, M, N, K, fmt):
    g = np.random.default_rng(M + N + K)
    x = _rows(g, M, K, fmt)
    h, w = _weights(skg, g, (N, K))
    return x, h, w


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", sizes.PRODUCTS)
def test_exact(skg, M, N, K, fmt):
    x, h, w = _made(skg, M, N, K, fmt)
    xd, wd = torch.from_numpy(x).to(DEV), torch.from_numpy(w).to(DEV).t().contiguous()
    bias = torch.from_numpy(np.random.default_rng(N).integers(-64, 65, N)).bfloat16().to(DEV)
    assert (xd.abs() @ wd.abs()).max() + 64 < (2.0 ** 14 if fmt == "e4m3" else 2.0 ** 22)
    want = (xd @ wd + bias.double()).float()
    xb = xd.bfloat16()
    out = skg.gemm_mxfp4(xb, h, x_format=fmt, bias=bias, out_dtype=torch.float32)
    assert torch.equal(out, want)
    assert torch.equal(skg.gemm_mxfp4(xb, h, x_format=fmt, bias=bias), want.bfloat16())
    q, e = skg.quant_mx(xb, fmt)
    assert torch.equal(skg.gemm_mxfp4(q, h, xe=e, x_format=fmt, bias=bias, out_dtype=torch.float32), want)


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", sizes.PRODUCTS)
def test_nan_stays_in_its_row_and_column(skg, M, N, K, fmt, codes):
    """NaN and an infinity at the ends of rows of x, a NaN scale in a row of W."""
    g = np.random.default_rng(M * N)
    x, c = torch.from_numpy(_rows(g, M, K, fmt)).bfloat16(), g.integers(0, 16, (N, K))
    e = np.full((N, K // 32), 127)
    cb = torch.from_numpy((c[:, 0::2] | c[:, 1::2] << 4).astype(np.uint8)).to(DEV)

    def run(x, e):
        h = skg.mxfp4_pack(cb, torch.from_numpy(e.astype(np.uint8)).to(DEV))
        q, xe = skg.quant_mx(x.to(DEV), fmt) if codes else (x.to(DEV), None)
        return skg.gemm_mxfp4(q, h, xe=xe, x_format=fmt, out_dtype=torch.float32).cpu()

    clean = run(x, e)
    assert torch.isfinite(clean).all()
    bad = torch.zeros(M, N, dtype=torch.bool)
    x2, e2 = x.clone(), e.copy()
    for i, (row, at, v) in enumerate(((M // 3, 0, math.nan), (M // 2, K - 1, math.inf), (M - 1, K // 2, -math.inf))):
        if row > 0 or M == 1 and i == 0:
            x2[row, at] = v
            bad[row] = True
    for n, b in ((N // 2, 0), (N - 1, K // 32 - 1)):
        e2[n, b] = 255
        bad[:, n] = True
    out = run(x2, e2)
    assert torch.equal(torch.isnan(out), bad)
    assert torch.equal(out[~bad], clean[~bad])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,k,E,H,I", sizes.EXPERTS)
def test_experts_rows_do_not_touch_each_other(skg, T, k, E, H, I, fmt):
    """Every third token NaN, infinite or of weight NaN: the others' bits stay."""
    g = np.random.default_rng(T + E)
    w13, _ = _weights(skg, g, (E, 2 * I, H), 120)
    w2, _ = _weights(skg, g, (E, H, I), 120)
    x = torch.from_numpy(g.standard_normal((T, H))).bfloat16()
    ids = torch.from_numpy(np.argsort(g.random((T, E)), -1)[:, :k].astype(np.int32).copy())
    w = torch.from_numpy(g.random((T, k)) + 0.1).float()
    clean = skg.moe_mxfp4(x.to(DEV), ids.to(DEV), w.to(DEV), w13, w2, x_format=fmt).cpu()
    assert torch.isfinite(clean).all()
    hit = torch.arange(T) % 3 == 1
    x2, wt = x.clone(), w.clone()
    x2[1::9, 0] = math.nan
    x2[4::9, H - 1] = math.inf
    wt[7::9, k - 1] = math.nan
    out = skg.moe_mxfp4(x2.to(DEV), ids.to(DEV), wt.to(DEV), w13, w2, x_format=fmt).cpu()
    assert torch.equal(out[~hit], clean[~hit])
    assert torch.isnan(out[hit]).all()
