"""The sums of the MXFP4 products are fp32's, in both formats of the rows.

Derived: rows and weights are chosen so that every product is a multiple of
2^-10 (e4m3; 2^-2 in e2m1) and the sum of all their magnitudes is below 2^14
(2^18): every partial sum, in whatever order, then is an fp32 number and the
result exact.  Products next to each other differ by up to 2^16, so that a sum
that holds fewer bits shows.
For the experts the hidden value is v = g * u / (1 + exp(-g)) of two such exact
sums; the kernel's exponential, reciprocal and products leave it within
(8 + 2 |g|) 2^-23 of its value, and its code is that of the exact value wherever
that lies twice as far from a tie.
"""
import math

import numpy as np
import pytest
import torch

from tests import mx_reference as ref

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


def _rows(g, M, K, fmt):
    """Values of codes with scale 1; in e4m3 tiny ones, and a few large ones with
    small ones beside them, of whose products the sum has to keep all bits."""
    if fmt == "e2m1":
        x = ref.E2M1_VALUES[g.integers(0, 8, (M, K))]
    else:
        x = ref.E4M3_VALUES[g.integers(0, 33, (M, K))]  # up to 2^-3
        for i, row in enumerate(x):
            n, lo, hi = ((24, 88, 105), (4, 112, 127), (12, 56, 113))[i % 3]  # 16 to 64; 128 to 448; 1 to 128
            at = g.permutation(K)[:n]
            row[at ^ 1] = ref.E4M3_VALUES[g.integers(56, 72, len(at))]  # 1 to 3.75
            row[at] = ref.E4M3_VALUES[g.integers(lo, hi, len(at))]
    x *= np.where(g.integers(0, 2, (M, K)) == 1, -1.0, 1.0)
    x[:, ::32] = 448.0 if fmt == "e4m3" else 6.0  # the block's largest, so that its scale is 1
    return x


def _weights(skg, g, shape, scale=127):
    """(packed, values): any codes, but 0 for the first value of a block."""
    c = g.integers(0, 16, shape)
    c[..., ::32] = 0
    e = np.full((*shape[:-1], shape[-1] // 32), scale)
    h = skg.mxfp4_pack(torch.from_numpy(ref.pack_bytes(c, "e2m1")).to(DEV), torch.from_numpy(e.astype(np.uint8)).to(DEV))
    return h, ref.dequantise(c, e, "e2m1")


# one row, whole and ragged blocks of rows, each tile
SIZES = [(1, 40, 7168), (1, 1000, 96), (7, 500, 2880), (16, 576, 4096), (37, 1111, 2880), (102, 539, 5472),
         (173, 470, 4768), (43, 1173, 5088), (24, 4096, 1056), (128, 2112, 544), (500, 1100, 160), (512, 600, 96),
         (512, 2100, 544), (490, 2180, 1120)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", SIZES)
def test_product(skg, M, N, K, fmt):
    g = np.random.default_rng(M + N + K)
    x = _rows(g, M, K, fmt)
    h, w = _weights(skg, g, (N, K))
    assert (np.abs(x) @ np.abs(w).T).max() < (2.0 ** 14 if fmt == "e4m3" else 2.0 ** 18)
    want = torch.from_numpy(x @ w.T).float()
    assert torch.equal(want.double(), torch.from_numpy(x @ w.T))
    xd = torch.from_numpy(x).bfloat16().to(DEV)
    assert torch.equal(skg.gemm_mxfp4(xd, h, x_format=fmt, out_dtype=torch.float32).cpu(), want)
    q, e = skg.quant_mx(xd, fmt)
    assert torch.equal(skg.gemm_mxfp4(q, h, xe=e, x_format=fmt, out_dtype=torch.float32).cpu(), want)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,k,E,H,I", [(1, 1, 1, 96, 64), (5, 2, 6, 1056, 992), (72, 4, 72, 480, 480),
                                       (200, 4, 40, 288, 288), (600, 8, 12, 96, 96), (2500, 2, 20, 128, 96)])
def test_experts_hidden_codes(skg, T, k, E, H, I, fmt):
    """W2 hands the hidden codes on as they are."""
    g = np.random.default_rng(T + H)
    x = _rows(g, T, H, fmt)
    w13, v13 = _weights(skg, g, (E, 2 * I, H), 127 - 9 if fmt == "e4m3" else 127 - 8)
    c = np.zeros((E, H, I), dtype=np.int64)
    c[:, np.arange(I), np.arange(I)] = 2  # 1.0
    w2 = skg.mxfp4_pack(torch.from_numpy(ref.pack_bytes(c, "e2m1")).to(DEV),
                        torch.full((E, H, I // 32), 127, dtype=torch.uint8, device=DEV))
    ids = torch.from_numpy(np.argsort(g.random((T, E)), -1)[:, :k].astype(np.int32).copy())
    weights = torch.zeros(T, k)
    weights[:, 0] = 1.0
    out = skg.moe_mxfp4(torch.from_numpy(x).bfloat16().to(DEV), ids.to(DEV), weights.to(DEV), w13, w2, x_format=fmt)
    got = ref.f64(out)
    assert np.all(got[:, I:] == 0)
    sure = 0
    for t in range(T):
        gate, up = np.split(v13[int(ids[t, 0])] @ x[t], 2)
        v = gate / (1.0 + np.exp(-gate)) * up
        near = 2 * (8 + 2 * np.abs(gate)) * 2.0 ** -23
        lo, hi = ref.rounded(v * (1 - near), fmt), ref.rounded(v * (1 + near), fmt)
        # a block whose scale is not certain is left out whole: its values round twice
        certain = np.repeat((ref.quantise(v * (1 - near), fmt)[1] == ref.quantise(v * (1 + near), fmt)[1]), 32) & (lo == hi)
        assert np.array_equal(got[t, :I][certain], lo[certain]), t
        sure += certain.sum()
    assert sure > 0.99 * T * I
