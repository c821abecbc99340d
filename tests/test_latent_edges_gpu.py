"""Latent attention at the ends of its domain on the GPU: scales whose products leave
fp32, rows that hold infinities and NaN in every form of the kernel, long caches.
Against the plain implementations of tests/latent_reference.py and its bounds."""
import pytest
import torch

from tests import latent_reference as ref
from tests.test_latent_gpu import DEV, SCALE, _cache, _dev, _ints, _randn, _starts, skg  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("counts,lens,H", [([1], [70], 3), ([40, 7], [300, 9], 20)])
def test_scales_whose_product_leaves_fp32(skg, counts, lens, H):  # noqa: F811
    """Softmax scale 2^126, cache scale 4: scores of zero stay zero, and scores that fit are there."""
    page, softmax = 16, 2.0 ** 126
    cache, _, table = _cache(1, lens, page, True)
    rows = torch.randint(0, 5, cache.shape, generator=torch.Generator().manual_seed(2)).float()
    cache = (rows * (1 - 2 * (torch.arange(576) & 1))).to(torch.float8_e4m3fn)
    scale = torch.tensor([4.0])
    T = sum(counts)
    q = torch.zeros(T, H, 576)
    q[:, 1:, 7] = 2.0 ** -126     # scores 4 times a code; head 0: all zero
    q[:, 2:, 520] = -2.0 ** -126
    q = q.bfloat16()
    out, bound = ref.attention(q, cache, scale, table, lens, _starts(counts).tolist(), softmax)
    got = skg.latent_attention(*_dev(q, cache, table, _ints(lens)), softmax, q_starts=_starts(counts).to(DEV), scale=scale.to(DEV))
    ref.check(got, out, bound)
