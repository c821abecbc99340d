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


@pytest.mark.parametrize("counts,lens", [([1], [6205]), ([1, 1], [6205, 40])])
def test_scale_whose_quotient_is_no_normal_number(skg, counts, lens):  # noqa: F811
    """A mean of equal rows is that row: 448 2^-130 is a number of bf16, and every sum on the way (a multiple of 448
    below 2^24 of them) one of fp32.  2^-130 / 6205 is 84.49 times fp32's smallest number, of which 84 is 0.6 % off."""
    page, H = 64, 3
    cache, _, table = _cache(5, lens, page, True)
    cache = torch.full(cache.shape, 448.0).to(torch.float8_e4m3fn)
    cache[..., 1::2] = torch.tensor(-1.0).to(torch.float8_e4m3fn)
    scale = torch.tensor([2.0 ** -130])
    q = torch.zeros(len(lens), H, 576, dtype=torch.bfloat16)
    got = skg.latent_attention(*_dev(q, cache, table, _ints(lens)), SCALE, scale=scale.to(DEV)).cpu()
    assert (got[..., 0::2].double() == 448 * 2.0 ** -130).all()
    assert (got[..., 1::2].double() == -(2.0 ** -130)).all()
