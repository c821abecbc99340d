"""route with more tokens than one grid holds."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def skg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import latency_skinny_gemm_amd as m
    m.lib()
    return m


@pytest.mark.parametrize("T,E,k,o", [((1 << 26) + 3, 9, 9, dict(scores="sigmoid")),   # a wave a token
                                     ((1 << 28) + 5, 8, 1, dict())])                  # 16 lanes a token
def test_more_tokens_than_a_grid_holds(skg, T, E, k, o):
    """2^32 work-items and more: the same 2^20 tokens over and over, with the
    same choices and weights over and over."""
    n = 1 << 20
    l = torch.randn(n, E, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    one = skg.route(l, k, **o)
    many = skg.route(torch.cat([l.repeat(T // n, 1), l[:T % n]]), k, **o)
    assert all(a.shape == (T, k) for a in many)
    for a, b in zip(many, one):
        assert torch.equal(a[T // n * n:], b[:T % n])
        for i in range(T // n):
            assert torch.equal(a[i * n:(i + 1) * n], b), i
