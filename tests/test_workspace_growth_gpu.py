"""A workspace that grows leaves its old buffers allocated (a captured graph may
use them): how much memory that takes."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def skg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import latency_skinny_gemm_amd as m
    m.lib()
    return m


def _taken(f):
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0]
    f()
    torch.cuda.synchronize()
    return before - torch.cuda.mem_get_info()[0]


def test_requests_that_creep_up_leave_a_bounded_rest(skg):
    """A buffer is half as large again as the one it replaces, at least: the last
    is at most 1.5 times the largest request, and all before it together at most
    twice the last.  4.5 times the largest request in all; 60 requests of
    growing size, each with a buffer of its own, would be 45 times."""
    sizes = [1000 + 50 * i for i in range(61)]
    args = dict(k=4, H=2880, I=2880, E=8)
    skg.release_all()
    one = _taken(lambda: skg.reserve_moe(max_T=sizes[-1], **args, stream=torch.cuda.Stream()))
    skg.release_all()
    s = torch.cuda.Stream()

    def creep():
        for T in sizes:
            skg.reserve_moe(max_T=T, **args, stream=s)

    many = _taken(creep)
    skg.release_all()
    assert one > 100 << 20
    assert many <= 4.5 * one + (64 << 20)


def test_a_call_in_a_grown_workspace_and_after_release(skg):
    """The workspace grows between calls of one stream; results stay."""
    E, k, H, I = 8, 2, 96, 64
    g = torch.Generator(device="cuda").manual_seed(1)

    def weight(*shape):
        return skg.mxfp4_pack(*skg.quant_mx(torch.randn(*shape, device="cuda", generator=g).bfloat16(), "e2m1"))

    w13, w2 = weight(E, 2 * I, H), weight(E, H, I)
    x = torch.randn(9000, H, device="cuda", generator=g).bfloat16()
    ids = torch.randint(0, E, (9000, k), device="cuda", generator=g).int()
    w = torch.rand(9000, k, device="cuda", generator=g)
    skg.release_all()
    first = {T: skg.moe_mxfp4(x[:T], ids[:T], w[:T], w13, w2).clone() for T in (3000, 3100, 9000)}
    torch.cuda.synchronize()
    skg.release_all()
    for T in (9000, 3100, 3000):
        assert torch.equal(skg.moe_mxfp4(x[:T], ids[:T], w[:T], w13, w2), first[T])
