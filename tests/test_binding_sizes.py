"""Sizes past 31 bits are refused by the binding: ctypes would hand their low half
to the library (2^32 rows as none, and the output as it was allocated)."""
import pytest
import torch

import latency_skinny_gemm_amd as skg
from latency_skinny_gemm_amd import moe


@pytest.mark.parametrize("lead", [(1 << 31,), (1 << 32,), (1 << 16, 1 << 16), (3, 1 << 30)])
def test_row_counts_past_31_bits_are_refused(lead):
    with pytest.raises(skg.SkinnyGemmError) as err:
        moe._rows(lead)
    assert err.value.status == skg.ERR_UNSUPPORTED
    assert moe._rows(()) == 1 and moe._rows((0, 1 << 40)) == 0 and moe._rows(((1 << 31) - 1,)) == (1 << 31) - 1


@pytest.mark.gpu
def test_calls_with_more_rows_are_refused():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dev = "cuda:0"
    x = torch.empty(1 << 32, 8, dtype=torch.bfloat16, device=dev)  # never touched
    calls = [lambda: skg.rmsnorm(x, torch.ones(8, dtype=torch.bfloat16, device=dev)),
             lambda: skg.route(x.view(-1)[:1 << 32].view(-1, 1), 1),
             lambda: skg.route(torch.zeros(2, 16, device=dev), 1 + (1 << 32)),
             lambda: skg.route(torch.zeros(2, 16, device=dev), 1, groups=1 + (1 << 32))]
    for call in calls:
        with pytest.raises(skg.SkinnyGemmError) as err:
            call()
        assert err.value.status == skg.ERR_UNSUPPORTED
    del x
    torch.cuda.empty_cache()
