"""What the binding of latent attention refuses before it looks for a device."""
import pytest

import latency_skinny_gemm_amd as skg


class _Stream:
    """Never used: the refusal comes first."""
    device = "cuda:0"
    cuda_stream = 0


@pytest.mark.parametrize("heads", [1 << 31, (1 << 32) + 16, -1])
def test_head_counts_past_31_bits_are_refused(heads):
    """ctypes would reserve for their low half: 16 heads."""
    with pytest.raises(skg.SkinnyGemmError) as err:
        skg.reserve_latent(heads, stream=_Stream())
    assert err.value.status == skg.ERR_UNSUPPORTED
