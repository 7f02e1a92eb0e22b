"""Sizes at the edge of what one launch reaches, in the C ABI of the operators
around the SSD layer (CPU only; every refusal comes before any HIP call)."""
import pytest

from test_block_abi_host import gate_bwd, gate_fwd


@pytest.mark.parametrize("call", [gate_fwd, gate_bwd])
def test_channels_whose_reduction_would_have_two_to_the_32_threads(call):
    """64 columns of the gradient of the weight take 1024 threads."""
    D = (1 << 28) - 1
    wide = dict(xs=D, zs=D) if call is gate_fwd else dict(xs=D, zs=D, dzs=D)
    assert call(rows=1, D=D, groups=16385, **wide) == -4
