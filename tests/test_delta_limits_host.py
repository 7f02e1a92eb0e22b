"""Sizes at the border of what the gated delta rule over packed prompts can launch (CPU
only; every refusal comes before any HIP call)."""
import pytest

import selective_state_space_16_amd as ssm
from test_delta_abi_host import fwd


def walk_threads(seqs, H, P, G):
    """Four threads per column of a state, the groups of all sequences rounded up to whole
    eights (one for each XCD)."""
    return (G * seqs + 7) // 8 * 8 * (H // G) * P * 4


@pytest.mark.parametrize("seqs,H,P,G", [(129, 32512, 256, 1), (257, 32512, 128, 1), (513, 32512, 64, 1), (173, 32000, 192, 2), (1673, 10000, 64, 1)])
def test_launches_that_rounding_takes_to_2_to_the_32_threads_are_refused(seqs, H, P, G):
    assert walk_threads(seqs, H, P, G) >= 2 ** 32 > seqs * H * P * 4
    kw = dict(H=H, P=P, G=G, N=64, num_slots=1, vs=H * P, ds=H, bs=H)
    assert fwd(seqs=seqs, rows=0, **kw) == -4
    assert ssm.ssm_delta_fwd_cache_workspace_bytes(seqs, 0, H, P, G, 64, ssm.SSM_BF16) == 0
    # refused further on where it fits: no workspace
    fit = seqs // 8 * 8
    assert walk_threads(fit, H, P, G) < 2 ** 32
    assert fwd(seqs=fit, rows=0, ws=None, **kw) == -6
    assert ssm.ssm_delta_fwd_cache_workspace_bytes(fit, 0, H, P, G, 64, ssm.SSM_BF16) > 0
