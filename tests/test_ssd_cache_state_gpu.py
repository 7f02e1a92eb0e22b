"""The state that packed prompts leave (ssm_ssd_fwd_cache) where independent
parts of it are of unlike size, against the plain 64-bit definition (needs
MI355X): a float32 state holds each of its elements to its own absolute terms,
whatever its neighbours, its other columns or other tokens hold.

The bound is that of the operator's other tests: 32 float32 roundings per term
and 3 per token that carries it, relative to the element's absolute terms (the
convolution's included). Powers of two scale a channel's taps and bias, so they
scale its absolute terms as well.
"""
import pytest
import torch

from block_util import ssd_inputs, ssd_reference, to_gpu
from gpu_util import say
from test_ssd_cache_gpu import U, before, prompt

pytestmark = pytest.mark.gpu


def unlike(d, which, most):
    """Scales the channels of B, or of x, by powers of two from 1 down to 2^-most."""
    H, P, G, N = d["H"], d["P"], d["G"], d["N"]
    first, n, width = (0, H * P, P) if which == "x" else (H * P, G * N, N)
    f = torch.exp2(-torch.linspace(0, most, width).round())[torch.randperm(width, generator=torch.Generator().manual_seed(1))]
    f = f.repeat(n // width)
    d["conv_w"][first:first + n] *= f[:, None]
    if d["conv_b"] is not None:
        d["conv_b"][first:first + n] *= f


def state_within(d, g, what):
    _, st, _, _, sa = ssd_reference(d, before(d))
    got = g["state_cache"].cpu().double()
    tol = (32 + 3 * max(d["lens"])) * U * sa
    say(f"  {what}: state worst of bound {float(((got - st).abs() / tol.clamp_min(1e-300)).max()):.3f}")
    assert torch.isfinite(got).all()
    assert ((got - st).abs() <= tol).all(), what


@pytest.mark.parametrize("lens", [[60, 9, 130], [1400]])
@pytest.mark.parametrize("N", [64, 128])
@pytest.mark.parametrize("which", ["B", "x"])
def test_channels_of_unlike_size(which, N, lens):
    say(f"case unlike {which} N={N} {lens}")
    d = ssd_inputs(lens, 2, 64, 1, N, seed=31 + N, scale=4.0)
    d["state_cache"] *= 0  # the absolute terms of an earlier state would cover a quiet column
    unlike(d, which, 40)
    g = to_gpu(d)
    prompt(g, before(d).cuda())
    torch.cuda.synchronize()
    state_within(d, g, which)


def test_tokens_of_unlike_step():
    """Columns of B that only the first tokens fill, whose steps are 2^-40 of the
    later ones' (and nothing decays much): the later tokens add exact zeros."""
    say("case unlike steps")
    d = ssd_inputs([60, 100], 2, 64, 1, 64, seed=33)
    d["resume"][:] = 0
    d["A"] *= 1e-3
    d["dt_bias"][:] = 0
    cols = slice(64 + 128, 64 + 128 + 32)  # half the columns of B
    d["conv_b"][128:128 + 32] = 0
    for lo, n in ((0, 60), (60, 100)):
        d["proj"][lo:lo + 20, 64 + d["C"]:64 + d["C"] + 2] = -27.0
        d["proj"][lo + 10:lo + n, cols] = 0
    g = to_gpu(d)
    prompt(g, before(d).cuda())
    torch.cuda.synchronize()
    state_within(d, g, "steps")
