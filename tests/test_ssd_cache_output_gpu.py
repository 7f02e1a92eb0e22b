"""y of packed prompts (ssm_ssd_fwd_cache) to the bits that its products carry,
and where independent parts of its inputs are of unlike size, against the plain
64-bit definition (needs MI355X).

The bound of an element: half a step of its bfloat16 rounding, 2^-8 of its value;
operands of 16 significant bits, 2^-16 of the absolute terms each time one is
rounded or the product of two small parts is left out: three for a term of the
chunk itself (x, its factor, the product), three for one through the state (the
state, C, the product) and four more inside the state (x, w o x, B, the
product), so at most 8 with one to spare, relative to the element's own absolute
terms behind the SiLU; and 40 float32 roundings and 3 per token that carries a
term, relative to its absolute terms with the convolution's included (powers of
two on a channel's taps and bias scale both).

Two values that lie e apart round to bfloat16 values one step apart with
probability e / step, so over many elements the squared distance from the
definition's own rounding is the sum of e step. Seven roundings of up to 2^-16
that are uniform and independent of each other, the same for all terms at worst,
are 2^-16 sqrt(7 / 3) on average; two 2^-16 are allowed, and 32 float32 roundings
(40 and 3 per token, likewise, of at most 300 tokens). Where all terms are of one
sign the sum of the terms is the value itself, and operands of 11 bits fail this.
"""
import pytest
import torch

from block_util import F8, owned, silu, softplus, ssd_inputs, ssd_reference, to_gpu, views
from gpu_util import say
from test_ssd_cache_gpu import U, before, prompt
from test_ssd_cache_state_gpu import unlike

pytestmark = pytest.mark.gpu


def terms_behind_silu(d):
    """The absolute terms of y by token, with x, B and C as the SiLU leaves them."""
    H, P, G, N, C = d["H"], d["P"], d["G"], d["N"], d["C"]
    raw, dtr = (t.to(F8) for t in views(d))
    zero = lambda v, *n: torch.zeros(n, dtype=F8) if v is None else v.to(F8)  # noqa: E731
    b, bias, D = zero(d["conv_b"], C), zero(d["dt_bias"], H), zero(d["Dskip"], H).abs()
    out, row, grp = torch.zeros(raw.shape[0], H, P, dtype=F8), 0, torch.arange(H) // (H // G)
    for s, (n, slot) in enumerate(zip(d["lens"], owned(d["slots"], d["state_cache"].shape[0]))):
        go = d["resume"][s] != 0
        past = d["conv_cache"][slot].to(F8).t() if go else torch.zeros(3, C, dtype=F8)
        S = d["state_cache"][slot].to(F8).abs() if go else torch.zeros(H, P, N, dtype=F8)
        seq = torch.cat([past, raw[row:row + n]])
        v = silu(sum(seq[j:j + n] * d["conv_w"][:, j].to(F8) for j in range(4)) + b).abs()
        dt = softplus(dtr[row:row + n] + bias)
        x = v[:, :H * P].reshape(n, H, P)
        B, Cm = v[:, H * P:H * P + G * N].reshape(n, G, N)[:, grp], v[:, H * P + G * N:].reshape(n, G, N)[:, grp]
        for t in range(n):
            S = torch.exp(dt[t] * d["A"].to(F8))[:, None, None] * S + (dt[t][:, None] * x[t])[:, :, None] * B[t][:, None, :]
            out[row + t] = (S * Cm[t][:, None, :]).sum(2) + D[:, None] * x[t]
        row += n
    return out


def positive(d):
    """Makes every term of y positive."""
    d["proj"][:, 64:64 + d["C"]].abs_()
    for k in ("conv_w", "conv_b", "conv_cache", "state_cache"):
        d[k].abs_()


def output_within(d, what, average=None):
    """Each element's error; and over the rows `average`, if given, that from the
    definition's rounding."""
    g, y0 = to_gpu(d), before(d)
    got = prompt(g, y0.cuda()).cpu().double()
    torch.cuda.synchronize()
    rows = sum(d["lens"])
    assert torch.equal(got[rows:], y0[rows:].double())
    y, _, _, ya, _ = (t[:rows] if t.shape[0] == y0.shape[0] else t for t in ssd_reference(d, y0))
    got, terms = got[:rows], terms_behind_silu(d)[:rows]
    tol = 2.0 ** -8 * y.abs() + 8 * 2.0 ** -16 * terms + (40 + 3 * max(d["lens"])) * U * ya
    err = (got - y).abs()
    say(f"  {what}: y worst of bound {float((err / tol.clamp_min(1e-300)).max()):.3f}")
    assert torch.isfinite(got).all()
    assert (err <= tol).all(), what
    if average is not None:
        got, y, terms, ya = got[average], y[average], terms[average], ya[average]
        exact = y.bfloat16().double()
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -100))) - 7)
        off, most = (got - exact).norm(), torch.sqrt(((2 * 2.0 ** -16 * terms + 32 * U * ya) * step).sum())
        say(f"  {what}: from the definition's rounding relL2 {float(off / exact.norm()):.2e} of {float(most / exact.norm()):.2e}")
        assert off <= most, what


@pytest.mark.parametrize("lens,H,P,G,N", [([300], 3, 64, 1, 128), ([64, 65, 1, 200], 4, 64, 2, 64), ([130], 2, 192, 1, 128)])
@pytest.mark.parametrize("step", [(1e-6, 1e-5), (1e-2, 1e-1)])
def test_bits(lens, H, P, G, N, step):
    """Every term positive; y is D x with steps of nothing, and mostly the sums with others."""
    say(f"case bits {lens} H={H} P={P} G={G} N={N} {step}")
    d = ssd_inputs(lens, H, P, G, N, seed=41, spare=2, step=step)
    positive(d)
    output_within(d, "all", average=slice(None))


@pytest.mark.parametrize("lens", [[60, 9, 130], [1400]])
@pytest.mark.parametrize("N", [64, 128])
@pytest.mark.parametrize("which", ["B", "x"])
def test_channels_of_unlike_size(which, N, lens):
    say(f"case unlike {which} N={N} {lens}")
    d = ssd_inputs(lens, 2, 64, 1, N, seed=42 + N, scale=4.0)
    d["state_cache"] *= 0
    unlike(d, which, 40)
    output_within(d, which)


@pytest.mark.parametrize("few", [1e-4, 1.0])
def test_one_loud_channel(few):
    """One channel of a head 2^18 times louder than the others over many chunks, with
    little decay (`few` of the usual) and with the usual."""
    say(f"case loud channel {few}")
    d = ssd_inputs([1344], 2, 64, 1, 128, seed=43)
    d["A"] *= few
    d["conv_w"][5] *= 2.0 ** 18
    d["conv_b"][5] *= 2.0 ** 18
    output_within(d, "loud")


@pytest.mark.parametrize("axis", ["rows", "columns"])
def test_state_of_unlike_size(axis):
    """A resumed state with rows (channels), or columns, of 2^-32 to 2^32."""
    say(f"case state {axis}")
    d = ssd_inputs([90, 70], 2, 64, 1, 128, seed=44)
    d["resume"][:] = 1
    n = 64 if axis == "rows" else 128
    f = torch.exp2(torch.linspace(-32, 32, n).round())[torch.randperm(n, generator=torch.Generator().manual_seed(2))]
    d["state_cache"] *= f[:, None] if axis == "rows" else f
    if axis == "columns":  # C reads the louder a column the less
        d["conv_w"][128 + 128:] /= f[:, None]
        d["conv_b"][128 + 128:] /= f
    output_within(d, axis)


def test_tokens_of_unlike_step():
    """Tokens with steps of 2^-40 ahead of ones with steps of about one in a chunk:
    what stands in y of the first is theirs alone."""
    say("case unlike steps")
    d = ssd_inputs([60, 100], 2, 64, 1, 64, seed=45, dskip=False)
    d["resume"][:] = 0
    d["dt_bias"][:] = 0
    for row in (0, 60):
        d["proj"][row:row + 30, 64 + d["C"]:64 + d["C"] + 2] = -27.0
    output_within(d, "steps")


def test_tokens_of_unlike_size():
    """Tokens whose x, B and C are 2^30 times as large as their neighbours'."""
    say("case unlike tokens")
    d = ssd_inputs([150], 2, 64, 1, 128, seed=46)
    for row in (25, 50, 140):
        d["proj"][row, 64:64 + d["C"]] *= 2.0 ** 30
    output_within(d, "tokens")


def test_decays_behind_steps_that_forget():
    """Ordinary tokens behind ones whose steps leave nothing (a decay of 2^-256 or
    less each): the decays between them are differences of sums of thousands."""
    say("case behind forgetting steps")
    d = ssd_inputs([64] * 4, 2, 64, 1, 64, seed=47, dskip=False)
    for row in range(0, 256, 64):
        d["proj"][row:row + 50, 64 + d["C"]:64 + d["C"] + 2] = 300.0
    positive(d)
    output_within(d, "behind", average=torch.arange(256) % 64 >= 50)
