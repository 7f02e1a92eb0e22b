"""The short causal convolution and SiLU on a cache of windows, over packed prompts
(ssm_conv_fwd_cache) and over single tokens (ssm_conv_step_cache), against the plain
64-bit definition (needs MI355X).

Error bound: four products and a bias, added one after the other (at most 5
roundings of 2^-24 each of the absolute terms), carried through SiLU, whose slope is
at most 1.1; SiLU's own exponential, sum, reciprocal and product (its argument is
rounded once more: |u| 2^-24, and u e^-u stays below 1/2 where u is positive, below u
where it is not) 6 more; then half a step of the type. 16 in all.
"""
import pytest
import torch

import selective_state_space_16_amd as ssm
from delta_util import conv_reference
from gpu_util import say

pytestmark = pytest.mark.gpu
F8 = torch.float64


def make(lens, C, dtype, seed=0, spare=0, slots=None, num_slots=None, pad=8, bias=True):
    g = torch.Generator().manual_seed(seed)
    n, rows = len(lens), sum(lens) + spare
    num_slots = num_slots or n + 2
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return dict(lens=lens, wide=r(rows, C + pad).to(dtype), C=C, w=torch.rand(C, 4, generator=g) - 0.5, b=r(C) * 0.1 if bias else None,
                cu=torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32),
                slots=torch.randperm(num_slots, generator=g)[:n].int() if slots is None else torch.tensor(slots, dtype=torch.int32),
                resume=(torch.rand(n, generator=g) < 0.5).int(), cache=r(num_slots, C, 3).to(dtype))


def gpu(d):
    return {k: v.cuda() if torch.is_tensor(v) else v for k, v in d.items()}


def prompt(g, y=None, **kw):
    return ssm.ssm_conv_fwd_cache(g["wide"][:, :g["C"]], g["w"], g["cu"], g["slots"], g["cache"], conv_b=g["b"], y=y, **{"resume": g["resume"], **kw})


def step(g, y=None, **kw):
    return ssm.ssm_conv_step_cache(g["wide"][:, :g["C"]], g["w"], g["slots"], g["cache"], conv_b=g["b"], y=y, **kw)


def compare(d, g, y, y0, resume):
    yr, cache, mag = conv_reference(d["wide"][:, :d["C"]], d["w"], d["b"], d["lens"], d["slots"], resume, d["cache"], y0)
    half = 2.0 ** -8 if y.dtype == torch.bfloat16 else 2.0 ** -24
    assert ((y.cpu().to(F8) - yr).abs() <= half * yr.abs() + 16 * 2.0 ** -24 * mag).all()
    assert torch.equal(g["cache"].cpu().to(F8), cache)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,C,pad", [
    ([1], 8, 0), ([2], 7, 0), ([3], 64, 8), ([0], 16, 8), ([64, 0, 1, 2, 3, 4, 65, 66, 67, 128], 24, 8), ([5] * 90, 1, 3),
    ([1000], 257, 0), ([70, 200, 63], 2056, 8), ([130], 4104, 16), ([33, 31], 520, 5), ([1] * 300, 40, 8)])
def test_prompts(lens, C, pad, dtype):
    say(f"case conv prompts {lens[:6]} x{len(lens)} C={C} pad={pad} {dtype}")
    d = make(lens, C, dtype, seed=sum(lens) + C, spare=2, pad=pad)
    g, y0 = gpu(d), torch.full((sum(lens) + 2, C), 7.0, dtype=dtype)
    y = prompt(g, y0.cuda())
    torch.cuda.synchronize()
    compare(d, g, y, y0, d["resume"])


def test_without_bias_and_flags_and_left_out_sequences():
    say("case conv slots")
    d = make([70, 5, 66, 3, 9], 72, torch.bfloat16, seed=8, spare=5, slots=[2, -1, 2, 9, 0], num_slots=4, bias=False)
    g, y0 = gpu(d), torch.full((158, 72), 7.0, dtype=torch.bfloat16)
    y = prompt(g, y0.cuda(), resume=None)
    torch.cuda.synchronize()
    compare(d, g, y, y0, None)
    assert bool((y[-5:] == 7).all()) and bool((y[70:144] == 0).all())


@pytest.mark.parametrize("cu", [[0, 500, 100], [-5, 30, 64], [90, 20, 10], [0, 0, 2 ** 31 - 1], [64, 64, 64]])
def test_offsets_outside_the_rows_stay_inside_the_tensors(cu):
    say(f"case conv offsets {cu}")
    g = gpu(make([40, 24], 64, torch.bfloat16, seed=9))
    y = torch.full((64 + 128, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    win = torch.full((12, 64, 3), 7.0, dtype=torch.bfloat16, device="cuda")
    g["cache"], g["cu"] = win[4:8], torch.tensor(cu, dtype=torch.int32, device="cuda")
    prompt(g, y[64:128])
    torch.cuda.synchronize()
    assert (y[:64] == 7).all() and (y[128:] == 7).all() and (win[:4] == 7).all() and (win[8:] == 7).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("batch,C,pad", [(1, 8, 0), (5, 1001, 3), (33, 2560, 8), (300, 24, 0), (2, 4100, 4)])
def test_tokens(batch, C, pad, dtype):
    say(f"case conv tokens {batch} {C} {dtype}")
    d = make([1] * batch, C, dtype, seed=batch, pad=pad)
    if batch > 4:
        d["slots"][3], d["slots"][1] = d["slots"][2], -1
    g, y0 = gpu(d), torch.zeros(batch, C, dtype=dtype)
    y = step(g, y0.cuda())
    torch.cuda.synchronize()
    compare(d, g, y, y0, torch.ones(batch))


def test_pieces_give_the_bits_of_the_whole():
    """A prompt in pieces, its last tokens one at a time, on another stream: each row
    is the same sum."""
    say("case conv pieces")
    d = make([150], 200, torch.bfloat16, seed=11, slots=[1])
    whole, g = gpu(d), gpu(d)
    yw, ys, row = prompt(whole, resume=None), [], 0
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    for n in (64, 1, 70, 2):
        part = dict(g, wide=g["wide"][row:row + n], cu=torch.tensor([0, n], dtype=torch.int32, device="cuda"))
        flag = torch.tensor([1 if row else 0], dtype=torch.int32, device="cuda")
        other.wait_stream(torch.cuda.current_stream())
        ys.append(prompt(part, resume=flag, stream=other))
        torch.cuda.current_stream().wait_stream(other)
        row += n
    for t in range(row, 150):
        ys.append(step(dict(g, wide=g["wide"][t:t + 1])))
    torch.cuda.synchronize()
    assert torch.equal(torch.cat(ys), yw) and torch.equal(g["cache"], whole["cache"])


def test_captured_calls_take_new_lengths():
    say("case conv graph")
    lens = [[100, 30, 62], [0, 150, 42], [192, 0, 0], [1, 1, 190]]
    ds = [make(ls, 96, torch.float32, seed=20 + i) for i, ls in enumerate(lens)]
    eager = [gpu(d) for d in ds]
    want = [prompt(g) for g in eager]
    live = gpu(ds[0])
    y = torch.zeros_like(want[0])
    prompt(live, y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        prompt(live, y)
    for d, g, w in zip(ds, eager, want):
        for key in ("wide", "w", "b", "cu", "slots", "resume", "cache"):
            live[key].copy_(d[key])
        graph.replay()
        prompt(gpu(d))
        torch.cuda.synchronize()
        assert torch.equal(y, w) and torch.equal(live["cache"], g["cache"])


def test_a_value_that_is_not_finite_reaches_four_tokens():
    say("case conv nan")
    d = make([100], 64, torch.bfloat16, seed=12)
    d["wide"][50, 3] = float("inf")
    y = prompt(gpu(d)).float().cpu()
    bad = ~torch.isfinite(y)
    keep = torch.zeros_like(bad)
    keep[50:54, 3] = True
    assert not (bad & ~keep).any() and bad[50:54, 3].any()


def test_a_token_written_over_its_input():
    say("case conv in place")
    d = make([1] * 3, 64, torch.float32, seed=13, pad=0)
    g, h = gpu(d), gpu(d)
    want = step(g)
    step(h, y=h["wide"])
    torch.cuda.synchronize()
    assert torch.equal(want, h["wide"]) and torch.equal(g["cache"], h["cache"])
