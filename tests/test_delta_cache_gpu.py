"""The gated delta rule on a cache of states, over packed prompts
(ssm_delta_fwd_cache) and over single tokens (ssm_delta_step_cache), against the
plain 64-bit definition (needs MI355X).

Error bounds (delta_reference says how errors are carried):
- the state: a token's sums have at most 128 terms, one rounding of 2^-24 each in
  the worst order, and about 20 more roundings per term (the lengths of key and
  query, softplus, decay, gates, the parts that an operand is split into): c =
  148 * 2^-24 of the absolute values. Errors of rounding are as often up as down, so
  in the 2-norm the root of that count is left, 12 * 2^-24 < 1e-6; twice that is
  asserted.
- y is rounded once to its type: half a step, 2^-8 (bfloat16) or 2^-24 (float32). In
  a prompt its products take operands of 16 bits (2^-17 each, at most four of them
  in a term: cy = 2^-15); a single token's are float32. In the 2-norm a rounding that
  is anywhere within half a step is at most 2^-8 / sqrt(3) = 2.26e-3 (bfloat16), and
  float32 results are as near as the state.
"""
import pytest
import torch

import selective_state_space_16_amd as ssm
from block_util import owned, to_gpu
from delta_util import delta_inputs, delta_reference, parts
from gpu_util import say

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
C = 148 * U


def prompt(g, y=None, **kw):
    kw = {"resume": g["resume"], **kw}
    return ssm.ssm_delta_fwd_cache(*parts(g), g["A"], g["cu"], g["slots"], g["state_cache"], dt_bias=g["dt_bias"], y=y, **kw)


def step(g, y=None, **kw):
    return ssm.ssm_delta_step_cache(*parts(g), g["A"], g["slots"], g["state_cache"], dt_bias=g["dt_bias"], y=y, **kw)


def before(d):
    return torch.full((d["qkv"].shape[0], d["H"], d["P"]), 7.0, dtype=d["qkv"].dtype)


def compare(d, g, y, y0, resume=True, products=True, what="", **kw):
    """`y` and the cache in `g` against the definition on the inputs `d`."""
    yr, st, yt, stol = delta_reference(d, y0, resume, c=C, cy=2.0 ** -15 if products else 0.0, **kw)
    got, gs = y.cpu().double(), g["state_cache"].cpu().double()
    half = 2.0 ** -8 if d["qkv"].dtype == torch.bfloat16 else 2.0 ** -24
    ty = half * yr.abs() + yt
    rel = lambda a, b: float((a - b).norm() / b.norm().clamp_min(1e-300))  # noqa: E731
    worst = lambda a, b, tol: float(((a - b).abs() / tol.clamp_min(1e-300)).max()) if a.numel() else 0.0  # noqa: E731
    say(f"  {what} y relL2={rel(got, yr):.2e} of bound {worst(got, yr, ty):.2f}, state relL2={rel(gs, st):.2e} of bound {worst(gs, st, stol):.2f}")
    assert torch.isfinite(got).all() and torch.isfinite(gs).all()
    assert ((got - yr).abs() <= ty).all(), "y"
    assert ((gs - st).abs() <= stol).all(), "state"
    assert rel(gs, st) <= 2e-6
    inside = slice(0, sum(d["lens"]))
    assert rel(got[inside], yr[inside]) <= (2.3e-3 if half > U else 2e-6)
    mine = set(owned(d["slots"], st.shape[0]))
    for k in range(st.shape[0]):
        if k not in mine:
            assert torch.equal(g["state_cache"][k].cpu(), d["state_cache"][k]), "a slot of no sequence"


CASES = [
    ([1], 2, 64, 1, 128), ([37], 3, 64, 3, 64), ([64], 2, 64, 1, 64), ([65], 2, 64, 2, 128), ([128], 1, 128, 1, 128),
    ([0, 1, 2, 3, 4, 5], 4, 64, 2, 64), ([63, 64, 65, 127, 128, 129], 4, 64, 1, 128), ([300, 0, 5], 6, 128, 2, 128),
    ([1] * 70, 1, 64, 1, 64), ([200, 33], 2, 128, 1, 64), ([90], 3, 192, 3, 64), ([130, 7], 2, 256, 2, 128),
    ([0], 2, 64, 1, 128), ([0, 0, 9], 5, 64, 5, 64), ([1500], 2, 64, 1, 128), ([700, 40, 1111], 2, 128, 1, 64),
    ([16, 15, 17, 31, 32, 33, 47, 48, 49], 2, 64, 2, 128),
]


@pytest.mark.parametrize("lens,H,P,G,N", CASES)
def test_prompts(lens, H, P, G, N):
    say(f"case delta prompts {lens[:6]} x{len(lens)} H={H} P={P} G={G} N={N}")
    d = delta_inputs(lens, H, P, G, N, seed=sum(lens) + H, spare=3)
    g, y0 = to_gpu(d), before(d)
    y = prompt(g, y0.cuda())
    torch.cuda.synchronize()
    compare(d, g, y, y0)


@pytest.mark.parametrize("kw,call", [
    (dict(dt_bias=False), {}), ({}, dict(resume=None)), ({}, dict(scale=1.0)), ({}, dict(norm_eps=0.5)),
    (dict(scale=0.05), dict(norm_eps=-1.0)), (dict(scale=1e-4), {}), (dict(scale=1e4), {}),
    (dict(same_keys=0.9), {}), (dict(same_keys=1.0), {}), (dict(step=(1.0, 30.0)), {}), (dict(step=(1e-7, 1e-6)), {}),
    (dict(A=(0.0, 0.0)), {}), (dict(A=(1e4, 1e5)), {})])
def test_prompts_of_other_kinds(kw, call):
    """Without a bias or flags, other lengths and scales, keys that are nearly or
    wholly the same, decays near one, of one and to nothing."""
    say(f"case delta prompts {kw} {call}")
    d = delta_inputs([150, 20, 64], 2, 64, 1, 128, seed=6, **kw)
    g, y0 = to_gpu(d), before(d)
    y = prompt(g, y0.cuda(), **call)
    torch.cuda.synchronize()
    ref = {k: v for k, v in call.items() if k != "resume"}
    compare(d, g, y, y0, resume="resume" not in call, **ref)


def test_left_out_sequences_and_rows_behind_the_last():
    say("case delta slots")
    d = delta_inputs([70, 5, 66, 3, 9], 2, 64, 1, 64, seed=8, spare=5, slots=[2, -1, 2, 9, 0], num_slots=4)
    g, y0 = to_gpu(d), before(d)
    y = prompt(g, y0.cuda())
    torch.cuda.synchronize()
    compare(d, g, y, y0)
    assert bool((y[-5:] == 7).all()) and bool((y[70:144] == 0).all())


@pytest.mark.parametrize("cu", [[0, 500, 100], [-5, 30, 64], [90, 20, 10], [0, 0, 2 ** 31 - 1], [64, 64, 64]])
def test_offsets_outside_the_rows_stay_inside_the_tensors(cu):
    """What they compute is unspecified; guards around every tensor keep their values."""
    say(f"case delta offsets {cu}")
    d = delta_inputs([40, 24], 2, 64, 1, 64, seed=9)
    g = to_gpu(d)
    y = torch.full((64 + 128, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    st = torch.full((12, 2, 64, 64), 7.0, device="cuda")
    g["state_cache"], g["cu"] = st[4:8], torch.tensor(cu, dtype=torch.int32, device="cuda")
    prompt(g, y[64:128])
    torch.cuda.synchronize()
    assert (y[:64] == 7).all() and (y[128:] == 7).all() and (st[:4] == 7).all() and (st[8:] == 7).all()


@pytest.mark.parametrize("what", ["v", "k", "q", "dt", "beta"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), 3e38])
def test_values_that_are_not_finite_reach_no_earlier_token(what, value):
    """A value that is not finite (or whose squares are not) spoils its own token and
    those behind it, never one before it or another sequence."""
    say(f"case delta {what} {value}")
    d = delta_inputs([100, 90], 2, 64, 1, 64, seed=10)
    at = 75
    clean = to_gpu(d)
    yc = prompt(clean)
    bad = {k: (v.clone() if torch.is_tensor(v) else v) for k, v in d.items()}
    dict(zip(("q", "k", "v", "beta", "dt"), (parts(bad)[i] for i in (0, 1, 2, 4, 3))))[what][at, 1] = value
    g = to_gpu(bad)
    y = prompt(g)
    torch.cuda.synchronize()
    assert torch.isfinite(y[:at]).all() and torch.isfinite(y[100:]).all()
    assert torch.equal(y[:64], yc[:64]) and torch.equal(y[100:], yc[100:])
    assert (y[64:at].float() - yc[64:at].float()).abs().max() <= 2.0 ** -6 * yc[64:at].float().abs().max()
    if what == "v" and value != 3e38:
        assert not torch.isfinite(y[at:100].float()).all(), "a value that is not finite shows"


def test_resuming_continues_a_sequence():
    """One call over 200 tokens and calls over its pieces: the states agree as two
    orders of the same sums do."""
    say("case delta pieces")
    d = delta_inputs([200], 3, 64, 1, 128, seed=11, slots=[1])
    whole = to_gpu(d)
    yw = prompt(whole, resume=None)
    piece, ys, row = to_gpu(d), [], 0
    for n in (64, 1, 70, 3, 62):
        part = dict(piece, qkv=piece["qkv"][row:row + n], gates=piece["gates"][row:row + n],
                    cu=torch.tensor([0, n], dtype=torch.int32, device="cuda"))
        ys.append(prompt(part, resume=torch.tensor([1 if row else 0], dtype=torch.int32, device="cuda")))
        row += n
    torch.cuda.synchronize()
    _, _, yt, st = delta_reference(d, before(d), False, c=C, cy=2.0 ** -15)
    got = torch.cat(ys).cpu().double()
    assert ((whole["state_cache"] - piece["state_cache"]).cpu().double().abs() <= 2 * st).all()
    assert ((got - yw.cpu().double()).abs() <= 2 * yt + 2.0 ** -7 * got.abs()).all()


def test_slices_streams_and_equal_bits():
    """Rows further apart, a workspace larger than needed and full of NaN, another
    stream: the same bits."""
    say("case delta streams")
    d = delta_inputs([130, 300, 4], 4, 64, 2, 128, seed=12)
    g = to_gpu(d)
    y = prompt(g)
    h = to_gpu(d)
    wide = torch.zeros(h["qkv"].shape[0], h["qkv"].shape[1] + 72, dtype=torch.bfloat16, device="cuda")
    wide[:, 64:-8] = h["qkv"]
    h["qkv"] = wide[:, 64:-8]
    need = ssm.ssm_delta_fwd_cache_workspace_bytes(3, 434, 4, 64, 2, 128, ssm.SSM_BF16)
    ws = torch.full((need // 4 + 64,), float("nan"), device="cuda")
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    y2 = prompt(h, workspace=ws, stream=other)
    other.synchronize()
    assert torch.equal(y, y2) and torch.equal(g["state_cache"], h["state_cache"])


def test_captured_calls_take_new_lengths():
    """A captured call replayed over other offsets, slots and flags, with eager calls
    on another workspace between the replays."""
    say("case delta graph")
    lens = [[100, 30, 62], [0, 150, 42], [64, 64, 64], [192, 0, 0], [1, 1, 190]]
    ds = [delta_inputs(ls, 2, 64, 1, 128, seed=20 + i) for i, ls in enumerate(lens)]
    eager = [to_gpu(d) for d in ds]
    want = [prompt(g) for g in eager]
    live = to_gpu(ds[0])
    y = torch.zeros_like(want[0])
    ws = torch.empty(ssm.ssm_delta_fwd_cache_workspace_bytes(3, 192, 2, 64, 1, 128, ssm.SSM_BF16), dtype=torch.uint8, device="cuda")
    prompt(live, y, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        prompt(live, y, workspace=ws)
    for d, g, w in zip(ds, eager, want):
        for key in ("qkv", "gates", "cu", "slots", "resume", "A", "dt_bias", "state_cache"):
            live[key].copy_(d[key])
        graph.replay()
        prompt(to_gpu(d))
        torch.cuda.synchronize()
        assert torch.equal(y, w) and torch.equal(live["state_cache"], g["state_cache"])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("batch,H,P,G,N", [(1, 2, 64, 1, 128), (5, 3, 64, 3, 64), (3, 4, 128, 2, 128), (2, 2, 256, 1, 64), (300, 1, 64, 1, 64), (2, 5, 192, 1, 128)])
def test_tokens(batch, H, P, G, N, dtype):
    say(f"case delta tokens {batch} H={H} P={P} G={G} N={N} {dtype}")
    d = delta_inputs([1] * batch, H, P, G, N, seed=batch + H, dtype=dtype)
    d["resume"] = torch.ones(batch, dtype=torch.int32)
    g, y0 = to_gpu(d), before(d)
    y = step(g, y0.cuda())
    torch.cuda.synchronize()
    compare(d, g, y, y0, products=False)


def test_padding_rows_of_tokens():
    say("case delta padding")
    d = delta_inputs([1] * 6, 2, 64, 1, 128, seed=14, slots=[3, -1, 0, 3, 8, 2], num_slots=5)
    d["resume"] = torch.ones(6, dtype=torch.int32)
    g, y0 = to_gpu(d), before(d)
    y = step(g, y0.cuda())
    torch.cuda.synchronize()
    compare(d, g, y, y0, products=False)
    assert (y[[1, 3, 4]] == 0).all()


@pytest.mark.parametrize("kw,call", [(dict(dt_bias=False), {}), ({}, dict(scale=1.0, norm_eps=0.5)), (dict(scale=0.05), dict(norm_eps=-1.0)), (dict(A=(1e4, 1e5)), {})])
def test_tokens_of_other_kinds(kw, call):
    say(f"case delta tokens {kw} {call}")
    d = delta_inputs([1] * 4, 2, 64, 2, 64, seed=15, **kw)
    d["resume"] = torch.ones(4, dtype=torch.int32)
    g, y0 = to_gpu(d), before(d)
    y = step(g, y0.cuda(), **call)
    torch.cuda.synchronize()
    compare(d, g, y, y0, products=False, **call)


def test_tokens_continue_a_prompt():
    """A prompt, then its later tokens one at a time: the state and outputs of one
    longer prompt, up to the order of the sums."""
    say("case delta prompt then tokens")
    d = delta_inputs([80], 4, 64, 2, 128, seed=16, slots=[1])
    whole, g = to_gpu(d), to_gpu(d)
    yw = prompt(whole, resume=None)
    first = dict(g, qkv=g["qkv"][:70], gates=g["gates"][:70], cu=torch.tensor([0, 70], dtype=torch.int32, device="cuda"))
    ys = [prompt(first, resume=None)]
    for t in range(70, 80):
        ys.append(step(dict(g, qkv=g["qkv"][t:t + 1], gates=g["gates"][t:t + 1])))
    torch.cuda.synchronize()
    _, _, yt, st = delta_reference(d, before(d), False, c=C, cy=2.0 ** -15)
    got = torch.cat(ys).cpu().double()
    assert ((whole["state_cache"] - g["state_cache"]).cpu().double().abs() <= 2 * st).all()
    assert ((got - yw.cpu().double()).abs() <= 2 * yt + 2.0 ** -7 * got.abs()).all()


def test_captured_tokens():
    say("case delta tokens graph")
    d = delta_inputs([1] * 3, 2, 64, 1, 64, seed=17)
    g, live = to_gpu(d), to_gpu(d)
    y = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    step(dict(live, state_cache=live["state_cache"].clone()), y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(live, y)
    for _ in range(4):
        want = step(g)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(live["state_cache"], g["state_cache"])


def test_states_beyond_the_last_level_cache():
    """More state than the caches hold (512 MB), where it is streamed."""
    say("case delta tokens, large")
    d = delta_inputs([1] * 4, 2, 128, 1, 128, seed=18)
    batch, H, P, N = 128, 64, 128, 128
    gen = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    q, k, v, dt, be = (r(batch, n).bfloat16() for n in (N, N, H * P, H, H))
    A, st = -torch.rand(H, device="cuda") - 1, r(batch, H, P, N) * 0.3
    slots = torch.arange(batch, dtype=torch.int32, device="cuda")
    part = st[5:9].clone()
    y = ssm.ssm_delta_step_cache(q, k, v, dt, be, A, slots, st)
    y2 = ssm.ssm_delta_step_cache(q[5:9], k[5:9], v[5:9], dt[5:9], be[5:9], A, slots[:4], part)
    torch.cuda.synchronize()
    assert torch.equal(y[5:9], y2) and torch.equal(st[5:9], part)
    del d
