"""The gated delta rule over packed prompts by every kernel that a call may be given:
teams of waves on 16 columns of a state, and workgroups of four or eight waves of 16
columns each, for states of 64 and of 128 elements per column (needs MI355X). Which one
a call takes goes by its heads, columns and sequences: WAYS reaches each with few heads
and many sequences, nearly all of them empty. Error bounds as in test_delta_cache_gpu.py.
"""
import pytest
import torch

import selective_state_space_16_amd as ssm
from block_util import owned, to_gpu
from delta_util import delta_inputs, delta_reference, parts
from gpu_util import say
from test_delta_cache_gpu import C, before, prompt

pytestmark = pytest.mark.gpu
H, G = 2, 1
# (columns P, sequences): teams, walk of four waves, the same with three workgroups a head, walk of eight
WAYS = [(64, 8), (64, 90), (192, 40), (128, 90)]
ALL = [(P, seqs, N) for P, seqs in WAYS for N in (64, 128)]


def inputs(lens, P, seqs, N, *, seed, slots=(), spare=0, **kw):
    """`lens` among `seqs` sequences, spread over them, the others empty."""
    n = seqs // len(lens)
    full = [0] * seqs
    for i, v in enumerate(lens):
        full[i * n] = v
    d = delta_inputs(full, H, P, G, N, seed=seed, spare=spare, **kw)
    for i, v in enumerate(slots):
        if v is not None:
            d["slots"][i * n] = v
    d["at"] = [sum(full[:i * n]) for i in range(len(lens))]  # the first rows of the sequences that are not empty
    return d


def compare(d, g, y, y0, what="", **kw):
    """`y` and the cache against the definition, which says where they are not finite."""
    yr, st, yt, stol = delta_reference(d, y0, c=C, cy=2.0 ** -15, **kw)
    got, gs = y.cpu().double(), g["state_cache"].cpu().double()
    ok, oks = torch.isfinite(yr), torch.isfinite(st)
    ty = 2.0 ** -8 * yr.abs() + yt
    worst = lambda a, b, tol, m: float((((a - b).abs() / tol.clamp_min(1e-300))[m]).max()) if bool(m.any()) else 0.0  # noqa: E731
    say(f"  {what} y of bound {worst(got, yr, ty, ok):.2f}, state of bound {worst(gs, st, stol.expand(st.shape), oks):.2f}")
    assert torch.equal(torch.isfinite(got), ok) and torch.equal(torch.isfinite(gs), oks)
    assert ((got - yr).abs() <= ty)[ok].all(), "y"
    assert ((gs - st).abs() <= stol)[oks].all(), "state"
    mine = set(owned(d["slots"], st.shape[0]))
    for k in range(st.shape[0]):
        if k not in mine:
            assert torch.equal(g["state_cache"][k].cpu(), d["state_cache"][k]), "a slot of no sequence"


@pytest.mark.parametrize("P,seqs,N", ALL)
@pytest.mark.parametrize("at", [3, 63, 70])
def test_an_infinite_value_stays_in_its_column(P, seqs, N, at):
    """A value of one column that is not finite, in a chunk that others follow: every other
    column, of every token, is what the definition says."""
    say(f"case delta walks, infinite value at {at} P={P} N={N} sequences={seqs}")
    d = inputs([200, 70, 130], P, seqs, N, seed=at + N)
    for k, col in enumerate((17, P + 5)):  # of either head, of the first sequence and the last
        parts(d)[2][d["at"][2 * k] + at, col] = (float("inf"), float("nan"))[k]
    g, y0 = to_gpu(d), before(d)
    y = prompt(g, y0.cuda())
    torch.cuda.synchronize()
    compare(d, g, y, y0)


def cancelling(P, seqs, N):
    """Outputs that are small differences of large terms. The first sequence starts from
    nothing and takes tokens in threes: two whose keys are alone in their directions and
    whose updates are nearly alike, then a query of their difference with a key of zeros;
    the second resumes a state whose columns are nearly alike in pairs, under such queries
    alone. Everything that is summed up is positive."""
    d = inputs([96, 70], P, seqs, N, seed=P + N)
    g = torch.Generator().manual_seed(N)
    q, k, v, dt, be = parts(d)
    q.zero_(), k.zero_(), v.zero_()
    a = torch.exp(torch.logaddexp(dt.double() + d["dt_bias"].double(), torch.zeros(())) * d["A"].double())
    beta = torch.sigmoid(be.double())
    for i in range(32):
        t = d["at"][0] + 3 * i
        k[t, 2 * i], k[t + 1, 2 * i + 1] = (torch.rand(2, generator=g) + 0.5).bfloat16()
        v[t] = (torch.rand(H * P, generator=g) + 0.5).bfloat16()
        v[t + 1] = (v[t].double() * (beta[t] * a[t + 1] / beta[t + 1]).repeat_interleave(P)).bfloat16()
        q[t + 2, 2 * i], q[t + 2, 2 * i + 1] = 1, -1
    n = seqs // 2
    for t in range(70):
        i = 2 * int(torch.randint(N // 2, (1,), generator=g))
        q[d["at"][1] + t, i], q[d["at"][1] + t, i + 1] = 1, -1
    d["resume"][0], d["resume"][n] = 0, 1
    st = d["state_cache"][d["slots"][n]]
    st.abs_()
    st[..., 1::2] = st[..., ::2] * (1 + 2.0 ** -12 * torch.rand(H, P, N // 2, generator=g))
    return d


@pytest.mark.parametrize("P,seqs,N", ALL)
def test_outputs_are_products_of_float32_operands(P, seqs, N):
    """Where two terms nearly cancel, what each was rounded to before shows. In float32 a
    term takes at most 24 roundings: of beta 5, of u and its factors in T and M (two
    lengths, a decay with its exponent, their products) 11, the sum of two terms with what
    an operand of three parts leaves out 8; y is then rounded once to bfloat16."""
    say(f"case delta walks, cancelling terms P={P} N={N} sequences={seqs}")
    d = cancelling(P, seqs, N)
    g, y0 = to_gpu(d), before(d)
    y = prompt(g, y0.cuda())
    torch.cuda.synchronize()
    yr = delta_reference(d, y0)[0]
    big = dict(d, qkv=d["qkv"].clone())
    parts(big)[0].abs_()
    terms = delta_reference(big, y0)[0]
    err, tol = (y.cpu().double() - yr).abs(), 2.0 ** -8 * yr.abs() + 24 * 2.0 ** -24 * terms
    say(f"  of bound {float((err / tol.clamp_min(1e-300)).max()):.2f}, size of the terms {float((terms.sum() / yr.abs().sum())):.0f} times")
    assert (err <= tol).all()


@pytest.mark.parametrize("P,seqs,N", ALL)
def test_lengths_without_a_floor_under_them(P, seqs, N):
    """norm_eps = 0 is a floor too small to change any length here: the same bits, also of
    sequences that end inside a chunk, whose rows behind the last token have no length."""
    say(f"case delta walks, norm_eps = 0 P={P} N={N} sequences={seqs}")
    d = inputs([150, 1, 64, 37], P, seqs, N, seed=P + N + 1)
    g, h, y0 = to_gpu(d), to_gpu(d), before(d)
    y, z = prompt(g, y0.cuda(), norm_eps=0.0), prompt(h, y0.cuda(), norm_eps=1e-30)
    torch.cuda.synchronize()
    compare(d, g, y, y0, norm_eps=0.0)
    assert torch.equal(y, z) and torch.equal(g["state_cache"], h["state_cache"])


@pytest.mark.parametrize("P,seqs,N", ALL)
@pytest.mark.parametrize("lens", [[65], [64, 128, 192], [1, 63, 150, 2, 129], [700, 333]])
def test_against_the_definition(lens, P, seqs, N):
    say(f"case delta walks {lens} P={P} N={N} sequences={seqs}")
    d = inputs(lens, P, seqs, N, seed=sum(lens) + N, spare=3)
    g, y0 = to_gpu(d), before(d)
    y = prompt(g, y0.cuda())
    torch.cuda.synchronize()
    compare(d, g, y, y0)
    assert bool((y[-3:] == 7).all())


@pytest.mark.parametrize("P,seqs,N", ALL)
def test_left_out_sequences(P, seqs, N):
    """Slots out of range or of an earlier sequence, of sequences with tokens and without."""
    say(f"case delta walks, left out P={P} N={N} sequences={seqs}")
    d = inputs([70, 130, 66, 9], P, seqs, N, seed=N, slots=(None, -1, seqs + 2, None), spare=5)
    n = seqs // 4
    d["slots"][3 * n] = d["slots"][0]
    d["slots"][1] = -7
    g, y0 = to_gpu(d), before(d)
    y = prompt(g, y0.cuda())
    torch.cuda.synchronize()
    compare(d, g, y, y0)
    assert bool((y[70:-5] == 0).all()) and bool((y[-5:] == 7).all())


@pytest.mark.parametrize("P,seqs,N", ALL)
@pytest.mark.parametrize("kw,call", [(dict(scale=0.05), dict(norm_eps=-1.0)), (dict(same_keys=0.9), {}), (dict(same_keys=1.0), dict(scale=1.0)),
                                     (dict(step=(1.0, 30.0)), {}), (dict(A=(0.0, 0.0)), {}), (dict(A=(1e4, 1e5)), {}), (dict(dt_bias=False), {})])
def test_other_kinds(kw, call, P, seqs, N):
    say(f"case delta walks {kw} {call} P={P} N={N} sequences={seqs}")
    d = inputs([150, 20, 64], P, seqs, N, seed=6, **kw)
    g, y0 = to_gpu(d), before(d)
    y = prompt(g, y0.cuda(), **call)
    torch.cuda.synchronize()
    compare(d, g, y, y0, **call)


@pytest.mark.parametrize("P,seqs,N", ALL)
@pytest.mark.parametrize("what", ["k", "q", "dt", "beta"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_values_that_are_not_finite(what, value, P, seqs, N):
    """What the definition makes of them, in the last chunk and in one that others follow:
    keys spoil their group from their token on, queries one token, a step or gate of
    infinity a head's token or nothing."""
    say(f"case delta walks, {what} {value} P={P} N={N} sequences={seqs}")
    d = inputs([200, 90, 70], P, seqs, N, seed=N + 2)
    q, k, _, dt, be = parts(d)
    for at in (d["at"][0] + 70, d["at"][1] + 75):
        dict(q=q, k=k, dt=dt, beta=be)[what][at, 1] = value
    g, y0 = to_gpu(d), before(d)
    y = prompt(g, y0.cuda())
    torch.cuda.synchronize()
    compare(d, g, y, y0)


@pytest.mark.parametrize("P,seqs,N", ALL)
def test_offsets_outside_the_rows_stay_inside_the_tensors(P, seqs, N):
    """What they compute is unspecified; guards around every tensor keep their values."""
    say(f"case delta walks, offsets P={P} N={N} sequences={seqs}")
    gen = torch.Generator().manual_seed(seqs)
    for kind in range(4):
        d = inputs([40, 88], P, seqs, N, seed=9)
        cu = torch.randint(-200, 400, (seqs + 1,), generator=gen, dtype=torch.int32)
        if kind == 1:
            cu = cu.sort().values
        elif kind == 2:
            cu = cu.sort(descending=True).values
        elif kind == 3:
            cu[::2], cu[1::2] = 2 ** 31 - 1, -2 ** 31
        g = to_gpu(d)
        y = torch.full((128 + 128, H, P), 7.0, dtype=torch.bfloat16, device="cuda")
        st = torch.full((seqs + 8, H, P, N), 7.0, device="cuda")
        g["state_cache"], g["cu"] = st[4:seqs + 4], cu.cuda()
        prompt(g, y[64:192])
        torch.cuda.synchronize()
        assert (y[:64] == 7).all() and (y[192:] == 7).all() and (st[:4] == 7).all() and (st[seqs + 4:] == 7).all()


@pytest.mark.parametrize("P,seqs,N", ALL)
def test_slices_streams_and_equal_bits(P, seqs, N):
    say(f"case delta walks, streams P={P} N={N} sequences={seqs}")
    d = inputs([130, 300, 4], P, seqs, N, seed=12)
    g, h = to_gpu(d), to_gpu(d)
    y = prompt(g)
    rows = h["qkv"].shape[0]
    wide = torch.zeros(rows, h["qkv"].shape[1] + 72, dtype=torch.bfloat16, device="cuda")
    wide[:, 64:-8] = h["qkv"]
    h["qkv"] = wide[:, 64:-8]
    need = ssm.ssm_delta_fwd_cache_workspace_bytes(seqs, rows, H, P, G, N, ssm.SSM_BF16)
    ws = torch.full((need // 4 + 64,), float("nan"), device="cuda")
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    z = prompt(h, workspace=ws, stream=other)
    other.synchronize()
    assert torch.equal(y, z) and torch.equal(g["state_cache"], h["state_cache"])


@pytest.mark.parametrize("P,seqs,N", ALL)
def test_captured_calls_take_new_lengths(P, seqs, N):
    say(f"case delta walks, graph P={P} N={N} sequences={seqs}")
    lens = [[100, 30, 62], [0, 150, 42], [192, 0, 0], [1, 1, 190]]
    ds = [inputs(ls, P, seqs, N, seed=20 + i) for i, ls in enumerate(lens)]
    eager = [to_gpu(d) for d in ds]
    want = [prompt(g) for g in eager]
    live = to_gpu(ds[0])
    y = torch.zeros_like(want[0])
    ws = torch.empty(ssm.ssm_delta_fwd_cache_workspace_bytes(seqs, 192, H, P, G, N, ssm.SSM_BF16), dtype=torch.uint8, device="cuda")
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


@pytest.mark.parametrize("P,seqs,N", ALL)
def test_two_calls_at_once(P, seqs, N):
    """Two streams, a workspace and a cache each: the bits of the calls one after the other."""
    say(f"case delta walks, two calls P={P} N={N} sequences={seqs}")
    ds = [inputs([300, 129, 64], P, seqs, N, seed=30 + i) for i in range(2)]
    alone, both = [to_gpu(d) for d in ds], [to_gpu(d) for d in ds]
    want = [prompt(g) for g in alone]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ds]
    got = [prompt(g, stream=s) for g, s in zip(both, streams)]
    torch.cuda.synchronize()
    for a, b, u, v in zip(alone, both, want, got):
        assert torch.equal(u, v) and torch.equal(a["state_cache"], b["state_cache"])
