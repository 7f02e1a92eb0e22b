"""The SSD layer on a cache of states, over packed prompts (ssm_ssd_fwd_cache)
and over single tokens (ssm_ssd_step_cache), against the plain 64-bit
definition (needs MI355X).

Error bounds, against sums of absolute terms (`y_abs`, `st_abs`: the same
recurrence over |terms|, the convolution's included):
- y is rounded to its type once: half a step, 2^-8 (bfloat16) or 2^-24
  (float32) of its value. The prompt operator's products for y take operands
  of 11 significant bits: C, B, their product, its decayed form, x and the
  state copy are each rounded at most once, and a state that has been updated
  with rounded operands is rounded twice more; at most 8 roundings of 2^-11
  relative to the absolute terms.
- the state is float32 throughout: operands of 22 significant bits, and per
  term about 32 float32 roundings (convolution, SiLU, softplus, decay) and 3 per
  token that it is carried through: its decay exp2 is off by at most one unit in
  the last place (2 roundings) and the sum adds one; a term carried over n tokens
  whose decays are near one keeps all of them, 3 n 2^-24. A decay exp(c) with c
  summed in float32 has a relative error of 2^-24 |c| per rounding of c, and the
  term it multiplies shrinks by exp(c): |c| exp(-|c|) < 1/2.
"""
import pytest
import torch

import selective_state_space_16_amd as ssm
from block_util import owned, ssd_inputs, ssd_reference, to_gpu, views
from gpu_util import say

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def prompt(g, y, **kw):
    xBC, dt = views(g)
    kw = {"resume": g["resume"], **kw}
    return ssm.ssm_ssd_fwd_cache(xBC, dt, g["A"], g["conv_w"], g["cu"], g["slots"], g["conv_cache"], g["state_cache"],
                                 conv_b=g["conv_b"], dt_bias=g["dt_bias"], Dskip=g["Dskip"], y=y, **kw)


def step(g, y=None, **kw):
    xBC, dt = views(g)
    return ssm.ssm_ssd_step_cache(xBC, dt, g["A"], g["conv_w"], g["slots"], g["conv_cache"], g["state_cache"],
                                  conv_b=g["conv_b"], dt_bias=g["dt_bias"], Dskip=g["Dskip"], y=y, **kw)


def before(d):
    rows = d["proj"].shape[0]
    return torch.full((rows, d["H"], d["P"]), 7.0, dtype=d["proj"].dtype)


def compare(d, g, y, y0, what=None, resume=True, products=True):
    """`y` and the caches in `g` against the definition on the inputs `d`."""
    yr, st, win, ya, sa = ssd_reference(d, y0, resume)
    got, gs = y.cpu().double(), g["state_cache"].cpu().double()
    half = 2.0 ** -8 if d["proj"].dtype == torch.bfloat16 else 2.0 ** -24
    carried = 3 * max(d["lens"], default=0)
    tol_s = (32 + carried) * U * sa
    tol_y = half * yr.abs() + (8 * 2.0 ** -11 if products else (40 + carried) * U) * ya
    ey, es = ((got - yr).abs() - tol_y).max(), ((gs - st).abs() - tol_s).max()
    rel = lambda a, b: float((a - b).norm() / b.norm().clamp_min(1e-300))  # noqa: E731
    say(f"  {what or ''} y relL2={rel(got, yr):.2e} worst of bound {float(((got - yr).abs() / tol_y.clamp_min(1e-300)).max()):.2f}, "
        f"state relL2={rel(gs, st):.2e} worst of bound {float(((gs - st).abs() / tol_s.clamp_min(1e-300)).max()):.2f}")
    assert torch.isfinite(got).all() and torch.isfinite(gs).all()
    assert ey <= 0, "y"
    assert es <= 0, "state"
    assert torch.equal(g["conv_cache"].cpu().double(), win), "window"
    # slots that no sequence owns keep their bits
    mine = set(owned(d["slots"], st.shape[0]))
    for k in range(st.shape[0]):
        if k not in mine:
            assert torch.equal(g["state_cache"][k].cpu(), d["state_cache"][k])


CASES = [
    ([1], 2, 64, 1, 128), ([37], 3, 64, 1, 128), ([64], 2, 64, 1, 64), ([65], 2, 64, 2, 128),
    ([0, 1, 2, 3, 4, 5], 4, 64, 2, 64), ([63, 64, 65, 127, 128, 129], 4, 64, 1, 128),
    ([300, 0, 5], 6, 64, 2, 128), ([1] * 70, 1, 64, 1, 64), ([200, 33], 2, 128, 1, 64), ([90], 3, 192, 3, 64),
    ([130, 7], 2, 256, 2, 128), ([0], 2, 64, 1, 128), ([0, 0, 9], 5, 64, 5, 64), ([2500], 2, 64, 1, 128),
    ([1300, 40, 2050], 2, 64, 1, 64), ([700], 9, 64, 1, 128),
]


@pytest.mark.parametrize("lens,H,P,G,N", CASES)
def test_prompts(lens, H, P, G, N):
    say(f"case prompts {lens[:6]} x{len(lens)} H={H} P={P} G={G} N={N}")
    d = ssd_inputs(lens, H, P, G, N, seed=sum(lens) + H, spare=3)
    g, y0 = to_gpu(d), before(d)
    y = prompt(g, y0.cuda())
    torch.cuda.synchronize()
    compare(d, g, y, y0)


@pytest.mark.parametrize("drop", ["conv_b", "dt_bias", "dskip"])
def test_optional_inputs(drop):
    say(f"case without {drop}")
    d = ssd_inputs([70, 3], 2, 64, 1, 128, seed=5, **{drop: False})
    g, y0 = to_gpu(d), before(d)
    y = prompt(g, y0.cuda(), resume=None)
    torch.cuda.synchronize()
    compare(d, g, y, y0, resume=False)


@pytest.mark.parametrize("scale", [1e-3, 30.0, 3e4])
def test_magnitudes(scale):
    """Inputs far from one: the products' operands are scaled by what they hold."""
    say(f"case magnitudes {scale}")
    d = ssd_inputs([150, 20], 2, 64, 1, 128, seed=6, scale=scale)
    g, y0 = to_gpu(d), before(d)
    y = prompt(g, y0.cuda())
    torch.cuda.synchronize()
    compare(d, g, y, y0)


@pytest.mark.parametrize("step_range", [(1e-6, 1e-5), (1.0, 30.0), (1e-4, 8.0)])
def test_decays(step_range):
    """Steps so small that nothing decays and so large that a token forgets all."""
    say(f"case decays {step_range}")
    d = ssd_inputs([400, 65], 4, 64, 2, 64, seed=7, step=step_range)
    g, y0 = to_gpu(d), before(d)
    y = prompt(g, y0.cuda())
    torch.cuda.synchronize()
    compare(d, g, y, y0)


def test_uneven_tokens():
    """Tokens a thousand times larger and smaller than their neighbours."""
    d = ssd_inputs([200], 2, 64, 1, 128, seed=8)
    f = torch.exp2(torch.randint(-10, 11, (200,), generator=torch.Generator().manual_seed(3)).float())
    d["proj"][:, 64:64 + d["C"]] = (d["proj"][:, 64:64 + d["C"]].float() * f[:, None]).bfloat16()
    say("case uneven tokens")
    g, y0 = to_gpu(d), before(d)
    y = prompt(g, y0.cuda())
    torch.cuda.synchronize()
    compare(d, g, y, y0)


def test_left_out_sequences():
    """Slots out of range and slots named twice: zeros, and no cache entry touched."""
    say("case left out")
    d = ssd_inputs([20, 70, 0, 33, 5], 2, 64, 1, 64, seed=9, slots=[2, -1, 7, 2, 4], num_slots=5, spare=2)
    g, y0 = to_gpu(d), before(d)
    y = prompt(g, y0.cuda())
    torch.cuda.synchronize()
    compare(d, g, y, y0)


def test_offsets_out_of_range_stay_inside():
    """Offsets behind the rows, negative or decreasing: the rows of y that no
    valid range covers and the tensors around stay as they were."""
    say("case bad offsets")
    d = ssd_inputs([40, 40], 2, 64, 1, 64, seed=10)
    g = to_gpu(d)
    for bad in ([0, 40, 1000], [-5, 40, 80], [0, 60, 30], [2 ** 31 - 1, -2 ** 31, 50]):
        g["cu"] = torch.tensor(bad, dtype=torch.int32, device="cuda")
        prompt(g, torch.zeros(80, 2, 64, dtype=torch.bfloat16, device="cuda"))
        torch.cuda.synchronize()
    free = [k for k in range(4) if k not in d["slots"].tolist()]
    assert torch.equal(g["state_cache"][free].cpu(), d["state_cache"][free])


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_nonfinite_stays_where_it_belongs(value):
    """A NaN or infinity in one token's x reaches that channel from that token on
    and nothing else: not the tokens before it, not other channels, not the
    sequences around it."""
    say(f"case {value}")
    d = ssd_inputs([50, 100, 30], 2, 64, 1, 128, seed=11)
    y0 = before(d)
    ref = prompt(to_gpu(d), y0.cuda()).cpu()
    d2 = dict(d, proj=d["proj"].clone())
    d2["proj"][50 + 40, 64 + 64 + 5] = value  # sequence 1, token 40, head 1, channel 5
    g = to_gpu(d2)
    y = prompt(g, y0.cuda()).cpu()
    torch.cuda.synchronize()
    assert torch.equal(y[:90], ref[:90]) and torch.equal(y[150:], ref[150:])
    others = torch.ones(2, 64, dtype=torch.bool)
    others[1, 5] = False
    assert torch.isfinite(y[90:150][:, others]).all()
    assert torch.equal(y[90:150, 0], ref[90:150, 0])
    assert not torch.isfinite(y[94:150, 1, 5]).any()
    slot = int(d["slots"][1])
    assert not torch.isfinite(g["state_cache"][slot, 1, 5]).any()
    assert torch.isfinite(g["state_cache"][slot, 0]).all() and torch.isfinite(g["state_cache"][slot, 1, :5]).all()


def test_nonfinite_cache_of_a_new_sequence():
    """A sequence that does not resume takes nothing from its slot."""
    say("case stale slot")
    d = ssd_inputs([70, 0], 2, 64, 1, 64, seed=12)
    g, y0 = to_gpu(d), before(d)
    g["state_cache"].fill_(float("nan"))
    g["conv_cache"].fill_(float("nan"))
    y = prompt(g, y0.cuda(), resume=None)
    torch.cuda.synchronize()
    z = dict(d, state_cache=torch.zeros_like(d["state_cache"]), conv_cache=torch.zeros_like(d["conv_cache"]))
    yr, st, win, ya, sa = ssd_reference(z, y0, False)
    assert ((y.cpu().double() - yr).abs() <= 2.0 ** -8 * yr.abs() + 8 * 2.0 ** -11 * ya).all()
    for s in d["slots"].tolist():
        assert ((g["state_cache"][s].cpu().double() - st[s]).abs() <= (32 + 3 * 70) * U * sa[s]).all()
        assert torch.equal(g["conv_cache"][s].cpu().double(), win[s])


def test_infinite_values_behind_a_sequence_and_spare_rows():
    """Rows behind the last sequence may hold anything and are left alone."""
    say("case spare rows")
    d = ssd_inputs([30, 34], 2, 64, 1, 64, seed=13, spare=70)
    clean = prompt(to_gpu(d), before(d).cuda()).cpu()
    d["proj"][64:] = float("nan")
    g, y0 = to_gpu(d), before(d)
    y = prompt(g, y0.cuda()).cpu()
    torch.cuda.synchronize()
    assert torch.equal(y, clean) and torch.equal(y[64:], y0[64:])
    assert torch.isfinite(g["state_cache"]).all()


def test_pieces_equal_the_whole():
    """A prompt cut in three calls that resume, and the tail token by token,
    against the definition over the whole."""
    say("case pieces")
    n, cuts = 330, [0, 1, 130, 321]
    d = ssd_inputs([n], 2, 64, 1, 128, seed=14, num_slots=2)
    d["resume"] = torch.zeros(1, dtype=torch.int32)
    g, y0 = to_gpu(d), before(d)
    y = torch.zeros(n, 2, 64, dtype=torch.bfloat16, device="cuda")
    for k in range(3):
        lo, hi = cuts[k], cuts[k + 1]
        part = dict(g, proj=g["proj"][lo:hi], cu=torch.tensor([0, hi - lo], dtype=torch.int32, device="cuda"))
        y[lo:hi] = prompt(part, None, resume=torch.tensor([int(k > 0)], dtype=torch.int32, device="cuda"))
    for t in range(321, n):
        y[t:t + 1] = step(dict(g, proj=g["proj"][t:t + 1]))
    torch.cuda.synchronize()
    compare(d, g, y, y0)


@pytest.mark.parametrize("lens,H,P,G,N", [([300, 1, 90], 4, 64, 2, 128), ([2500, 200], 2, 64, 1, 64)])
def test_equal_inputs_give_equal_bits(lens, H, P, G, N):
    say(f"case bits {lens}")
    d = ssd_inputs(lens, H, P, G, N, seed=15)
    outs = []
    for _ in range(3):
        g = to_gpu(d)
        y = prompt(g, before(d).cuda())
        outs.append((y, g["state_cache"], g["conv_cache"]))
    torch.cuda.synchronize()
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))


def test_graph_replay_with_other_lengths():
    """A captured call replayed with other offsets, slots and flags, eager calls
    of other sizes between, equals the eager call bit for bit."""
    say("case graph")
    d = ssd_inputs([150, 20, 30], 4, 64, 2, 128, seed=16)
    other = to_gpu(ssd_inputs([90, 500], 2, 64, 1, 64, seed=17))
    g = to_gpu(d)
    y = torch.zeros(200, 4, 64, dtype=torch.bfloat16, device="cuda")
    need = ssm.ssm_ssd_fwd_cache_workspace_bytes(3, 200, 4, 64, 2, 128, ssm.SSM_BF16)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    prompt(g, y, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        prompt(g, y, workspace=ws, stream=torch.cuda.current_stream())
    for rep, (cu, sl, rs) in enumerate([([0, 150, 170, 200], [0, 1, 2], [1, 0, 1]), ([0, 0, 1, 200], [3, 4, 0], [0, 1, 1]),
                                        ([0, 64, 128, 140], [1, -1, 3], [1, 1, 0]), ([0, 150, 170, 200], [0, 1, 2], [0, 0, 0])]):
        for k, v in (("cu", cu), ("slots", sl), ("resume", rs)):
            g[k].copy_(torch.tensor(v, dtype=torch.int32))
        e = {k: (v.clone() if torch.is_tensor(v) else v) for k, v in g.items()}
        y.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        ye = prompt(e, torch.full_like(y, 3))
        prompt(other, None)
        torch.cuda.synchronize()
        assert torch.equal(y, ye) and torch.equal(g["state_cache"], e["state_cache"]) and torch.equal(
            g["conv_cache"], e["conv_cache"]), f"replay {rep}"


def test_two_streams():
    """Two calls on streams of their own, each with its workspace."""
    say("case streams")
    ds = [ssd_inputs([400, 30], 2, 64, 1, 128, seed=18 + k) for k in range(2)]
    gs = [to_gpu(d) for d in ds]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ds]
    ys = [prompt(g, before(d).cuda(), stream=s) for g, d, s in zip(gs, ds, streams)]
    torch.cuda.synchronize()
    for d, g, y in zip(ds, gs, ys):
        compare(d, g, y, before(d))


STEPS = [(1, 2, 64, 1, 128), (5, 4, 64, 2, 64), (3, 3, 128, 3, 128), (70, 1, 64, 1, 64), (2, 2, 256, 1, 64)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("batch,H,P,G,N", STEPS)
def test_steps(batch, H, P, G, N, dtype):
    """Three tokens, one call each, against the definition over sequences of one
    token that resume."""
    say(f"case step batch={batch} H={H} P={P} G={G} N={N} {dtype}")
    d = ssd_inputs([1] * batch, H, P, G, N, seed=batch + H, dtype=dtype)
    d["resume"] = torch.ones(batch, dtype=torch.int32)
    g = to_gpu(d)
    for k in range(3):
        d = dict(d, proj=torch.roll(d["proj"], k, 0))
        g["proj"] = d["proj"].cuda()
        d["state_cache"], d["conv_cache"] = g["state_cache"].cpu(), g["conv_cache"].cpu()
        y = step(g)
        torch.cuda.synchronize()
        compare(d, g, y, before(d), products=False)


def test_step_padding_rows():
    say("case step padding")
    d = ssd_inputs([1] * 6, 2, 64, 1, 64, seed=21, slots=[3, -1, 0, 3, 9, 1], num_slots=5)
    d["resume"] = torch.ones(6, dtype=torch.int32)
    g = to_gpu(d)
    y = step(g, before(d).cuda())
    torch.cuda.synchronize()
    compare(d, g, y, before(d), products=False)
    assert not y[1].any() and not y[3].any() and not y[4].any()


def test_step_graph_replay():
    say("case step graph")
    d = ssd_inputs([1] * 9, 4, 64, 2, 128, seed=22)
    g = to_gpu(d)
    ws = torch.empty(ssm.ssm_ssd_step_cache_workspace_bytes(9, 4, 64, 2, 128), dtype=torch.uint8, device="cuda")
    y = torch.zeros(9, 4, 64, dtype=torch.bfloat16, device="cuda")
    step(g, y, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(g, y, workspace=ws, stream=torch.cuda.current_stream())
    for rep in range(4):
        g["slots"].copy_(torch.randperm(11)[:9].to(torch.int32) - int(rep == 2))
        e = {k: (v.clone() if torch.is_tensor(v) else v) for k, v in g.items()}
        graph.replay()
        ye = step(e)
        torch.cuda.synchronize()
        assert torch.equal(y, ye) and torch.equal(g["state_cache"], e["state_cache"]) and torch.equal(
            g["conv_cache"], e["conv_cache"]), f"replay {rep}"


def test_large_cache_offsets():
    """A slot whose state lies more than 2^32 bytes into the cache."""
    say("case large cache")
    H, P, G, N, slots = 80, 64, 1, 128, 1700  # 4.46 GB of states
    d = ssd_inputs([70], 2, P, G, N, seed=23, num_slots=2)
    C = H * P + 2 * G * N
    gen = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    st = torch.zeros(slots, H, P, N, device="cuda")
    win = torch.zeros(slots, C, 3, dtype=torch.bfloat16, device="cuda")
    xBC, dt = rnd(70, C).bfloat16(), rnd(70, H).bfloat16()
    w, A = rnd(C, 4) * 0.3, -torch.rand(H, generator=gen, device="cuda") - 0.1
    low = torch.tensor([0], dtype=torch.int32, device="cuda")
    high = torch.tensor([slots - 1], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 70], dtype=torch.int32, device="cuda")
    ys = [ssm.ssm_ssd_fwd_cache(xBC, dt, A, w, cu, s, win, st) for s in (low, high)]
    zs = [ssm.ssm_ssd_step_cache(xBC[:1], dt[:1], A, w, s, win, st) for s in (low, high)]
    torch.cuda.synchronize()
    assert torch.equal(ys[0], ys[1]) and torch.equal(zs[0], zs[1]) and ys[0].abs().max() > 0
    assert torch.equal(st[0], st[-1]) and torch.equal(win[0], win[-1]) and not st[1:-1].any()
    del d


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("where", ["B", "C", "dt"])
def test_nonfinite_shared_inputs(where, value):
    """A NaN or infinity in one token's B, C or step size: the tokens before it,
    the sequences around it and the heads that do not read it keep their bits;
    its own y is not finite, and neither is the state that takes it up."""
    say(f"case {where} {value}")
    d = ssd_inputs([50, 100, 30], 2, 64, 2, 128, seed=21)
    y0 = before(d)
    g0 = to_gpu(d)
    ref = prompt(g0, y0.cuda()).cpu()
    d2 = dict(d, proj=d["proj"].clone())
    col = {"B": 64 + 128 + 128 + 9, "C": 64 + 128 + 256 + 128 + 9, "dt": 64 + d["C"] + 1}[where]  # of group (head) 1
    d2["proj"][50 + 40, col] = value  # sequence 1, token 40
    g = to_gpu(d2)
    y = prompt(g, y0.cuda()).cpu()
    torch.cuda.synchronize()
    assert torch.equal(y[:90], ref[:90]) and torch.equal(y[150:], ref[150:]) and torch.equal(y[:, 0], ref[:, 0])
    slot = int(d["slots"][1])
    if where == "C":  # three tokens more, through the convolution
        assert not torch.isfinite(y[90:94, 1]).any() and torch.isfinite(y[94:]).all()
        assert torch.equal(g["state_cache"].cpu(), g0["state_cache"].cpu())
    elif where == "B":  # state column 9 of the head
        assert not torch.isfinite(y[90:150, 1]).any()
        assert not torch.isfinite(g["state_cache"][slot, 1, :, 9]).any()
    else:
        assert not torch.isfinite(y[90:150, 1]).any() and not torch.isfinite(g["state_cache"][slot, 1]).any()
    assert torch.equal(g["state_cache"][slot, 0].cpu(), g0["state_cache"][slot, 0].cpu())


def test_steps_that_forget_everything():
    """Steps of 50 to 2000, whose summed decays have no bits left for a token's
    own: a decay below 2^-256 leaves nothing of any float32 state, so summed
    exponents of at most 2^14 are exact to 2^-10, one and a half of the eight
    roundings of 2^-11 (the diagonal has six more). So tight a bound takes the
    terms as they are behind the SiLU, (C . B) dt x + D x, and 32 float32
    roundings of the convolution's absolute terms ahead of it."""
    say("case forgetting steps")
    d = ssd_inputs([200, 65], 4, 64, 2, 128, seed=22, step=(50.0, 2000.0))
    g, y0 = to_gpu(d), before(d)
    y = prompt(g, y0.cuda())
    torch.cuda.synchronize()
    compare(d, g, y, y0)
    yr, _, _, ya, _ = ssd_reference(d, y0)
    raw, dt = (t.double() for t in views(d))
    u = sum(raw[j:j + 197] * d["conv_w"][:, j].double() for j in range(4)) + d["conv_b"].double()  # tokens 3 .. of the first
    v = u * torch.sigmoid(u)
    x, B, Cm = v[:, :256].view(-1, 4, 64), v[:, 256:512].view(-1, 2, 128), v[:, 512:].view(-1, 2, 128)
    cb = (Cm * B).abs().sum(2).repeat_interleave(2, 1)[:, :, None]
    step_size = torch.nn.functional.softplus(dt[3:200] + d["dt_bias"].double())[:, :, None]
    terms = (cb * step_size + d["Dskip"].double()[:, None]) * x.abs()
    err = (y[3:200].cpu().double() - yr[3:200]).abs()
    tol = 2.0 ** -8 * yr[3:200].abs() + 8 * 2.0 ** -11 * terms + 32 * U * ya[3:200]
    say(f"  worst of the tight bound {float((err / tol).max()):.2f}")
    assert (err <= tol).all()


def test_no_tokens_keep_the_slot():
    """A resumed sequence of no tokens leaves its slot's bits, whatever it holds."""
    say("case no tokens")
    d = ssd_inputs([0, 5], 2, 64, 1, 64, seed=23)
    d["resume"][:] = 1
    s = int(d["slots"][0])
    d["state_cache"][s, 0, 0, :4] = torch.tensor([1e-40, 1e30, float("nan"), -3e-39])
    g, y0 = to_gpu(d), before(d)
    prompt(g, y0.cuda())
    torch.cuda.synchronize()
    assert torch.equal(g["state_cache"][s].cpu().view(torch.int32), d["state_cache"][s].view(torch.int32))
    assert torch.equal(g["conv_cache"][s].cpu().view(torch.int16), d["conv_cache"][s].view(torch.int16))


@pytest.mark.parametrize("batch,N,dtype", [(161, 128, torch.bfloat16), (322, 64, torch.float32)])
def test_steps_on_more_state_than_the_caches_hold(batch, N, dtype):
    """A batch whose states pass through the caches equals its halves, whose stay."""
    say(f"case step streamed batch={batch} N={N} {dtype}")
    gen = torch.Generator(device="cuda").manual_seed(24)
    H, P, G = 80, 64, 2
    C, half = H * P + 2 * G * N, batch // 2
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x, dt = rnd(batch, C).to(dtype), rnd(batch, H).to(dtype)
    conv, state = rnd(batch, C, 3).to(dtype), rnd(batch, H, P, N)
    slots = torch.randperm(batch, generator=gen, device="cuda").to(torch.int32)
    A, w = -torch.rand(H, generator=gen, device="cuda") - 0.5, rnd(C, 4) * 0.3
    conv2, state2 = conv.clone(), state.clone()
    y = ssm.ssm_ssd_step_cache(x, dt, A, w, slots, conv, state)
    parts = [ssm.ssm_ssd_step_cache(x[k].contiguous(), dt[k].contiguous(), A, w, slots[k].clone(), conv2, state2)
             for k in (slice(0, half), slice(half, batch))]
    torch.cuda.synchronize()
    assert torch.equal(y, torch.cat(parts)) and torch.equal(conv, conv2) and torch.equal(state, state2)


def test_overlapping_offsets_stay_inside():
    """Offsets that go back take more segments than the workspace is for: the
    caches' other slots and what lies behind the workspace keep their bits."""
    say("case overlapping offsets")
    d = ssd_inputs([100, 100, 0, 0, 0, 0, 0, 0, 0], 2, 64, 1, 64, seed=25)
    g = to_gpu(d)
    g["cu"] = torch.tensor([0, 200, 0, 200, 0, 200, 0, 200, 0, 200], dtype=torch.int32, device="cuda")
    need = ssm.ssm_ssd_fwd_cache_workspace_bytes(9, 200, 2, 64, 1, 64, ssm.SSM_BF16)
    ws = torch.full((need + 65536,), 77, dtype=torch.uint8, device="cuda")
    xBC, dt = views(g)
    prompt(g, torch.zeros(200, 2, 64, dtype=torch.bfloat16, device="cuda"), workspace=ws[:need])
    torch.cuda.synchronize()
    assert (ws[need:] == 77).all()
    free = [k for k in range(11) if k not in d["slots"].tolist()]
    assert torch.equal(g["state_cache"][free].cpu(), d["state_cache"][free])
