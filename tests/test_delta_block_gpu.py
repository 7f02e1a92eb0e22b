"""A gated delta block run as it would be used: residual sum and layer norm, a
projection, the convolution on its cache, the gated delta rule on its cache, the gate
norm behind it; over packed prompts and then over single tokens, eager and captured
(needs MI355X).

The block's outputs are compared with the same block in 64 bits whose intermediate
results are rounded to bfloat16 where the block's are. Each of the five roundings in a
row moves a value by at most 2^-8 of it, and where two roundings differ because the value
before was near a border, by twice that: in the 2-norm of a whole output the operators'
own errors stay below the root of five of them, each 2^-8 / sqrt(3) at most, and a border
is crossed on either side as often, which doubles it: 2 sqrt(5) 2^-8 / sqrt(3) < 1.1e-2.
"""
import torch
import pytest

import selective_state_space_16_amd as ssm
from block_util import F8, gate_norm_reference
from delta_util import conv_reference, delta_reference, layer_norm_reference
from gpu_util import say

pytestmark = pytest.mark.gpu
bf = torch.bfloat16
D, H, P, G, N = 256, 4, 64, 2, 64
C = 2 * G * N + H * P


def weights(seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return dict(ln_w=1 + 0.1 * r(D), ln_b=0.1 * r(D), proj=(r(D, C + 2 * H + H * P) * D ** -0.5).to(bf), conv_w=torch.rand(C, 4, generator=g) - 0.5,
                conv_b=0.1 * r(C), A=-torch.rand(H, generator=g) * 8 - 1, dt_bias=r(H) - 3, gate_w=1 + 0.1 * r(H * P))


def block(w, x, res, cu, slots, resume, conv, state):
    """One call over packed prompts, or one token per request (cu None)."""
    y, res = ssm.ssm_add_layer_norm_fwd(x, w["ln_w"], w["ln_b"], residual=res)
    row = y @ w["proj"]
    z, gates = row[:, C + 2 * H:], row[:, C:C + 2 * H]
    qkv, dt, be = row[:, :C], gates[:, :H], gates[:, H:]
    if cu is None:
        u = ssm.ssm_conv_step_cache(qkv, w["conv_w"], slots, conv, conv_b=w["conv_b"])
        o = ssm.ssm_delta_step_cache(u[:, :G * N], u[:, G * N:2 * G * N], u[:, 2 * G * N:], dt, be, w["A"], slots, state, dt_bias=w["dt_bias"])
    else:
        u = ssm.ssm_conv_fwd_cache(qkv, w["conv_w"], cu, slots, conv, conv_b=w["conv_b"], resume=resume)
        o = ssm.ssm_delta_fwd_cache(u[:, :G * N], u[:, G * N:2 * G * N], u[:, 2 * G * N:], dt, be, w["A"], cu, slots, state, dt_bias=w["dt_bias"], resume=resume)
    return ssm.ssm_gate_norm_fwd(o.reshape(-1, H * P), z, w["gate_w"]), res


def reference(w, x, res, lens, slots, resume, conv, state):
    y, r = layer_norm_reference(x, res, None, w["ln_w"], w["ln_b"], 1e-5)
    row = (y.to(bf).to(F8) @ w["proj"].to(F8)).to(bf)
    u, conv, _ = conv_reference(row[:, :C], w["conv_w"], w["conv_b"], lens, slots, resume, conv, torch.zeros(x.shape[0], C))
    d = dict(H=H, P=P, G=G, N=N, lens=lens, qkv=u.to(bf), gates=row[:, C:C + 2 * H], slots=slots, resume=resume, dt_bias=w["dt_bias"], A=w["A"],
             state_cache=state)
    o, state, _, _ = delta_reference(d, torch.zeros(x.shape[0], H, P))
    return gate_norm_reference(o.to(bf).reshape(-1, H * P), row[:, C + 2 * H:], w["gate_w"], 1, 1e-5), r, conv, state


def near(got, want, tol=1.1e-2):
    got, want = got.cpu().to(F8), want.to(F8)
    rel = float((got - want).norm() / want.norm())
    say(f"  relL2 {rel:.2e}")
    assert torch.isfinite(got).all() and rel <= tol


def test_prompts_then_tokens_through_a_block():
    say("case delta block")
    w, g = weights(), torch.Generator().manual_seed(1)
    gw = {k: v.cuda() for k, v in w.items()}
    lens, slots = [70, 1, 130], torch.tensor([2, 0, 3], dtype=torch.int32)
    rows = sum(lens)
    x, res = torch.randn(rows, D, generator=g).to(bf), torch.randn(rows, D, generator=g)
    conv, state = torch.zeros(5, C, 3, dtype=bf), torch.zeros(5, H, P, N)
    gc, gs = conv.cuda(), state.cuda()
    cu = torch.tensor([0, 70, 71, 201], dtype=torch.int32, device="cuda")
    y, r = block(gw, x.cuda(), res.cuda(), cu, slots.cuda(), None, gc, gs)
    yr, rr, conv, state = reference(w, x, res, lens, slots, torch.zeros(3), conv, state)
    torch.cuda.synchronize()
    near(y, yr), near(r, rr, 1e-6), near(gs, state), near(gc, conv)
    # five tokens per request; from the second on, the captured run
    graph, live = None, dict(x=torch.zeros(3, D, dtype=bf, device="cuda"), res=torch.zeros(3, D, device="cuda"), slots=slots.cuda())
    for i in range(5):
        x, res = torch.randn(3, D, generator=g).to(bf), torch.randn(3, D, generator=g)
        live["x"].copy_(x), live["res"].copy_(res)
        c0, s0 = gc.cpu(), gs.cpu()
        if i == 1:
            keep = gc.clone(), gs.clone()
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                out = block(gw, live["x"], live["res"], None, live["slots"], None, gc, gs)
            gc.copy_(keep[0]), gs.copy_(keep[1])
        if graph is None:
            out = block(gw, live["x"], live["res"], None, live["slots"], None, gc, gs)
        else:
            graph.replay()
        torch.cuda.synchronize()
        yr, rr, conv, state = reference(w, x, res, [1] * 3, slots, torch.ones(3), c0, s0)
        near(out[0], yr), near(out[1], rr, 1e-6), near(gs, state), near(gc, conv)


def test_ragged_prompts_by_every_way_the_chunks_are_walked():
    """The same sequences in calls that fill the chip less and more: the variants that the
    number of heads and sequences selects agree as two orders of the same sums do."""
    say("case delta variants")
    gen = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda").to(bf)  # noqa: E731
    for n, p in ((64, 128), (128, 128), (128, 64), (64, 192)):
        heads, lens = 2, [150, 64, 33]
        rows = sum(lens)
        q, k, v, dt, be = r(rows, n), r(rows, n), r(rows, heads * p), r(rows, heads), r(rows, heads)
        A, st = -torch.rand(heads, device="cuda") - 0.5, torch.randn(3, heads, p, n, device="cuda") * 0.3
        cu, slots, on = (torch.tensor(t, dtype=torch.int32, device="cuda") for t in ([0, 150, 214, 247], [2, 0, 1], [1, 0, 1]))
        s1 = st.clone()
        y1 = ssm.ssm_delta_fwd_cache(q, k, v, dt, be, A, cu, slots, s1, resume=on)
        for copies in (8, 24, 90):  # more heads, all alike
            wide = lambda t, c: t.reshape(rows, -1).repeat(1, c)  # noqa: E731
            s2 = st.repeat(1, copies, 1, 1)
            y2 = ssm.ssm_delta_fwd_cache(q, k, wide(v, copies), wide(dt, copies), wide(be, copies), A.repeat(copies), cu, slots, s2, resume=on)
            torch.cuda.synchronize()
            first = s2[:, :heads]
            assert torch.equal(s2, first.repeat(1, copies, 1, 1)) and torch.equal(y2, y2[:, :heads].repeat(1, copies, 1))
            assert float((first - s1).norm() / s1.norm()) <= 2e-6
            assert float((y2[:, :heads].float() - y1.float()).norm() / y1.float().norm()) <= 2.0 ** -8
