"""The operators of a block as a model runs them, one behind the other on one
stream (needs MI355X): the residual sum and norm, the projection, the SSD layer
on its cache over packed prompts, the gate and norm, two blocks deep; then
tokens one at a time on the same caches; and the norms' gradients chained.

Every output is held against the 64-bit definition on the inputs that its kernel
was given, with the bounds of the single operators' tests, so that a wrong
stride, slot, order or buffer anywhere in the chain shows at that place.
"""
import pytest
import torch

import selective_state_space_16_amd as ssm
from block_util import F8, add_norm_reference, gate_norm_reference, owned
from gpu_util import say
from test_norms_gpu import HALF, U, gate_inputs, gate_terms, near
from test_ssd_cache_gpu import compare

pytestmark = pytest.mark.gpu
EPS = 1e-5


class Block:
    """One block's weights and caches; `run` takes the stream of hidden states
    (rows, D) and the residual, for prompts (`cu`) or single tokens."""

    def __init__(self, D, H, P, G, N, groups, slots, seed, project=True):
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=g).cuda()  # noqa: E731
        self.D, self.H, self.P, self.G, self.N, self.groups = D, H, P, G, N, groups
        self.inner, self.C = H * P, H * P + 2 * G * N
        self.width = (self.inner + self.C + H + 7) // 8 * 8  # z | x B C | dt | padding
        self.w_norm, self.w_gate = rnd(D) * 0.2 + 1, rnd(self.inner) * 0.2 + 1
        self.w_in = rnd(D, self.width) * D ** -0.5 if project else None
        self.w_out = rnd(self.inner, D) * self.inner ** -0.5 if project else None
        self.conv_w, self.conv_b = rnd(self.C, 4) * 0.3, rnd(self.C) * 0.1
        self.dt_bias, self.A, self.skip = rnd(H) - 3, -torch.exp(rnd(H)), rnd(H) * 0.3 + 1
        self.conv = rnd(slots, self.C, 3).bfloat16()
        self.state = rnd(slots, H, P, N) * 0.3

    def cut(self, proj):
        a, b = self.inner, self.inner + self.C
        return proj[:, :a], proj[:, a:b], proj[:, b:b + self.H]

    def run(self, x, residual, slots, cu=None, resume=None, tape=None, workspace=None):
        y1, r = ssm.ssm_add_norm_fwd(x, self.w_norm, residual=residual, eps=EPS)
        proj = (y1.float() @ self.w_in).bfloat16() if self.w_in is not None else y1
        z, xbc, dt = self.cut(proj)
        y0 = torch.zeros(x.shape[0], self.H, self.P, dtype=torch.bfloat16, device="cuda")
        held = (self.conv.clone(), self.state.clone()) if tape is not None else None
        rest = dict(conv_b=self.conv_b, dt_bias=self.dt_bias, Dskip=self.skip, y=y0, workspace=workspace)
        if cu is None:
            y2 = ssm.ssm_ssd_step_cache(xbc, dt, self.A, self.conv_w, slots, self.conv, self.state, **rest)
        else:
            y2 = ssm.ssm_ssd_fwd_cache(xbc, dt, self.A, self.conv_w, cu, slots, self.conv, self.state, resume=resume, **rest)
        y3 = ssm.ssm_gate_norm_fwd(y2.view(x.shape[0], self.inner), z, self.w_gate, groups=self.groups, eps=EPS)
        if tape is not None:
            after = self.conv.clone(), self.state.clone()
            tape.append((self, x, residual, y1, r, proj, y2, y3, held, after))
        if self.w_out is not None:
            return (y3.float() @ self.w_out).bfloat16(), r
        out = torch.zeros_like(x)
        out[:, :self.inner] = y3
        return out, r


def check(tape, lens, slots, resume, single):
    """Every kernel of the run against its definition on its own inputs."""
    for k, (blk, x, residual, y1, r, proj, y2, y3, held, after) in enumerate(tape):
        x, residual, y1c, rc = x.cpu(), None if residual is None else residual.cpu(), y1, r
        w = blk.w_norm.cpu()
        yr, rr = add_norm_reference(x, residual, None, w, EPS)
        big = x.to(F8).abs() + (0 if residual is None else residual.to(F8).abs())
        near(rc, rr, big, 2, f"block {k} r")
        rstd = 1 / torch.sqrt(rr.square().mean(1, keepdim=True) + EPS)
        near(y1c, yr, big * rstd * w.abs() + yr.abs(), 48, f"block {k} norm")
        z, xbc, dt = (t.cpu() for t in blk.cut(proj))
        d = dict(H=blk.H, P=blk.P, G=blk.G, N=blk.N, C=blk.C, lens=lens, slots=slots.cpu(), resume=resume,
                 proj=torch.cat([torch.zeros(x.shape[0], 64, dtype=xbc.dtype), xbc, dt], 1), conv_w=blk.conv_w.cpu(),
                 conv_b=blk.conv_b.cpu(), dt_bias=blk.dt_bias.cpu(), A=blk.A.cpu(), Dskip=blk.skip.cpu(),
                 conv_cache=held[0].cpu(), state_cache=held[1].cpu())
        compare(d, dict(conv_cache=after[0], state_cache=after[1]), y2, torch.zeros(y2.shape, dtype=y2.dtype),
                f"block {k}", products=not single)
        y2c = y2.cpu().view(x.shape[0], blk.inner)
        ref = gate_norm_reference(y2c, z, blk.w_gate.cpu(), blk.groups, EPS)
        near(y3, ref, ref.abs(), 48, f"block {k} gate norm")


def test_prompts_then_tokens():
    """Three prompts of unlike lengths through two blocks, rows behind the last
    one unused, then four tokens each, with a padding row in the batch."""
    say("case block prompts then tokens")
    D, lens, spare = 320, [150, 1, 66], 3
    blocks = [Block(D, 4, 64, 2, 64, 2, 6, 1), Block(D, 2, 128, 1, 128, 1, 6, 2)]
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 150, 151, 217], dtype=torch.int32, device="cuda")
    resume = torch.tensor([0, 1, 0], dtype=torch.int32, device="cuda")
    x = torch.randn(217 + spare, D, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    res, tape = None, []
    for b in blocks:
        x, res = b.run(x, res, slots, cu, resume, tape)
    torch.cuda.synchronize()
    check(tape, lens, slots, resume.cpu(), False)
    slots = torch.tensor([2, -1, 4, 0], dtype=torch.int32, device="cuda")
    for t in range(4):
        x = torch.randn(4, D, generator=torch.Generator().manual_seed(9 + t)).bfloat16().cuda()
        res, tape = None, []
        for b in blocks:
            x, res = b.run(x, res, slots, tape=tape)
        torch.cuda.synchronize()
        assert owned(slots, 6) == [2, -1, 4, 0] and not tape[0][6][1].any()
        check(tape, [1] * 4, slots, torch.ones(4), True)


def test_captured_run():
    """Two blocks over prompts and two tokens behind them, captured once, their
    workspace shared by every call of the graph, replayed on restored caches
    with eager calls between: equal bits each time."""
    say("case block captured")
    shapes = [(4, 64, 2, 64, 2), (2, 128, 1, 64, 1)]  # both rows: z | x B C | dt of 776 at most
    D = 256 + 256 + 2 * 2 * 64 + 8
    blocks = [Block(D, *s, 6, 5 + k, project=False) for k, s in enumerate(shapes)]
    g = torch.Generator().manual_seed(6)
    x0, x1 = (torch.randn(n, D, generator=g).bfloat16().cuda() for n in (130, 2))
    slots = torch.tensor([1, 5], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 99, 130], dtype=torch.int32, device="cuda")
    need = max(ssm.ssm_ssd_fwd_cache_workspace_bytes(2, 130, b.H, b.P, b.G, b.N, ssm.SSM_BF16) for b in blocks)
    need = max([need] + [ssm.ssm_ssd_step_cache_workspace_bytes(2, b.H, b.P, b.G, b.N) for b in blocks])
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    first = [(b.conv.clone(), b.state.clone()) for b in blocks]

    def run():
        x, r, outs = x0, None, []
        for b in blocks:
            x, r = b.run(x, r, slots, cu, workspace=ws)
        outs += [x, r]
        for _ in range(2):
            x, r = x1, None
            for b in blocks:
                x, r = b.run(x, r, slots, workspace=ws)
            outs += [x, r]
        return outs

    def restore():
        for b, (c, s) in zip(blocks, first):
            b.conv.copy_(c)
            b.state.copy_(s)

    eager = run()
    torch.cuda.synchronize()
    caches = [(b.conv.clone(), b.state.clone()) for b in blocks]
    restore()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run()
    for rep in range(4):
        restore()
        for o in outs:
            o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, outs)), f"replay {rep}"
        assert all(torch.equal(b.conv, c) and torch.equal(b.state, s) for b, (c, s) in zip(blocks, caches)), f"replay {rep}"
        restore()
        again = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, again)), f"eager {rep}"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_chained_gradients(dtype):
    """x, residual -> add norm -> (u | z) -> gate norm, backwards: dx of the first
    from dy of the second. The bound is the first step's (rounding of the
    intermediate gradient and its float32 terms), carried through the absolute
    terms of the second, plus the second's own; products of two errors are under
    one hundredth of either."""
    say(f"case chained gradients {dtype}")
    rows, inner = 70, 520
    e = gate_inputs(rows, 2 * inner, dtype, 12)
    x, residual, scale = e["x"], e["z"].float(), e["weight"] + 0.5
    w1, w2 = gate_inputs(1, 2 * inner, dtype, 13)["weight"], gate_inputs(1, inner, dtype, 14)["weight"]
    dy = gate_inputs(rows, inner, dtype, 15)["dy"]
    c = lambda t: t.cuda()  # noqa: E731
    y1, r = ssm.ssm_add_norm_fwd(c(x), c(w1), residual=c(residual), scale=c(scale), eps=EPS)
    got = ssm.ssm_gate_norm_bwd(c(dy), y1[:, :inner], y1[:, inner:], c(w2), groups=2, eps=EPS)
    back = ssm.ssm_add_norm_bwd(torch.cat([got["dx"], got["dz"]], 1), r, c(w1), x=c(x), scale=c(scale), eps=EPS)
    torch.cuda.synchronize()
    y1, r = y1.cpu(), r.cpu().to(F8)
    u, z = (t.to(F8).requires_grad_() for t in (y1[:, :inner], y1[:, inner:]))
    du, dz = torch.autograd.grad((gate_norm_reference(u, z, w2, 2, EPS) * dy.to(F8)).sum(), (u, z))
    tu, tz, _ = gate_terms(dict(x=y1[:, :inner], z=y1[:, inner:], weight=w2, dy=dy), 2)
    mid = torch.cat([du, dz], 1)
    mid_err = HALF[dtype] * mid.abs() + 56 * U * torch.cat([tu, tz], 1)
    leaf, w = r.clone().requires_grad_(), w1.to(F8).requires_grad_()
    out = leaf / torch.sqrt(leaf.square().mean(1, keepdim=True) + EPS) * w
    dr, dw = torch.autograd.grad((out * mid).sum(), (leaf, w))
    rstd = 1 / torch.sqrt(r.square().mean(1, keepdim=True) + EPS)
    hat = r * rstd
    carry = lambda t: rstd * ((t * w1).abs() + hat.abs() * (t * w1 * hat).abs().mean(1, keepdim=True))  # noqa: E731

    def within(name, value, ref, carried, terms, roundings):
        value = value.cpu()
        tol = HALF[value.dtype] * ref.abs() + 1.01 * carried + roundings * U * terms
        err = (value.to(F8) - ref).abs()
        say(f"  {name}: worst of bound {float((err / tol).max()):.3f}")
        assert (err <= tol).all(), name

    s = scale.to(F8).abs()
    within("dresidual", back["dresidual"], dr, carry(mid_err), carry(mid), 48)
    within("dx", back["dx"], dr * scale.to(F8), carry(mid_err) * s, carry(mid) * s, 49)
    within("dweight", back["dweight"], dw.detach(), (mid_err * hat.abs()).sum(0), (mid * hat).abs().sum(0), 65)
    ax = x.to(F8).abs()
    within("dscale", back["dscale"], (dr * x.to(F8)).sum(0), (carry(mid_err) * ax).sum(0), (carry(mid) * ax).sum(0), 113)
