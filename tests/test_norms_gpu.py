"""The norms of a block (ssm_add_norm_*, ssm_gate_norm_*) against plain 64-bit
references and their derivatives (needs MI355X).

Error bounds: an output is rounded to its type once (half a step: 2^-8 for
bfloat16, 2^-24 for float32, of its value). In float32 a row's two sums add D
terms in a tree of at most 16 + 6 + 4 levels, and every other factor (SiLU,
rstd, products) adds a few roundings: 48 roundings of 2^-24, relative to the
absolute terms of the output. The gradients of weight and scale add one
rounding per row that a workgroup holds and per partial row.
"""
import pytest
import torch

import selective_state_space_16_amd as ssm
from block_util import F8, add_norm_reference, gate_norm_reference
from gpu_util import say

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, FL = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, FL: 2.0 ** -24}


def near(got, ref, terms, roundings, what):
    got, half = got.detach().cpu(), HALF[got.dtype]
    tol = half * ref.abs() + roundings * U * terms
    err = (got.double() - ref).abs()
    say(f"  {what}: worst of bound {float((err / tol.clamp_min(1e-300)).max()) if err.numel() else 0:.3f}")
    assert torch.isfinite(got).all(), what
    assert (err <= tol).all(), what


SHAPES = [(1, 1), (3, 7), (5, 8), (2, 64), (130, 100), (4, 513), (9, 768), (6, 1001), (2049, 16), (3, 1536), (3, 2000), (3, 2560),
          (5, 2568), (2, 3000), (4, 4096), (3, 5000), (2, 8192), (2, 9001), (2, 16384), (2, 16383)]


def add_inputs(rows, D, dtype, wide, seed):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return dict(x=rnd(rows, D).to(dtype), residual=(2 * rnd(rows, D)).to(FL if wide else dtype), scale=rnd(D) * 0.5 + 1,
                weight=rnd(D) * 0.2 + 1, dy=rnd(rows, D).to(dtype), dres=rnd(rows, D).to(FL if wide else dtype))


@pytest.mark.parametrize("dtype,wide", [(BF, True), (BF, False), (FL, True)])
@pytest.mark.parametrize("rows,D", SHAPES)
def test_add_norm(rows, D, dtype, wide):
    say(f"case add norm {rows}x{D} {dtype} wide={wide}")
    d = add_inputs(rows, D, dtype, wide, rows + D)
    g = {k: v.cuda() for k, v in d.items()}
    for res, scale in ((True, True), (False, True), (True, False)):
        y, r = ssm.ssm_add_norm_fwd(g["x"], g["weight"], residual=g["residual"] if res else None,
                                    scale=g["scale"] if scale else None, eps=1e-5)
        yr, rr = add_norm_reference(d["x"], d["residual"] if res else None, d["scale"] if scale else None, d["weight"], 1e-5)
        big = d["x"].to(F8).abs() * (d["scale"].abs() if scale else 1) + (d["residual"].to(F8).abs() if res else 0)
        near(r, rr, big, 2, "r")
        rstd = 1 / torch.sqrt(rr.square().mean(1, keepdim=True) + 1e-5)
        near(y, yr, big * rstd * d["weight"].abs() + yr.abs(), 48, "y")


@pytest.mark.parametrize("dtype,wide", [(BF, True), (BF, False), (FL, True)])
@pytest.mark.parametrize("rows,D", SHAPES)
def test_add_norm_gradient(rows, D, dtype, wide):
    say(f"case add norm gradient {rows}x{D} {dtype} wide={wide}")
    d = add_inputs(rows, D, dtype, wide, rows + D + 1)
    g = {k: v.cuda() for k, v in d.items()}
    for scaled, up in ((True, True), (False, False)):
        out = ssm.ssm_add_norm_bwd(g["dy"], g["residual"], g["weight"], x=g["x"] if scaled else None,
                                   scale=g["scale"] if scaled else None, dres=g["dres"] if up else None)
        r = d["residual"].to(F8).requires_grad_()
        w = d["weight"].to(F8).requires_grad_()
        y = r / torch.sqrt(r.square().mean(1, keepdim=True) + 1e-5) * w
        loss = (y * d["dy"].to(F8)).sum() + ((r * d["dres"].to(F8)).sum() if up else 0)
        dr, dw = torch.autograd.grad(loss, (r, w))
        s, x = d["scale"].to(F8) if scaled else 1.0, d["x"].to(F8)
        rstd = 1 / torch.sqrt(r.detach().square().mean(1, keepdim=True) + 1e-5)
        hat, gg = r.detach() * rstd, d["dy"].to(F8) * d["weight"].to(F8)
        terms = rstd * (gg.abs() + hat.abs() * (gg * hat).abs().mean(1, keepdim=True)) + (d["dres"].to(F8).abs() if up else 0)
        near(out["dresidual"], dr, terms, 48, "dresidual")
        near(out["dx"], dr * s, terms * abs(s) if scaled else terms, 49, "dx")
        per = 64 + rows / 512
        near(out["dweight"], dw, (d["dy"].to(F8) * hat).abs().sum(0), per, "dweight")
        if scaled:
            near(out["dscale"], (dr * x).sum(0), (terms * x.abs()).sum(0), per + 48, "dscale")
        else:
            assert out["dscale"] is None


def gate_inputs(rows, D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return dict(x=rnd(rows, D).to(dtype), z=(2 * rnd(rows, D)).to(dtype), weight=rnd(D) * 0.2 + 1, dy=rnd(rows, D).to(dtype))


def gate_terms(d, groups):
    rows = d["x"].shape[0]
    x, z, w, dy = (d[k].to(F8) for k in ("x", "z", "weight", "dy"))
    u = x * z * torch.sigmoid(z)
    by = lambda t: t.reshape(rows, groups, -1)  # noqa: E731
    rstd = 1 / torch.sqrt(by(u).square().mean(2, keepdim=True) + 1e-5)
    hat, g = by(u) * rstd, by(dy * w)
    du = (rstd * (g.abs() + hat.abs() * (g * hat).abs().mean(2, keepdim=True))).reshape(x.shape)
    s = torch.sigmoid(z)
    return du * (z * s).abs(), du * x.abs() * s * (1 + z.abs() * (1 - s)), (dy * hat.reshape(x.shape)).abs().sum(0)


@pytest.mark.parametrize("dtype", [BF, FL])
@pytest.mark.parametrize("groups", [1, 2, 5])
@pytest.mark.parametrize("rows,D", [(1, 1), (3, 7), (5, 8), (2, 64), (130, 100), (9, 768), (6, 1001), (2049, 16), (3, 2560), (3, 5120),
                                    (2, 8192), (2, 9001), (2, 16384)])
def test_gate_norm(rows, D, groups, dtype):
    D *= groups
    say(f"case gate norm {rows}x{D}/{groups} {dtype}")
    d = gate_inputs(rows, D, dtype, rows + D)
    g = {k: v.cuda() for k, v in d.items()}
    y = ssm.ssm_gate_norm_fwd(g["x"], g["z"], g["weight"], groups=groups)
    yr = gate_norm_reference(d["x"], d["z"], d["weight"], groups, 1e-5)
    near(y, yr, yr.abs(), 48, "y")
    out = ssm.ssm_gate_norm_bwd(g["dy"], g["x"], g["z"], g["weight"], groups=groups)
    leaves = [d[k].to(F8).requires_grad_() for k in ("x", "z", "weight")]
    grads = torch.autograd.grad((gate_norm_reference(*leaves, groups, 1e-5) * d["dy"].to(F8)).sum(), leaves)
    tx, tz, tw = gate_terms(d, groups)
    near(out["dx"], grads[0], tx, 56, "dx")
    near(out["dz"], grads[1], tz, 56, "dz")
    near(out["dweight"], grads[2], tw, 72 + rows / 512, "dweight")


@pytest.mark.parametrize("which", ["add", "gate"])
def test_gradients_against_differences(which):
    """Central differences of the kernel's own forward in float32: with a step h,
    an error of h^2 times the third derivative (about one here) and of 2^-24
    |loss terms| / h from the rounded outputs."""
    say(f"case differences {which}")
    rows, D, h = 2, 48, 2.0 ** -6
    g = torch.Generator().manual_seed(4)
    a, b, dy = (torch.randn(rows, D, generator=g).cuda() for _ in range(3))
    w = (torch.randn(D, generator=g) * 0.2 + 1).cuda()
    scale = (torch.rand(D, generator=g) + 0.5).cuda()
    if which == "add":
        f = lambda a, b, w: (ssm.ssm_add_norm_fwd(a, w, residual=b, scale=scale)[0].double() * dy.double()).sum()  # noqa: E731
        r = ssm.ssm_add_norm_fwd(a, w, residual=b, scale=scale)[1]
        o = ssm.ssm_add_norm_bwd(dy, r, w, x=a, scale=scale)
        grads = (o["dx"], o["dresidual"], o["dweight"])
    else:
        f = lambda a, b, w: (ssm.ssm_gate_norm_fwd(a, b, w).double() * dy.double()).sum()  # noqa: E731
        o = ssm.ssm_gate_norm_bwd(dy, a, b, w)
        grads = (o["dx"], o["dz"], o["dweight"])
    tol = 4 * h * h + 64 * D * U / h
    for i, (t, gr) in enumerate(zip((a, b, w), grads)):
        for k in (0, 17, t.numel() - 1):
            args = [a, b, w]
            up, down = t.clone(), t.clone()
            up.view(-1)[k] += h
            down.view(-1)[k] -= h
            args[i] = up
            hi = f(*args)
            args[i] = down
            diff = float((hi - f(*args)) / (2 * h))
            assert abs(diff - float(gr.reshape(-1)[k])) <= tol * (1 + abs(diff)), (i, k)


def test_rows_apart_and_alignment():
    """The gate as a slice of a wider row, dz written into one, and rows that are
    not whole 16-byte pieces: the same bits as dense rows of the same kind."""
    say("case strides")
    rows, D = 37, 256
    for dtype in (BF, FL):
        d = {k: v.cuda() for k, v in gate_inputs(rows, D, dtype, 3).items()}
        y = ssm.ssm_gate_norm_fwd(d["x"], d["z"], d["weight"])
        ref = ssm.ssm_gate_norm_bwd(d["dy"], d["x"], d["z"], d["weight"])
        for wide, off in ((3 * D, D), (D + 8, 0), (D + 3, 0)):
            store = torch.full((rows, wide), 9.0, dtype=dtype, device="cuda")
            dst = torch.full((rows, wide), 5.0, dtype=dtype, device="cuda")
            z, dz = store[:, off:off + D], dst[:, off:off + D]
            z.copy_(d["z"])
            got = ssm.ssm_gate_norm_fwd(d["x"], z, d["weight"])
            out = ssm.ssm_gate_norm_bwd(d["dy"], d["x"], z, d["weight"], out={"dz": dz})
            torch.cuda.synchronize()
            tol = 0 if wide % 8 == 0 else 4 * HALF[dtype]  # another order of the row's sum
            for p, q in ((got, y), (out["dx"], ref["dx"]), (dz, ref["dz"])):
                assert (p.float() - q.float()).abs().max() <= tol * q.float().abs().max()
            mask = torch.ones(wide, dtype=torch.bool, device="cuda")
            mask[off:off + D] = False
            assert (dst[:, mask] == 5).all()


def test_in_place():
    say("case in place")
    d = {k: v.cuda() for k, v in add_inputs(33, 520, BF, True, 8).items()}
    y, r = ssm.ssm_add_norm_fwd(d["x"], d["weight"], residual=d["residual"], scale=d["scale"])
    x2, r2 = d["x"].clone(), d["residual"].clone()
    ssm.ssm_add_norm_fwd(x2, d["weight"], residual=r2, scale=d["scale"], y=x2, residual_out=r2)
    ref = ssm.ssm_add_norm_bwd(d["dy"], r, d["weight"], x=d["x"], scale=d["scale"], dres=d["dres"])
    dy2, up2 = d["dy"].clone(), d["dres"].clone()
    out = ssm.ssm_add_norm_bwd(dy2, r, d["weight"], x=d["x"], scale=d["scale"], dres=up2, out={"dx": dy2, "dresidual": up2})
    torch.cuda.synchronize()
    assert torch.equal(x2, y) and torch.equal(r2, r)
    assert torch.equal(out["dx"], ref["dx"]) and torch.equal(up2, ref["dresidual"]) and torch.equal(out["dweight"], ref["dweight"])


def test_zero_and_special_rows():
    """A row of zeros stays zero (eps keeps the norm finite); a NaN stays in its row
    and in the weights' gradient; an infinite gate value of the closed side is
    NaN, as in the definition; no rows give zero gradients."""
    say("case special rows")
    d = {k: v.cuda() for k, v in gate_inputs(5, 64, FL, 9).items()}
    d["x"][1] = 0
    d["x"][3, 7] = float("nan")
    y = ssm.ssm_gate_norm_fwd(d["x"], d["z"], d["weight"])
    out = ssm.ssm_gate_norm_bwd(d["dy"], d["x"], d["z"], d["weight"])
    torch.cuda.synchronize()
    assert not y[1].any() and torch.isnan(y[3]).all()
    ok = [0, 1, 2, 4]
    assert torch.isfinite(y[ok]).all() and torch.isfinite(out["dx"][ok]).all() and torch.isfinite(out["dz"][ok]).all()
    empty = ssm.ssm_gate_norm_bwd(d["dy"][:0], d["x"][:0], d["z"][:0], d["weight"])
    both = ssm.ssm_add_norm_bwd(d["dy"][:0], d["x"][:0], d["weight"], x=d["x"][:0], scale=d["weight"])
    torch.cuda.synchronize()
    assert not empty["dweight"].any() and not both["dweight"].any() and not both["dscale"].any()


def test_bits_graph_and_stream():
    """Equal inputs give equal bits; a captured call replays like the eager one;
    a call on another stream with tensors that the binding allocates."""
    say("case bits, graph, stream")
    d = {k: v.cuda() for k, v in add_inputs(3000, 520, BF, True, 10).items()}
    e = {k: v.cuda() for k, v in gate_inputs(3000, 512, BF, 11).items()}
    run = lambda **kw: (ssm.ssm_add_norm_bwd(d["dy"], d["residual"], d["weight"], x=d["x"], scale=d["scale"], dres=d["dres"], **kw),  # noqa: E731
                        ssm.ssm_gate_norm_bwd(e["dy"], e["x"], e["z"], e["weight"], groups=2, **kw))
    a, b = run()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    a2, b2 = run(stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a[k], a2[k]) for k in a) and all(torch.equal(b[k], b2[k]) for k in b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a3, b3 = run(stream=torch.cuda.current_stream())
    for rep in range(4):
        for t in (*a3.values(), *b3.values()):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a[k], a3[k]) for k in a) and all(torch.equal(b[k], b3[k]) for k in b), f"replay {rep}"
        run()
        torch.cuda.synchronize()


def test_many_elements():
    """More than 2^32 bytes of a tensor: the last rows of a large batch equal the
    same rows alone."""
    say("case large")
    rows, D = 270000, 8192  # 4.4 GB in bfloat16
    x = torch.randn(1000, D, device="cuda").bfloat16().repeat(270, 1)
    w = torch.randn(D, device="cuda")
    y = ssm.ssm_gate_norm_fwd(x, x, w)
    tail = ssm.ssm_gate_norm_fwd(x[-1000:], x[-1000:], w)
    torch.cuda.synchronize()
    assert torch.equal(y[-1000:], tail) and torch.equal(y[:1000], tail)
    assert rows == x.shape[0]


@pytest.mark.parametrize("dtype", [BF, FL])
@pytest.mark.parametrize("rows,D", [(70, 24), (33, 61), (257, 65), (40, 128), (41, 129), (31, 200), (5, 255), (600, 256), (9, 257)])
def test_short_rows(rows, D, dtype):
    """Rows that share a wave, in workgroups that they fill in part."""
    test_add_norm(rows, D, dtype, True)
    test_add_norm_gradient(rows, D, dtype, True)
    test_gate_norm(rows, D, 2, dtype)
