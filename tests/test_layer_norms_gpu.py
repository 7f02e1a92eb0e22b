"""The residual sum and layer norm ahead of a block (ssm_add_layer_norm_fwd and
_bwd) against plain 64-bit definitions (needs MI355X).

Error bounds (u = 2^-24): r takes 2 roundings. A row's mean is a sum of float32
partial sums of at most 24 terms per lane, the rest in double: its error, at most 26 u
of the mean of |r|, is taken off again by the second pass up to 2 u of that pass's
values. (r - mean) / sd so has at most 6 roundings of itself, the 2 of r relative to
|r| / sd, and the error of the sum of squares (26 u at most, half of it after the
root): 26 u of |hat|; weight and bias add 2 u of their terms. The gradient adds the
means of g and of g hat, 30 u of the means of their absolute values each, and three
roundings; sums over rows have at most one rounding per row and workgroup, taken as
64 + rows / 256 roundings (512 workgroups' partial sums, in 16 slices)."""
import pytest
import torch

import selective_state_space_16_amd as ssm
from delta_util import layer_norm_reference
from gpu_util import say

pytestmark = pytest.mark.gpu
F8, U = torch.float64, 2.0 ** -24
EPS = 1e-5
bf, f4 = torch.bfloat16, torch.float32


def half(t):
    return 2.0 ** -8 if t == bf else U


def make(rows, D, dtype, res, scaled, seed=0, mean=0.5, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return dict(x=(r(rows, D) * spread + mean).to(dtype), residual=None if res is None else (r(rows, D) * 2 * spread).to(res),
                scale=torch.rand(D, generator=g) + 0.1 if scaled else None, weight=1 + 0.2 * r(D), bias=r(D) * 0.3,
                dy=r(rows, D).to(dtype), dres=None if res is None else r(rows, D).to(res))


def gpu(d):
    return {k: None if v is None else v.cuda() for k, v in d.items()}


def check_fwd(d, y, r):
    yr, rr = layer_norm_reference(d["x"], d["residual"], d["scale"], d["weight"], d["bias"], EPS)
    sd = torch.sqrt(rr.var(1, unbiased=False, keepdim=True) + EPS)
    mag = rr.abs() if d["residual"] is None else d["residual"].to(F8).abs() + (d["x"].to(F8) * (1 if d["scale"] is None else d["scale"].to(F8))).abs()
    hat = ((rr - rr.mean(1, keepdim=True)) / sd).abs()
    w = d["weight"].to(F8).abs()
    tol = half(y.dtype) * yr.abs() + U * (w * (28 * hat + 4 * (mag + mag.mean(1, keepdim=True)) / sd) + 2 * (0 if d["bias"] is None else d["bias"].to(F8).abs()))
    err = (y.cpu().to(F8) - yr).abs()
    say(f"  y of bound {float((err / tol).max()):.2f}")
    assert torch.isfinite(err).all() and (err <= tol).all()
    if r is not None:
        assert ((r.cpu().to(F8) - rr).abs() <= half(r.dtype) * rr.abs() + 2 * U * mag).all()


SHAPES = [(1, 1), (3, 7), (5, 8), (9, 63), (4, 65), (7, 100), (3, 255), (6, 257), (2, 500), (5, 513), (3, 1001), (4, 1025), (2, 1536), (3, 1537),
          (2, 2048), (2, 2560), (3, 2567), (2, 4096), (2, 5120), (1, 6144), (2, 6145), (1, 8192), (2, 8200), (1, 16384), (1, 16383), (600, 24)]


@pytest.mark.parametrize("rows,D", SHAPES)
@pytest.mark.parametrize("dtype,res", [(bf, f4), (bf, bf), (f4, f4), (bf, None), (f4, None)])
def test_forward(rows, D, dtype, res):
    say(f"case layer norm fwd {rows} x {D} {dtype} {res}")
    d = make(rows, D, dtype, res, scaled=D % 2 == 1, seed=rows + D)
    g = gpu(d)
    y, r = ssm.ssm_add_layer_norm_fwd(g["x"], g["weight"], g["bias"], residual=g["residual"], scale=g["scale"], eps=EPS)
    torch.cuda.synchronize()
    check_fwd(d, y, None if r is g["x"] else r)


def check_bwd(d, r, out, scale):
    f = lambda t: t.to(F8)  # noqa: E731
    r, dy, w = f(r), f(d["dy"]), f(d["weight"])
    D, rows = r.shape[1], r.shape[0]
    sd = torch.sqrt(r.var(1, unbiased=False, keepdim=True) + EPS)
    hat = (r - r.mean(1, keepdim=True)) / sd
    g = dy * w
    mean = lambda t: t.mean(1, keepdim=True)  # noqa: E731
    dres = 0 if d["dres"] is None else f(d["dres"])
    dr = (g - mean(g) - hat * mean(g * hat)) / sd + dres
    # an error of hat: 28 u of itself and 4 u of (|r| and its mean) / sd
    eh = U * (28 * hat.abs() + 4 * (r.abs() + mean(r.abs())) / sd)
    tol = (U * (34 * g.abs() + 34 * mean(g.abs()) + 64 * hat.abs() * mean((g * hat).abs())) + eh * mean((g * hat).abs())
           + hat.abs() * mean(g.abs() * eh)) / sd + 2 * U * (0 if d["dres"] is None else dres.abs())
    s = 1 if scale is None else f(scale)
    for name, want, t in (("dresidual", dr, tol), ("dx", dr * s, tol * s)):
        got = out[name].cpu()
        err, t = (f(got) - want).abs(), t + half(got.dtype) * want.abs() + U * want.abs()
        say(f"  {name} of bound {float((err / t).max()):.2f}")
        assert (err <= t).all(), name
    n = (64 + rows / 256) * U
    checks = [("dweight", (dy * hat).sum(0), ((dy * hat).abs() * n + dy.abs() * eh).sum(0)), ("dbias", dy.sum(0), n * dy.abs().sum(0))]
    if scale is not None:
        x = f(d["x"])
        checks.append(("dscale", (dr * x).sum(0), ((dr * x).abs() * n + tol * x.abs()).sum(0)))
    for name, want, t in checks:
        err = (f(out[name].cpu()) - want).abs()
        say(f"  {name} of bound {float((err / t.clamp_min(1e-300)).max()):.2f}")
        assert (err <= t).all(), name


@pytest.mark.parametrize("rows,D", SHAPES + [(700, 64), (1025, 40), (1, 64), (513, 2560)])
@pytest.mark.parametrize("dtype,res,scaled", [(bf, f4, True), (bf, f4, False), (bf, bf, False), (f4, f4, True), (bf, None, False)])
def test_backward(rows, D, dtype, res, scaled):
    say(f"case layer norm bwd {rows} x {D} {dtype} {res} {scaled}")
    d = make(rows, D, dtype, res, scaled, seed=rows + D + 1)
    r = d["residual"] if res is not None else d["x"]
    g = gpu(d)
    out = ssm.ssm_add_layer_norm_bwd(g["dy"], r.cuda(), g["weight"], x=g["x"] if scaled else None, scale=g["scale"], dres=g["dres"], eps=EPS)
    torch.cuda.synchronize()
    check_bwd(d, r, out, d["scale"])
    assert (out["dresidual"] is out["dx"]) == (r.dtype == dtype and not scaled)


def test_gradient_against_differences():
    """The formula's gradient against central differences of the kernel's own forward,
    in float32. A step of e along a random direction of r: the difference of two losses
    is off by their roundings, 2^-22 of sum |dy y| over 2 e, and by the third
    derivative, e^2 of the gradient's size with a factor below 8 for rows of unit
    spread."""
    say("case layer norm differences")
    d = make(3, 40, f4, f4, False, seed=4)
    g = gpu(d)
    r = (d["residual"] + d["x"]).cuda()
    out = ssm.ssm_add_layer_norm_bwd(g["dy"], r, g["weight"], eps=EPS)
    e = 1e-2
    for seed in range(4):
        v = torch.randn(3, 40, generator=torch.Generator().manual_seed(seed)).cuda()
        v = v / v.norm()
        loss = lambda t: (ssm.ssm_add_layer_norm_fwd(t, g["weight"], g["bias"], eps=EPS)[0].double() * g["dy"].double()).sum()  # noqa: B023,E731
        plus, minus = loss(r + e * v), loss(r - e * v)
        want = float((out["dresidual"].double() * v.double()).sum())
        size = float((g["dy"].double() * ssm.ssm_add_layer_norm_fwd(r, g["weight"], g["bias"], eps=EPS)[0].double()).abs().sum())
        got = float(plus - minus) / (2 * e)
        tol = 2.0 ** -22 * size / (2 * e) + 8 * e * e * float(out["dresidual"].norm())
        assert abs(got - want) <= tol, (got, want, tol)


@pytest.mark.parametrize("mean,spread", [(1e4, 1.0), (1e5, 1e-2), (-300.0, 1e-3), (3.0, 0.0), (0.0, 0.0), (0.0, 1e15), (0.0, 1e-20)])
def test_rows_of_large_means_and_none(mean, spread):
    say(f"case layer norm mean {mean} spread {spread}")
    d = make(4, 1000, f4, None, False, seed=5, mean=mean, spread=spread)
    g = gpu(d)
    y, _ = ssm.ssm_add_layer_norm_fwd(g["x"], g["weight"], g["bias"], eps=EPS)
    out = ssm.ssm_add_layer_norm_bwd(g["dy"], g["x"], g["weight"], eps=EPS)
    torch.cuda.synchronize()
    check_fwd(d, y, None)
    check_bwd(d, d["x"], out, None)


def test_values_that_are_not_finite_stay_in_their_row():
    say("case layer norm nan")
    d = make(5, 300, f4, f4, False, seed=6)
    d["x"][2, 17] = float("inf")
    g = gpu(d)
    y, r = ssm.ssm_add_layer_norm_fwd(g["x"], g["weight"], g["bias"], residual=g["residual"])
    keep = [0, 1, 3, 4]
    assert torch.isfinite(y[keep]).all() and torch.isfinite(r[keep]).all() and not torch.isfinite(y[2]).any()


def test_outputs_over_inputs_streams_graphs_and_equal_bits():
    say("case layer norm aliases")
    d = make(700, 264, bf, f4, True, seed=7)
    g, h = gpu(d), gpu(d)
    y, r = ssm.ssm_add_layer_norm_fwd(g["x"], g["weight"], g["bias"], residual=g["residual"], scale=g["scale"])
    x = h["x"].clone()
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    y2, r2 = ssm.ssm_add_layer_norm_fwd(h["x"], h["weight"], h["bias"], residual=h["residual"], scale=h["scale"], y=h["x"],
                                        residual_out=h["residual"], stream=other)
    other.synchronize()
    assert torch.equal(y, y2) and torch.equal(r, r2) and y2 is h["x"] and r2 is h["residual"]
    want = ssm.ssm_add_layer_norm_bwd(g["dy"], r, g["weight"], x=x, scale=g["scale"], dres=g["dres"])
    keep = {k: v.clone() for k, v in want.items()}
    ws = torch.full((ssm.ssm_add_layer_norm_bwd_workspace_bytes(700, 264) // 4,), float("nan"), device="cuda")
    out = {k: torch.zeros_like(v) for k, v in want.items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ssm.ssm_add_layer_norm_bwd(g["dy"], r, g["weight"], x=x, scale=g["scale"], dres=g["dres"], out=out, workspace=ws)
    for _ in range(3):
        for v in out.values():
            v.zero_()
        graph.replay()
        ssm.ssm_add_layer_norm_bwd(g["dy"], r, g["weight"], x=x, scale=g["scale"], dres=g["dres"])
        torch.cuda.synchronize()
        assert all(torch.equal(out[k], keep[k]) for k in keep)
    got = ssm.ssm_add_layer_norm_bwd(h["dy"], r, h["weight"], x=x, scale=h["scale"], dres=h["dres"],
                                     out=dict(dx=h["dy"], dresidual=h["dres"]))
    torch.cuda.synchronize()
    assert all(torch.equal(got[k], keep[k]) for k in keep)


def test_no_rows():
    say("case layer norm, no rows")
    w = torch.ones(24, device="cuda")
    e = torch.empty(0, 24, device="cuda")
    y, r = ssm.ssm_add_layer_norm_fwd(e, w)
    out = ssm.ssm_add_layer_norm_bwd(e, e, w, x=e, scale=w, out=dict(dweight=torch.ones(24, device="cuda"), dbias=torch.ones(24, device="cuda")))
    torch.cuda.synchronize()
    assert y.shape == (0, 24) and r is e and all((out[k] == 0).all() for k in ("dweight", "dbias", "dscale"))
