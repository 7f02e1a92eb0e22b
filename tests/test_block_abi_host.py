"""Argument checks of the operators around the SSD layer, in the C ABI and in
the binding (CPU only; every refusal comes before any HIP call)."""
import pytest
import torch

import selective_state_space_16_amd as ssm

P16, MIS = 0x10000, 0x10004
BIG = 1 << 40


def fwd(**kw):
    a = dict(seqs=2, rows=100, H=4, P=64, G=2, N=128, dtype=1, cu=P16, slots=P16, resume=None, num_slots=8, x=P16, xs=768,
             w=P16, b=None, dt=P16, ds=8, bias=None, A=P16, D=None, win=P16, st=P16, y=P16, ws=P16, wsb=BIG)
    a.update(kw)
    return ssm.lib().ssm_ssd_fwd_cache(*[a[k] for k in ("seqs", "rows", "H", "P", "G", "N", "dtype", "cu", "slots", "resume",
                                                        "num_slots", "x", "xs", "w", "b", "dt", "ds", "bias", "A", "D", "win",
                                                        "st", "y", "ws", "wsb")], None)


def step(**kw):
    a = dict(batch=2, H=4, P=64, G=2, N=128, dtype=0, slots=P16, num_slots=8, x=P16, xs=768, w=P16, b=None, dt=P16, ds=8,
             bias=None, A=P16, D=None, win=P16, st=P16, y=P16, ws=P16, wsb=BIG)
    a.update(kw)
    return ssm.lib().ssm_ssd_step_cache(*[a[k] for k in ("batch", "H", "P", "G", "N", "dtype", "slots", "num_slots", "x", "xs",
                                                         "w", "b", "dt", "ds", "bias", "A", "D", "win", "st", "y", "ws",
                                                         "wsb")], None)


SHARED = [
    (dict(H=-1), -2), (dict(num_slots=-1), -2), (dict(xs=-8), -2), (dict(dtype=3), -3), (dict(P=32), -4), (dict(P=80), -4),
    (dict(P=320), -4), (dict(P=0), -4), (dict(N=16), -4), (dict(N=256), -4), (dict(G=3), -2), (dict(G=0), -2), (dict(xs=760), -2),
    (dict(ds=3), -2), (dict(xs=1 << 23), -4), (dict(ds=1 << 23), -4), (dict(H=1 << 20, G=1), -4), (dict(num_slots=1 << 31), -2),
    (dict(num_slots=(1 << 31) - 1, H=4096, xs=1 << 20), -2), (dict(x=None), -1), (dict(w=None), -1), (dict(A=None), -1),
    (dict(win=None), -1), (dict(st=None), -1), (dict(y=None), -1), (dict(slots=None), -1), (dict(dt=None), -1), (dict(x=MIS), -5),
    (dict(st=MIS), -5), (dict(D=MIS), -5), (dict(slots=MIS), -5), (dict(ws=None), -6), (dict(wsb=16), -6),
]


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(seqs=-1), -2), (dict(rows=-1), -2), (dict(dtype=0), -4), (dict(seqs=65536), -4), (dict(rows=1 << 31), -4),
    (dict(cu=None), -1), (dict(resume=MIS), -5), (dict(xs=771), -5), (dict(xs=772), -5)])
def test_prompt_refusals(kw, code):
    assert fwd(**kw) == code


@pytest.mark.parametrize("kw,code", SHARED + [(dict(batch=-1), -2), (dict(batch=65536), -4), (dict(xs=770), -5)])
def test_step_refusals(kw, code):
    assert step(**kw) == code


def test_empty_calls_launch_nothing():
    assert fwd(seqs=0, ws=None, wsb=0) == 0 and fwd(H=0, G=1, xs=256, ws=None) == 0
    assert step(batch=0, ws=None, wsb=0) == 0 and step(H=0, G=1, xs=256, ws=None) == 0


def test_workspace_sizes():
    f = ssm.ssm_ssd_fwd_cache_workspace_bytes
    assert f(2, 100, 4, 64, 2, 128, 1) > 0
    for bad in ((0, 100, 4, 64, 2, 128, 1), (-1, 100, 4, 64, 2, 128, 1), (2, -1, 4, 64, 2, 128, 1), (2, 100, 4, 63, 2, 128, 1),
                (2, 100, 4, 64, 3, 128, 1), (2, 100, 4, 64, 2, 127, 1), (2, 100, 4, 64, 2, 128, 0), (2, 100, 4, 64, 0, 128, 1)):
        assert f(*bad) == 0
    # more rows or sequences never need less
    assert f(2, 5000, 4, 64, 2, 128, 1) >= f(2, 4999, 4, 64, 2, 128, 1) and f(9, 100, 4, 64, 2, 128, 1) >= f(8, 100, 4, 64, 2, 128, 1)
    s = ssm.ssm_ssd_step_cache_workspace_bytes
    assert s(2, 4, 64, 2, 128) >= 2 * (4 * 64 + 2 * 2 * 128 + 8) * 4
    assert s(0, 4, 64, 2, 128) == 0 and s(2, 4, 48, 2, 128) == 0 and s(2, 4, 64, 3, 128) == 0
    n = ssm.ssm_norm_bwd_workspace_bytes
    assert n(0, 64) == 0 and n(4, 0) == 0 and n(-1, 64) == 0 and n(1, 64) >= 512 and n(10 ** 6, 64) >= n(10, 64)


def add_fwd(**kw):
    a = dict(rows=3, D=64, dtype=1, res=0, x=P16, residual=None, scale=None, w=P16, eps=1e-5, y=P16, r=P16)
    a.update(kw)
    return ssm.lib().ssm_add_norm_fwd(*[a[k] for k in ("rows", "D", "dtype", "res", "x", "residual", "scale", "w", "eps", "y", "r")], None)


def add_bwd(**kw):
    a = dict(rows=3, D=64, dtype=1, res=0, dy=P16, r=P16, w=P16, x=None, scale=None, dres=None, eps=1e-5, dx=P16, dr=P16, dw=P16,
             ds=None, ws=P16, wsb=BIG)
    a.update(kw)
    return ssm.lib().ssm_add_norm_bwd(*[a[k] for k in ("rows", "D", "dtype", "res", "dy", "r", "w", "x", "scale", "dres", "eps", "dx",
                                                       "dr", "dw", "ds", "ws", "wsb")], None)


NORM = [(dict(rows=-1), -2), (dict(D=-1), -2), (dict(dtype=2), -3), (dict(D=1 << 20), -4), (dict(rows=1 << 46), -2), (dict(w=None), -1),
        (dict(w=MIS), -5)]


@pytest.mark.parametrize("kw,code", NORM + [(dict(res=1, dtype=0), -3), (dict(res=2), -3), (dict(D=16385), -4), (dict(x=None), -1),
                                            (dict(y=None), -1), (dict(r=None), -1), (dict(x=MIS), -5), (dict(residual=MIS), -5),
                                            (dict(rows=0), 0), (dict(D=0), 0)])
def test_add_norm_refusals(kw, code):
    assert add_fwd(**kw) == code


@pytest.mark.parametrize("kw,code", NORM + [(dict(res=1, dtype=0), -3), (dict(D=16385), -4), (dict(dy=None), -1), (dict(r=None), -1),
                                            (dict(dx=None), -1), (dict(dr=None), -1), (dict(dw=None), -1), (dict(scale=P16), -1),
                                            (dict(dw=MIS), -5), (dict(ws=None), -6), (dict(wsb=100), -6), (dict(D=0), 0)])
def test_add_norm_gradient_refusals(kw, code):
    assert add_bwd(**kw) == code


def gate_fwd(**kw):
    a = dict(rows=3, D=64, groups=2, dtype=1, x=P16, xs=64, z=P16, zs=192, w=P16, eps=1e-5, y=P16)
    a.update(kw)
    return ssm.lib().ssm_gate_norm_fwd(*[a[k] for k in ("rows", "D", "groups", "dtype", "x", "xs", "z", "zs", "w", "eps", "y")], None)


def gate_bwd(**kw):
    a = dict(rows=3, D=64, groups=2, dtype=1, dy=P16, x=P16, xs=64, z=P16, zs=192, w=P16, eps=1e-5, dx=P16, dz=P16, dzs=64, dw=P16,
             ws=P16, wsb=BIG)
    a.update(kw)
    return ssm.lib().ssm_gate_norm_bwd(*[a[k] for k in ("rows", "D", "groups", "dtype", "dy", "x", "xs", "z", "zs", "w", "eps", "dx",
                                                        "dz", "dzs", "dw", "ws", "wsb")], None)


GATE = [(dict(rows=-1), -2), (dict(groups=0), -2), (dict(groups=3), -2), (dict(groups=-1), -2), (dict(dtype=2), -3), (dict(xs=63), -2),
        (dict(zs=63), -2), (dict(zs=1 << 46), -2), (dict(D=32770, xs=32770, zs=32770, dzs=32770), -4),
        (dict(D=1 << 17, groups=1 << 17, xs=1 << 17, zs=1 << 17, dzs=1 << 17), -4), (dict(x=None), -1), (dict(z=None), -1),
        (dict(w=None), -1), (dict(z=MIS), -5)]


@pytest.mark.parametrize("kw,code", [(dict(k, **{}), c) for k, c in GATE] + [(dict(y=None), -1), (dict(y=MIS), -5), (dict(rows=0), 0)])
def test_gate_norm_refusals(kw, code):
    kw = {k: v for k, v in kw.items() if k != "dzs"}
    assert gate_fwd(**kw) == code


@pytest.mark.parametrize("kw,code", GATE + [(dict(dzs=63), -2), (dict(dx=None), -1), (dict(dz=None), -1), (dict(dw=None), -1),
                                            (dict(dx=MIS), -5), (dict(ws=None), -6), (dict(wsb=8), -6)])
def test_gate_norm_gradient_refusals(kw, code):
    assert gate_bwd(**kw) == code


def test_binding_refuses_cpu_tensors():
    x, w = torch.zeros(3, 64), torch.ones(64)
    for f in (lambda: ssm.ssm_add_norm_fwd(x, w), lambda: ssm.ssm_gate_norm_fwd(x, x, w),
              lambda: ssm.ssm_gate_norm_bwd(x, x, x, w), lambda: ssm.ssm_add_norm_bwd(x, x, w)):
        with pytest.raises((ValueError, AssertionError, RuntimeError)):
            f()
    i32 = torch.int32
    with pytest.raises(ValueError):
        ssm.ssm_ssd_step_cache(torch.zeros(2, 64 + 256), torch.zeros(2, 1), -torch.ones(1), torch.zeros(320, 4),
                               torch.zeros(2, dtype=i32), torch.zeros(3, 320, 3), torch.zeros(3, 1, 64, 128))
    with pytest.raises(ValueError):  # a row that does not hold whole groups
        ssm.ssm_ssd_step_cache(torch.zeros(2, 64 + 250), torch.zeros(2, 1), -torch.ones(1), torch.zeros(314, 4),
                               torch.zeros(2, dtype=i32), torch.zeros(3, 314, 3), torch.zeros(3, 1, 64, 128))
    with pytest.raises(TypeError):
        ssm.ssm_add_norm_fwd(torch.zeros(3, 64, dtype=torch.float16), w)


def test_grids_that_no_launch_reaches():
    """Sizes within every other limit whose launches would have 2^32 threads."""
    assert fwd(rows=(1 << 31) - 1, H=1, P=64, G=1, N=128, xs=320) == -4
    assert step(batch=65535, H=16384, G=1, xs=16384 * 64 + 256, ds=16384) == -4
    assert gate_bwd(rows=1, D=1 << 28, groups=1 << 15, xs=1 << 28, zs=1 << 28, dzs=1 << 28) == -4
    assert ssm.ssm_ssd_fwd_cache_workspace_bytes(1, (1 << 31) - 1, 1, 64, 1, 128, 1) == 0
    assert ssm.ssm_ssd_step_cache_workspace_bytes(65535, 16384, 64, 1, 128) == 0
