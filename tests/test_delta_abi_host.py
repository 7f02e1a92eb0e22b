"""Argument checks of the gated delta rule, the convolution on a cache and the layer
norm, in the C ABI and in the binding (CPU only; every refusal comes before any HIP
call)."""
import pytest
import torch

import selective_state_space_16_amd as ssm

P16, MIS, MIS2 = 0x10000, 0x10004, 0x10001
BIG = 1 << 40


def rows(a):
    return [a[k] for k in ("num_slots", "q", "qs", "k", "ks", "v", "vs", "dt", "ds", "bias", "be", "bs", "A", "scale", "eps", "st", "y")]


BASE = dict(num_slots=8, q=P16, qs=256, k=P16, ks=256, v=P16, vs=256, dt=P16, ds=8, bias=None, be=P16, bs=8, A=P16, scale=0.1, eps=1e-6,
            st=P16, y=P16)


def fwd(**kw):
    a = dict(BASE, seqs=2, rows=100, H=4, P=64, G=2, N=128, dtype=1, cu=P16, slots=P16, resume=None, ws=P16, wsb=BIG)
    a.update(kw)
    return ssm.lib().ssm_delta_fwd_cache(*[a[k] for k in ("seqs", "rows", "H", "P", "G", "N", "dtype", "cu", "slots", "resume")],
                                         *rows(a), a["ws"], a["wsb"], None)


def step(**kw):
    a = dict(BASE, batch=2, H=4, P=64, G=2, N=128, dtype=0, slots=P16)
    a.update(kw)
    return ssm.lib().ssm_delta_step_cache(*[a[k] for k in ("batch", "H", "P", "G", "N", "dtype", "slots")], *rows(a), None)


SHARED = [
    (dict(H=-1), -2), (dict(num_slots=-1), -2), (dict(qs=-8), -2), (dict(ks=248), -2), (dict(vs=255), -2), (dict(ds=3), -2), (dict(bs=3), -2),
    (dict(dtype=3), -3), (dict(P=32), -4), (dict(P=80), -4), (dict(P=320), -4), (dict(P=0), -4), (dict(N=16), -4), (dict(N=256), -4),
    (dict(G=3), -2), (dict(G=0), -2), (dict(qs=1 << 23), -4), (dict(vs=1 << 23), -4), (dict(bs=1 << 23), -4), (dict(H=1 << 16, G=1), -4),
    (dict(H=1 << 20, G=1), -4), (dict(num_slots=1 << 31), -2), (dict(num_slots=(1 << 31) - 1, H=4096, vs=1 << 20, ds=4096, bs=4096), -2),
    (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(dt=None), -1), (dict(be=None), -1), (dict(A=None), -1),
    (dict(st=None), -1), (dict(y=None), -1), (dict(slots=None), -1), (dict(q=MIS), -5), (dict(v=MIS), -5), (dict(st=MIS), -5),
    (dict(bias=MIS), -5), (dict(slots=MIS), -5), (dict(dt=MIS2), -5), (dict(be=MIS2), -5), (dict(y=MIS), -5),
]


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(seqs=-1), -2), (dict(rows=-1), -2), (dict(dtype=0), -4), (dict(seqs=65536), -4), (dict(rows=1 << 31), -4), (dict(cu=None), -1),
    (dict(resume=MIS), -5), (dict(qs=257), -5), (dict(ks=260), -5), (dict(vs=259), -5), (dict(ws=None), -6), (dict(wsb=16), -6), (dict(ws=MIS), -5),
    (dict(rows=(1 << 31) - 1), -4)])
def test_prompt_refusals(kw, code):
    assert fwd(**kw) == code


@pytest.mark.parametrize("kw,code", SHARED + [(dict(batch=-1), -2), (dict(batch=65536), -4), (dict(qs=258), -5), (dict(vs=257), -5),
                                              (dict(batch=65535, H=1024, G=1, vs=1 << 20, ds=1024, bs=1024), -4)])
def test_step_refusals(kw, code):
    assert step(**kw) == code


def test_empty_calls_launch_nothing():
    assert fwd(seqs=0, ws=None, wsb=0) == 0 and fwd(H=0, G=1, ws=None) == 0
    assert step(batch=0) == 0 and step(H=0, G=1) == 0
    assert conv(seqs=0) == 0 and conv(C=0) == 0 and conv_step(batch=0) == 0
    assert ln(rows=0) == 0 and ln(D=0) == 0 and ln_bwd(D=0) == 0


def test_gates_need_their_element_alignment_only():
    """Refused further on, so past the alignment: no workspace."""
    assert fwd(dt=0x10002, be=0x10006, ws=None) == -6


def test_workspace_sizes():
    f = ssm.ssm_delta_fwd_cache_workspace_bytes
    assert f(2, 100, 4, 64, 2, 128, 1) > 0
    for bad in ((0, 100, 4, 64, 2, 128, 1), (-1, 100, 4, 64, 2, 128, 1), (2, -1, 4, 64, 2, 128, 1), (2, 100, 4, 63, 2, 128, 1),
                (2, 100, 4, 64, 3, 128, 1), (2, 100, 4, 64, 0, 128, 1), (2, 100, 4, 64, 2, 128, 0), (2, 100, 0, 64, 2, 128, 1),
                (65536, 100, 4, 64, 2, 128, 1), (2, 1 << 31, 4, 64, 2, 128, 1)):
        assert f(*bad) == 0
    for H, P, G, N in ((4, 64, 2, 128), (24, 64, 24, 64), (32, 128, 16, 128)):
        sizes = [[f(s, r, H, P, G, N, 1) for r in (0, 1, 63, 64, 65, 1000, 5000, 40000)] for s in (1, 2, 9, 100, 3000)]
        for row in sizes:
            assert row == sorted(row)
        for a, b in zip(sizes, sizes[1:]):
            assert all(x <= y for x, y in zip(a, b))
    g = ssm.ssm_add_layer_norm_bwd_workspace_bytes
    assert g(0, 8) == 0 and g(8, 0) == 0 and g(-1, 8) == 0 and g(1, 8) == 96 and g(1 << 40, 64) == 512 * 3 * 64 * 4
    assert g(1 << 40, 1 << 40) == 0


def conv(**kw):
    a = dict(seqs=2, rows=100, C=64, dtype=1, cu=P16, slots=P16, resume=None, num_slots=8, x=P16, xs=64, w=P16, b=None, win=P16, y=P16)
    a.update(kw)
    return ssm.lib().ssm_conv_fwd_cache(*[a[k] for k in ("seqs", "rows", "C", "dtype", "cu", "slots", "resume", "num_slots", "x", "xs", "w",
                                                         "b", "win", "y")], None)


def conv_step(**kw):
    a = dict(batch=2, C=64, dtype=1, slots=P16, num_slots=8, x=P16, xs=64, w=P16, b=None, win=P16, y=P16)
    a.update(kw)
    return ssm.lib().ssm_conv_step_cache(*[a[k] for k in ("batch", "C", "dtype", "slots", "num_slots", "x", "xs", "w", "b", "win", "y")], None)


CONV = [(dict(C=-1), -2), (dict(num_slots=-1), -2), (dict(dtype=2), -3), (dict(C=1 << 23, xs=1 << 23), -4), (dict(xs=63), -2),
        (dict(xs=1 << 23), -4), (dict(num_slots=1 << 31), -2), (dict(num_slots=(1 << 31) - 1, C=1 << 20, xs=1 << 20), -2), (dict(x=None), -1),
        (dict(w=None), -1), (dict(win=None), -1), (dict(y=None), -1), (dict(slots=None), -1), (dict(x=MIS), -5), (dict(b=MIS), -5),
        (dict(win=MIS), -5), (dict(y=MIS), -5)]


@pytest.mark.parametrize("kw,code", CONV + [(dict(seqs=-1), -2), (dict(rows=-1), -2), (dict(seqs=65536), -4), (dict(rows=1 << 31), -4),
                                            (dict(cu=None), -1), (dict(resume=MIS), -5), (dict(rows=(1 << 31) - 1), -4)])
def test_conv_refusals(kw, code):
    assert conv(**kw) == code


@pytest.mark.parametrize("kw,code", CONV + [(dict(batch=-1), -2), (dict(batch=65536), -4), (dict(batch=65535, C=1 << 20, xs=1 << 20), -4)])
def test_conv_step_refusals(kw, code):
    assert conv_step(**kw) == code


def ln(**kw):
    a = dict(rows=4, D=64, dtype=1, res=0, x=P16, r=P16, s=None, w=P16, b=None, y=P16, ro=P16)
    a.update(kw)
    return ssm.lib().ssm_add_layer_norm_fwd(a["rows"], a["D"], a["dtype"], a["res"], a["x"], a["r"], a["s"], a["w"], a["b"], 1e-5, a["y"], a["ro"], None)


def ln_bwd(**kw):
    a = dict(rows=4, D=64, dtype=1, res=0, dy=P16, r=P16, w=P16, x=None, s=None, dres=None, dx=P16, dr=P16, dw=P16, db=P16, ds=None, ws=P16, wsb=BIG)
    a.update(kw)
    return ssm.lib().ssm_add_layer_norm_bwd(*[a[k] for k in ("rows", "D", "dtype", "res", "dy", "r", "w", "x", "s", "dres")], 1e-5,
                                            *[a[k] for k in ("dx", "dr", "dw", "db", "ds", "ws", "wsb")], None)


NORM = [(dict(rows=-1), -2), (dict(D=-1), -2), (dict(dtype=2), -3), (dict(res=2), -3), (dict(dtype=0, res=1), -3), (dict(D=16385), -4),
        (dict(rows=1 << 45), -2), (dict(w=None), -1), (dict(w=MIS), -5)]


@pytest.mark.parametrize("kw,code", NORM + [(dict(x=None), -1), (dict(y=None), -1), (dict(x=MIS), -5), (dict(b=MIS), -5), (dict(ro=MIS), -5)])
def test_layer_norm_refusals(kw, code):
    assert ln(**kw) == code


@pytest.mark.parametrize("kw,code", NORM + [(dict(dy=None), -1), (dict(r=None), -1), (dict(dx=None), -1), (dict(dw=None), -1), (dict(db=None), -1),
                                            (dict(s=P16), -1), (dict(dr=MIS), -5), (dict(db=MIS), -5), (dict(ws=None), -6), (dict(wsb=64), -6),
                                            (dict(ws=MIS), -5)])
def test_layer_norm_gradient_refusals(kw, code):
    assert ln_bwd(**kw) == code


def test_binding_refuses_cpu_tensors_and_other_shapes():
    z = torch.zeros
    i = z(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        ssm.ssm_delta_step_cache(z(2, 64), z(2, 64), z(2, 64), z(2, 1), z(2, 1), z(1), i, z(2, 1, 64, 64))
    with pytest.raises(ValueError, match="one row per request"):
        ssm.ssm_delta_step_cache(z(3, 64), z(3, 64), z(3, 64), z(3, 1), z(3, 1), z(1), i, z(2, 1, 64, 64))
    with pytest.raises(ValueError, match="does not hold keys"):
        ssm.ssm_delta_fwd_cache(z(3, 65), z(3, 65), z(3, 64), z(3, 1), z(3, 1), z(1), i, i, z(2, 1, 64, 64))
    with pytest.raises(ValueError, match="GPU"):
        ssm.ssm_conv_fwd_cache(z(3, 8), z(8, 4), i, i, z(2, 8, 3))
    with pytest.raises(ValueError, match="one row per request"):
        ssm.ssm_conv_step_cache(z(3, 8), z(8, 4), i, z(2, 8, 3))
    with pytest.raises(ValueError):
        ssm.ssm_conv_fwd_cache(z(3), z(8, 4), i, i, z(2, 8, 3))
    with pytest.raises(ValueError, match="GPU"):
        ssm.ssm_add_layer_norm_fwd(z(3, 8), z(8))
    with pytest.raises(ValueError, match="GPU"):
        ssm.ssm_add_layer_norm_bwd(z(3, 8), z(3, 8), z(8))
    with pytest.raises(TypeError):
        ssm.ssm_add_layer_norm_bwd(z(3, 8), z(3, 8, dtype=torch.float64), z(8))
