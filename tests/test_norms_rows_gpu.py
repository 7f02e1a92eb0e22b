"""The norms of a block where the other tests do not go: more rows than a
gradient's workgroups at every width (so that each passes over several rows), x
as a slice of wider rows, and gates that are infinite (needs MI355X). Bounds as
in test_norms_gpu.py."""
import pytest
import torch

import selective_state_space_16_amd as ssm
import test_norms_gpu as norms
from block_util import gate_norm_reference
from gpu_util import say
from test_norms_gpu import BF, FL, gate_inputs, near

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,wide", [(BF, True), (BF, False), (FL, True)])
@pytest.mark.parametrize("rows,D", [(1030, 1537), (1100, 2048), (1030, 2304), (1030, 2561), (600, 4100), (600, 5128), (530, 8192),
                                    (530, 9001)])
def test_add_norm_over_many_rows(rows, D, dtype, wide):
    norms.test_add_norm(rows, D, dtype, wide)
    norms.test_add_norm_gradient(rows, D, dtype, wide)


@pytest.mark.parametrize("dtype", [BF, FL])
@pytest.mark.parametrize("groups", [1, 2])
@pytest.mark.parametrize("rows,D", [(1030, 1537), (1100, 2048), (1030, 2304), (600, 4100), (600, 5128), (530, 8192)])
def test_gate_norm_over_many_rows(rows, D, groups, dtype):
    norms.test_gate_norm(rows, D, groups, dtype)


@pytest.mark.parametrize("dtype", [BF, FL])
@pytest.mark.parametrize("wide,off", [(1032, 8), (1600, 512), (523, 0)])
def test_x_as_a_slice(wide, off, dtype):
    """x (and z) with rows apart, in both passes."""
    say(f"case x apart {wide} {dtype}")
    rows, D = 41, 512
    d = gate_inputs(rows, D, dtype, 61)
    g = {k: v.cuda() for k, v in d.items()}
    x, z = (torch.full((rows, wide), 9.0, dtype=dtype, device="cuda")[:, off:off + D] for _ in range(2))
    x.copy_(g["x"])
    z.copy_(g["z"])
    y = ssm.ssm_gate_norm_fwd(x, z, g["weight"], groups=2)
    yr = gate_norm_reference(d["x"], d["z"], d["weight"], 2, 1e-5)
    near(y, yr, yr.abs(), 48, "y")
    out = ssm.ssm_gate_norm_bwd(g["dy"], x, z, g["weight"], groups=2)
    ref = ssm.ssm_gate_norm_bwd(g["dy"], g["x"], g["z"], g["weight"], groups=2)
    tol = 0 if wide % 8 == 0 else 4 * torch.finfo(dtype).eps / 2  # another order of the row's sum
    for k in ("dx", "dz", "dweight"):
        assert (out[k].double() - ref[k].double()).abs().max() <= tol * ref[k].double().abs().max(), k


@pytest.mark.parametrize("dtype", [BF, FL])
def test_infinite_gates(dtype):
    """z / (1 + exp(-z)) of minus infinity is infinity times nothing, NaN, and of
    infinity is infinite, whose row has no norm: NaN in both rows, as the
    definition gives, and nowhere else."""
    say(f"case infinite gates {dtype}")
    d = gate_inputs(6, 192, dtype, 62)
    d["z"][2, 5], d["z"][4, 190] = -float("inf"), float("inf")
    g = {k: v.cuda() for k, v in d.items()}
    y = ssm.ssm_gate_norm_fwd(g["x"], g["z"], g["weight"]).cpu()
    yr = gate_norm_reference(d["x"], d["z"], d["weight"], 1, 1e-5)
    ok = [0, 1, 3, 5]
    assert torch.isnan(y[2]).all() and torch.isnan(yr[2]).all() and torch.isnan(y[4, 190]) and torch.isnan(yr[4, 190])
    near(y[ok], yr[ok], yr[ok].abs(), 48, "other rows")
    out = ssm.ssm_gate_norm_bwd(g["dy"], g["x"], g["z"], g["weight"])
    assert torch.isfinite(out["dx"][ok]).all() and torch.isfinite(out["dz"][ok]).all()
