"""Packed prompts (ssm_ssd_fwd_cache) where the other tests do not go: more
sequences than the device plans segments for, whole layers of many heads, and
what lies around the tensors of a call with bad offsets (needs MI355X). Bounds
as in test_ssd_cache_gpu.py and test_ssd_cache_output_gpu.py."""
import pytest
import torch

import selective_state_space_16_amd as ssm
from block_util import ssd_inputs, to_gpu, views
from gpu_util import say
from test_ssd_cache_gpu import before, compare, prompt
from test_ssd_cache_output_gpu import output_within

pytestmark = pytest.mark.gpu


def ragged(n, long, seed):
    """n lengths from 0 to 6, one of them `long`."""
    lens = torch.randint(0, 7, (n,), generator=torch.Generator().manual_seed(seed)).tolist()
    lens[n // 2] = long
    return lens


@pytest.mark.parametrize("n,long,H,P,G,N", [(257, 2100, 2, 64, 1, 64), (300, 4200, 1, 64, 1, 128), (300, 130, 4, 128, 2, 64),
                                            (256, 2100, 2, 64, 1, 64), (1100, 65, 1, 64, 1, 64)])
def test_many_sequences(n, long, H, P, G, N):
    """Empty, resumed and short sequences around one that is longer than the longest
    segment, on both sides of the 256 that the device plans for."""
    say(f"case many {n} long={long} H={H} P={P} G={G} N={N}")
    d = ssd_inputs(ragged(n, long, 51), H, P, G, N, seed=52, spare=5)
    g, y0 = to_gpu(d), before(d)
    y = prompt(g, y0.cuda())
    torch.cuda.synchronize()
    compare(d, g, y, y0)


def test_many_sequences_some_left_out():
    """300 sequences, two of which name the slots of earlier ones and one none."""
    say("case many left out")
    d = ssd_inputs(ragged(300, 70, 53), 2, 64, 1, 64, seed=54)
    d["slots"][7], d["slots"][150], d["slots"][299] = d["slots"][3], -1, d["slots"][290]
    g, y0 = to_gpu(d), before(d)
    y = prompt(g, y0.cuda())
    torch.cuda.synchronize()
    compare(d, g, y, y0)


@pytest.mark.parametrize("lens,H,P,G,N", [([130, 0, 70, 1], 80, 64, 1, 128), ([200, 65], 48, 64, 8, 128), ([150, 90], 32, 128, 2, 64)])
def test_whole_layers(lens, H, P, G, N):
    """Every output and state of layers with many heads."""
    say(f"case layer {lens} H={H} P={P} G={G} N={N}")
    d = ssd_inputs(lens, H, P, G, N, seed=55, spare=2)
    g, y0 = to_gpu(d), before(d)
    y = prompt(g, y0.cuda())
    torch.cuda.synchronize()
    compare(d, g, y, y0)
    output_within(d, "layer")


@pytest.mark.parametrize("offsets,covered", [([0, 40, 1000], 80), ([-5, 40, 80], 80), ([0, 60, 30], 60), ([2 ** 31 - 1, -2 ** 31, 50], 50)])
def test_bad_offsets_leave_what_lies_around(offsets, covered):
    """y, both caches and the workspace inside larger buffers: the rows of y that no
    sequence's cut range covers, the slots that none names and the guards keep
    their bits."""
    say(f"case bad offsets {offsets}")
    d = ssd_inputs([40, 40], 2, 64, 1, 64, seed=56, num_slots=4)
    g = to_gpu(d)
    g["cu"] = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    need = ssm.ssm_ssd_fwd_cache_workspace_bytes(2, 80, 2, 64, 1, 64, ssm.SSM_BF16)
    guard = 4096

    def inside(t):
        """A copy of t in the middle of a buffer filled with 3, and that buffer."""
        n = t.numel()
        buf = torch.full((n + 2 * guard,), 3, dtype=t.dtype, device="cuda")
        buf[guard:guard + n] = t.reshape(-1)
        return buf[guard:guard + n].view(t.shape), buf

    y, y_buf = inside(torch.full((80, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda"))
    g["conv_cache"], conv_buf = inside(g["conv_cache"])
    g["state_cache"], state_buf = inside(g["state_cache"])
    ws, ws_buf = inside(torch.zeros(need, dtype=torch.uint8, device="cuda"))
    xBC, _ = views(g)
    prompt(g, y, workspace=ws)
    torch.cuda.synchronize()
    assert xBC.shape[0] == 80 and (y[covered:] == 7).all()
    for t, buf in ((y, y_buf), (g["conv_cache"], conv_buf), (g["state_cache"], state_buf), (ws, ws_buf)):
        assert (buf[:guard] == 3).all() and (buf[guard + t.numel():] == 3).all()
    free = [k for k in range(4) if k not in d["slots"].tolist()]
    assert torch.equal(g["state_cache"][free].cpu(), d["state_cache"][free])
    assert torch.equal(g["conv_cache"][free].cpu(), d["conv_cache"][free])
