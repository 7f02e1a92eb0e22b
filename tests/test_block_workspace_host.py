"""Workspace sizes of the operators around the SSD layer over sweeps of sizes (CPU
only): a workspace made for the largest batch serves every smaller one."""
import pytest

import selective_state_space_16_amd as ssm

LAYERS = [(80, 64, 1, 128), (24, 64, 1, 128), (32, 64, 2, 64), (4, 64, 1, 64), (1, 64, 1, 128), (40, 128, 4, 64), (300, 256, 1, 128),
          (3000, 256, 1, 64)]


def prompts(seqs, rows, layer):
    H, P, G, N = layer
    return ssm.ssm_ssd_fwd_cache_workspace_bytes(seqs, rows, H, P, G, N, ssm.SSM_BF16)


@pytest.mark.parametrize("layer", LAYERS)
def test_more_rows_never_need_less(layer):
    for seqs in (1, 2, 3, 8, 19, 20, 50, 51, 52, 255, 256, 257, 258, 1000):
        last = 0
        for rows in [*range(0, 9000, 7), *range(9000, 60000, 61), *range(60000, 1000000, 2711)]:
            need = prompts(seqs, rows, layer)
            if need == 0:
                break  # more than one call takes
            assert need >= last, (seqs, rows)
            last = need


@pytest.mark.parametrize("layer", LAYERS)
def test_more_sequences_never_need_less(layer):
    for rows in (0, 1, 63, 64, 100, 1000, 2753, 2769, 4096, 5000, 16384, 20000, 32768, 100000, 400000):
        last = 0
        for seqs in range(1, 700):
            need = prompts(seqs, rows, layer)
            if need == 0:
                break
            assert need >= last, (seqs, rows)
            last = need


def test_single_tokens_and_gradients():
    last = 0
    for batch in range(1, 3000):
        need = ssm.ssm_ssd_step_cache_workspace_bytes(batch, 24, 64, 1, 128)
        assert need >= last
        last = need
    last = 0
    for rows in range(1, 3000):
        need = ssm.ssm_norm_bwd_workspace_bytes(rows, 520)
        assert need >= last
        last = need


def test_sizes_stay_near_what_the_operands_take():
    """A long prompt through 80 heads: less than 0.5 GB for 16384 tokens, and not
    more than in proportion for eight times as many."""
    one, many = prompts(1, 16384, LAYERS[0]), prompts(1, 131072, LAYERS[0])
    assert one < 0.5e9 and many < 8.5 * one
