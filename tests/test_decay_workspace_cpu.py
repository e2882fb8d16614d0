"""Sizes of the decayed calls' workspace."""
import pytest
import torch

from linear_token_mixer_gb300 import build as B_
from linear_token_mixer_gb300 import fw

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def library():
    B_.build()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,T", [(4, 8, 2048), (1, 3, 65), (2, 8, 1023)])
def test_fp32_scans_keep_one_state_a_chunk(B, H, T, d):
    """The forward scan's; in the backward pass those of two scans, the second of which the third reads."""
    one = B * H * ((T + 63) // 64) * d * d * 4
    assert fw.decay_workspace(B, H, T, d, F32) == one
    assert fw.decay_workspace(B, H, T, d, F32, backward=True) == 2 * one


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [1, 63, 64])
def test_fp32_chains_of_one_chunk_keep_none(T, d):
    assert fw.decay_workspace(3, 5, T, d, F32) == 0
    assert fw.decay_workspace(3, 5, T, d, F32, backward=True) == 0


@pytest.mark.parametrize("d", [64, 128])
def test_bf16_scans_keep_the_states_of_segments(d):
    """None where chains fill the GPU; else a state a segment (the last one's place holds S0's copy), for
    the forward scan of a backward pass and for the two reverse ones, which have no more segments each."""
    assert fw.decay_workspace(8, 16, 4096, d, BF16) == fw.decay_workspace(8, 16, 4096, d, BF16, backward=True) == 0
    fwd = fw.decay_workspace(1, 3, 20000, d, BF16)
    both = fw.decay_workspace(1, 3, 20000, d, BF16, backward=True)
    state = 3 * d * d * 4
    assert fwd % state == 0 and both % state == 0 and fwd >= 2 * state
    assert fwd < both <= 3 * fwd
