"""The workspace of a selective prompt: what is written."""
import pytest
import torch

from linear_token_mixer_gb300 import build as B_
from linear_token_mixer_gb300 import fw


@pytest.mark.parametrize("B,H,T,d", [(1, 4, 300, 64), (3, 200, 65, 128), (2, 100, 129, 64), (1, 201, 200, 128)])
def test_bytes_of_a_workspace(B, H, T, d):
    B_.build()
    # fp32: a state and a decay (16 bytes apart) for each chunk of 64 tokens
    assert fw.select_workspace(B, H, T, d, torch.float32) == B * H * -(-T // 64) * (d * d * 4 + 16)
    # bf16, chunks of 128 tokens, chains in one piece: a token's log, step and weight, a chunk's decay and log (in whole
    # pairs of chunks), its blocks' logs
    n = B * H * -(-T // 128)
    assert fw.select_workspace(B, H, T, d) == n * (128 * 12 + 16) + (n + n % 2) * 8


@pytest.mark.parametrize("B,H,T,d,pieces", [(1, 8, 4096, 128, 4), (1, 8, 16384, 128, 10), (1, 16, 2048, 128, 4), (1, 32, 32768, 128, 4),
                                            (2, 32, 4096, 128, 2), (1, 16, 640, 128, 1), (2, 64, 32768, 128, 1),
                                            (1, 8, 4096, 64, 8), (1, 16, 2048, 64, 4), (2, 32, 8192, 64, 2)])
def test_pieces_of_a_chain(B, H, T, d, pieces):
    """Few chains go in as many pieces at once as was measured best for this scan; a state of each is in the workspace."""
    B_.build()
    n = B * H * -(-T // 128)
    states = fw.select_workspace(B, H, T, d) - n * (128 * 12 + 16) - (n + n % 2) * 8
    assert states == (B * H * pieces * d * d * 4 if pieces > 1 else 0)
