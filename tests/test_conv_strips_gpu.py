"""The convolution's gradients where a thread takes several strips, one after the other: its windows begin anew and its sums
of the taps' gradients go on."""
import pytest
import torch

from test_conv_gpu import BF16, F32, check, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("W", [4, 8])
@pytest.mark.parametrize("B,H,T,d,ragged", [(96, 10, 13, 1024, True), (40, 20, 13, 257, True), (64, 80, 9, 130, False),
                                            (3, 160, 600, 40, True)])
def test_several_strips_a_thread(B, H, T, d, ragged, W, dtype):
    x, g = inputs(B, H, T, d, W, dtype, seed=W)
    lens = None
    if ragged:
        lens = torch.randint(0, T + 1, (B,), generator=torch.Generator().manual_seed(d), dtype=torch.int32)
        lens[:3] = torch.tensor([1, T + 5, 0], dtype=torch.int32)
    check(x, g, dtype, lens=lens)
    check(x, g, dtype, silu=False, bias=False, state=False, lens=lens)
