"""Gated norm with parameters of each head over batches whose blocks take many rows of a head, from batch row to batch
row: their walk over a group's rows, in steps that are no multiple of a head's rows, and rows shorter than a block's."""
import pytest
import torch

from test_gated_norm_gpu import BF16, F32, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rms,after", [(False, False), (True, True)])
@pytest.mark.parametrize("B,H,T,width", [(6, 16, 1111, 64), (3, 5, 2000, 257), (40, 24, 37, 128), (4000, 2, 3, 64),
                                         (9, 2, 401, 1030)])
def test_batches_of_heads(B, H, T, width, rms, after, dtype):
    gen = torch.Generator().manual_seed(T)

    def rn(*s):
        return torch.randn(*s, generator=gen)

    shape = (B, H, T, width)
    # (a mean and a deviation of each row's own, so that a neighbour's statistics do not pass for a row's)
    x = {"x": ((1 + torch.rand(B, H, T, 1, generator=gen)) * rn(*shape) + rn(B, H, T, 1)).to(dtype),
         "gate": (2 * rn(*shape)).to(dtype), "residual": (3 * rn(*shape)).to(dtype), "weight": 1 + 0.3 * rn(H, width),
         "bias": rn(H, width), "scale": 0.5 + 0.3 * rn(H, width)}
    d = {"dy": rn(*shape).to(dtype), "dtotal": rn(*shape).to(dtype)}
    check(x, d, dtype, rms, after)


def test_the_cases_take_several_turns():
    """Rows of a head, of which blocks on 152 SMs hold at most 3 x 256 / 8 threads' worth at once for each head."""
    for B, H, T, width in [(6, 16, 1111, 64), (3, 5, 2000, 257), (40, 24, 37, 128), (4000, 2, 3, 64), (9, 2, 401, 1030)]:
        threads = 8
        while threads * 8 < width:
            threads *= 2
        at_once = max(152 * 3 // H, 1) * max(256 // threads, 1)
        assert B * T > at_once and B > 1
