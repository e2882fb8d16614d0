"""The largest shapes that the convolution's calls take, on either side of each bound: what is refused is refused by its
shape, and what is not gets as far as asking for a GPU.  (Made-up addresses, far apart.)"""
import ctypes

import pytest
import torch

from linear_token_mixer_gb300 import build as B_
from linear_token_mixer_gb300 import fw

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses")

P = [(i + 1) << 46 for i in range(12)]
SHAPE_ERR = -2


@pytest.fixture(scope="module")
def L():
    B_.build()
    return fw.lib()


def _codes(L, B, H, T, d, width=4):
    """(prefill, backward, workspace, step or None) of a shape."""
    s = ctypes.byref(fw.fw_shape(B, H, T, d, d))
    step = L.fw_conv_step(P[0], P[1], P[2], P[3], P[5], s, width, 0, 0, None) if T == 1 else None
    return (L.fw_conv_prefill(P[0], P[1], P[2], P[3], None, P[5], P[6], s, width, 0, 0, None),
            L.fw_conv_backward(P[4], P[0], P[1], P[2], P[3], None, P[7], P[5], P[8], P[9], P[10], s, width, 0, 0, P[11],
                               1 << 45, None), L.fw_conv_workspace(s, width), step)


@pytest.mark.parametrize("shape,forward,backward", [
    ((1, 32, 1, 65536), True, False), ((1, 31, 1, 65536), True, True),        # H ceil(d / 32)
    ((1, 1, 1, 65535 * 32), True, True), ((1, 1, 1, 65535 * 32 + 1), True, False),
    ((1, 1, 1, 1 << 24), True, False), ((1, 1, 1, (1 << 24) + 1), False, False),   # d
    ((1023, 32, 1, 65536), True, False), ((1024, 32, 1, 65536), False, False),     # B H d ceil(T / 8)
    ((1, 1, 8 * 32767, 65536), True, True), ((1, 1, 8 * 32767 + 1, 65536), False, False),
    ((32767, 65535, 1, 1), True, True), ((32769, 65535, 1, 1), False, False), ((1, 65536, 1, 1), False, False),   # H
    ((1, 1, 2**31 - 4097, 1), True, True), ((1, 1, 2**31 - 4096, 1), False, False)])   # T
def test_the_bounds_of_a_shape(L, shape, forward, backward):
    prefill, grads, workspace, step = _codes(L, *shape)
    assert (prefill != SHAPE_ERR) == forward and (step is None or step == prefill)
    assert (grads != SHAPE_ERR) == backward and (workspace > 0) == backward
    for code in (prefill, grads):
        assert code in (SHAPE_ERR, -10, -8, -6), code                        # a shape, or no GPU
