"""Layer norm's gradients in a workspace of exactly the size that is asked for, between guards.  Tolerances as for
the other layer norm tests (relative L2): fp32 results 3e-6, rows rounded to bf16 2^-8."""
import pytest
import torch

from linear_token_mixer_gb300 import fw

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def rel(a, r):
    assert torch.isfinite(a).all()
    return ((a.double() - r).norm() / r.norm()).item()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,width", [(1, 16384), (700, 16384), (700, 16385), (700, 16392), (1, 20000), (5, 20001),
                                        (1000, 20000), (700, 155648), (700, 155649), (2, 2 ** 21 + 1), (3000, 64)])
def test_exactly_the_size_that_is_asked_for(rows, width, dtype):
    gen = torch.Generator(device="cuda").manual_seed(width)
    x = torch.randn(rows, width, generator=gen, device="cuda").to(dtype)
    dy = torch.randn(rows, width, generator=gen, device="cuda").to(dtype)
    w = torch.randn(width, generator=gen, device="cuda")
    _, mean, rstd = fw.layer_norm(x, w)
    n, guard = fw.lib().fw_layer_norm_workspace(rows, width), 4096
    room = torch.full((n + 2 * guard,), 0x5a, dtype=torch.uint8, device="cuda")
    dx, dw, db = fw.layer_norm_backward(dy, x, w, mean, rstd, workspace=room[guard:guard + n])
    assert (room[:guard] == 0x5a).all() and (room[guard + n:] == 0x5a).all()
    xd, g = x.double(), dy.double()
    m = xd.mean(1, keepdim=True)
    r = torch.rsqrt(((xd - m) ** 2).mean(1, keepdim=True) + 1e-5)
    xd = (xd - m) * r
    assert rel(dw, (g * xd).sum(0)) <= 3e-6 and rel(db, g.sum(0)) <= 3e-6
    g *= w.double()
    want = r * (g - g.mean(1, keepdim=True) - xd * (g * xd).mean(1, keepdim=True))
    assert rel(dx, want) <= (3e-6 if dtype == F32 else 2.0 ** -8)
