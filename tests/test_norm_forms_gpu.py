"""Every form of the layer norm kernels that a width and a number of rows choose, against 64 bits: whole
vectors that fill a row's threads exactly, even widths that no 16-byte vector divides, odd ones, and rows
enough that a block takes several.

Tolerances as for the other layer norm tests (relative L2): 3e-6 for fp32 results, 2^-8 for rows
rounded to bf16.
"""
import pytest
import torch

from linear_token_mixer_gb300 import fw

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TOL = {F32: 3e-6, BF16: 2.0 ** -8}

EXACT = [16, 32, 64, 128, 256, 512, 1024, 2048, 4096, 8192, 16384, 32768]
EVEN = [62, 126, 258, 514, 1026, 2050, 4098, 5370, 8194, 16386]
ODD = [27, 99, 385, 2047, 12001]


def rel(a, r):
    assert torch.isfinite(a).all()
    return ((a.double() - r).norm() / r.norm()).item()


def check(rows, width, dtype, affine):
    gen = torch.Generator(device="cuda").manual_seed(width)
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x, dy = (rn(rows, width) + rn(rows, 1)).to(dtype), rn(rows, width).to(dtype)
    w, b = (rn(width), rn(width)) if affine else (None, None)
    y, mean, rstd = fw.layer_norm(x, w, b)
    dx, dw, db = fw.layer_norm_backward(dy, x, w, mean, rstd)
    xd, g = x.double(), dy.double()
    m = xd.mean(1, keepdim=True)
    r = torch.rsqrt(((xd - m) ** 2).mean(1, keepdim=True) + 1e-5)
    xh = (xd - m) * r
    assert rel(y, xh * w.double() + b.double() if affine else xh) <= TOL[dtype]
    assert rel(mean, m[:, 0]) <= TOL[F32] and rel(rstd, r[:, 0]) <= TOL[F32]
    gw = g * w.double() if affine else g
    want = r * (gw - gw.mean(1, keepdim=True) - xh * (gw * xh).mean(1, keepdim=True))
    assert rel(dx, want) <= TOL[dtype]
    assert rel(dw, (g * xh).sum(0)) <= TOL[F32] and rel(db, g.sum(0)) <= TOL[F32]


@pytest.mark.parametrize("affine", [True, False])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("width", EXACT + EVEN + ODD)
def test_many_rows(width, dtype, affine):
    check(max(1100, min(150001, 2 ** 24 // width + 1)), width, dtype, affine)


@pytest.mark.parametrize("affine", [True, False])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("width", EXACT + EVEN + ODD)
def test_few_rows(width, dtype, affine):
    check(37, width, dtype, affine)
