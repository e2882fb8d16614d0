"""Layer norm on the GPU against 64 bits.

Tolerances (relative L2).  fp32: a row's sums have at most log2(threads) + width/threads rounded
additions; with random signs, and the centred second pass, about sqrt(64) 2^-24 = 5e-7 on the
statistics and a few 2^-24 on each element: 3e-6.  bf16 rows: the same before one rounding of at
most 2^-8 relative: 2^-8 = 3.9e-3.  dw, db are fp32 sums over the rows of terms of random sign,
each with a few roundings: 3e-6 as well, times sqrt(rows) where the sum itself cancels to the size
of its terms' root sum of squares (it is compared as a vector over the columns, so it does not).
"""
import pytest
import torch

from linear_token_mixer_gb300 import fw
from linear_token_mixer_gb300 import inputs as I

import decay_ref as R

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TOL = {F32: 3e-6, BF16: 2.0 ** -8}
WIDTHS = [1, 2, 7, 8, 31, 32, 33, 64, 100, 128, 129, 200, 256, 512, 520, 1000, 1023, 1024, 2048,
          2056, 4095, 4096, 5000, 8191, 8192, 16384, 16392, 20001, 33000]


def rows_for(width):
    return 3 if width > 8000 else 70


def make(rows, width, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    mu = torch.randn(rows, 1, generator=g)
    x = (torch.randn(rows, width, generator=g) + mu).to(dtype)
    dy = torch.randn(rows, width, generator=g).to(dtype)
    return x, dy, torch.randn(width, generator=g), torch.randn(width, generator=g)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("width", WIDTHS)
def test_forward_and_backward(width, dtype):
    x, dy, w, b = make(rows_for(width), width, dtype, seed=width)
    eps = 1e-2 if width < 8 else 1e-5      # few columns: keep the variance off zero
    y, mean, rstd = fw.layer_norm(x.cuda(), w.cuda(), b.cuda(), eps=eps)
    ry, rm, rr = R.layer_norm(x, w, b, eps)
    assert y.dtype == dtype and R.rel(y, ry) <= TOL[dtype]
    assert R.rel(mean, rm) <= TOL[F32] and R.rel(rstd, rr) <= TOL[F32]
    dx, dw, db = fw.layer_norm_backward(dy.cuda(), x.cuda(), w.cuda(), mean, rstd)
    rdx, rdw, rdb = R.layer_norm_backward(dy, x, w, eps)
    if width > 2:                          # of one or two columns dx is a difference of equals
        assert R.rel(dx, rdx) <= TOL[dtype]
    assert R.rel(dw, rdw) <= TOL[F32] or width == 1
    assert R.rel(db, rdb) <= TOL[F32]


@pytest.mark.parametrize("width", [1, 2])
def test_the_narrowest_rows(width):
    """One column: y = bias and dx = 0 exactly; two: dx is small against dy / sqrt(var)."""
    x, dy, w, b = make(50, width, F32, seed=1)
    y, mean, rstd = fw.layer_norm(x.cuda(), w.cuda(), b.cuda(), eps=0.5)
    dx, dw, db = fw.layer_norm_backward(dy.cuda(), x.cuda(), w.cuda(), mean, rstd)
    rdx, rdw, _ = R.layer_norm_backward(dy, x, w, 0.5)
    assert (dx.cpu().double() - rdx).abs().max() <= 1e-5
    assert (dw.cpu().double() - rdw).abs().max() <= 1e-4
    if width == 1:
        assert torch.equal(y.cpu(), b.expand(50, 1))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 607, 608, 609, 5000])
@pytest.mark.parametrize("width", [64, 77, 384])
def test_row_counts(rows, width, dtype):
    x, dy, w, b = make(rows, width, dtype, seed=rows)
    y, mean, rstd = fw.layer_norm(x.cuda(), w.cuda(), b.cuda())
    dx, dw, db = fw.layer_norm_backward(dy.cuda(), x.cuda(), w.cuda(), mean, rstd)
    rdx, rdw, rdb = R.layer_norm_backward(dy, x, w)
    assert R.rel(y, R.layer_norm(x, w, b)[0]) <= TOL[dtype]
    assert R.rel(dx, rdx) <= TOL[dtype]
    assert R.rel(dw, rdw) <= TOL[F32] and R.rel(db, rdb) <= TOL[F32]


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_without_weight_or_bias(dtype):
    x, dy, w, b = make(40, 96, dtype)
    for ww, bb in ((None, None), (w, None), (None, b)):
        c = lambda t: None if t is None else t.cuda()  # noqa: E731
        y, mean, rstd = fw.layer_norm(x.cuda(), c(ww), c(bb))
        assert R.rel(y, R.layer_norm(x, ww, bb)[0]) <= TOL[dtype]
        dx, _, _ = fw.layer_norm_backward(dy.cuda(), x.cuda(), c(ww), mean, rstd)
        assert R.rel(dx, R.layer_norm_backward(dy, x, ww)[0]) <= TOL[dtype]
    y, mean, rstd = fw.layer_norm(x.cuda(), stats=False)
    assert mean is None and rstd is None


@pytest.mark.parametrize("width", [256, 1000, 40000])
def test_a_large_mean_costs_nothing(width):
    """Values of 1000 with a spread of 1: E[x^2] - E[x]^2 would lose the variance."""
    g = torch.Generator().manual_seed(1)
    x = 1000 + torch.randn(9, width, generator=g)
    y, _, _ = fw.layer_norm(x.cuda())
    # x itself has steps of 2^-14 there, and the mean one of half that: absolute, not relative
    assert (y.cpu().double() - R.layer_norm(x)[0]).abs().max() <= 4 * 2.0 ** -14


def test_constant_rows_and_non_finite_rows_stay_apart():
    x = torch.randn(6, 128)
    x[1] = 3.0
    x[2, 5] = float("nan")
    x[4, 7] = float("inf")
    y, mean, rstd = fw.layer_norm(x.cuda())
    y = y.cpu()
    assert torch.equal(y[1], torch.zeros(128))
    assert torch.isnan(y[2]).all() and not torch.isfinite(y[4]).any()
    ok = [0, 3, 5]
    assert R.rel(y[ok], R.layer_norm(x[ok])[0]) <= TOL[F32]


@pytest.mark.parametrize("width", [128, 130, 2048, 40000])
def test_in_place(width):
    x, dy, w, b = make(20, width, BF16, seed=2)
    xc = x.cuda()
    want, mean, rstd = fw.layer_norm(xc, w.cuda(), b.cuda())
    got = xc.clone()
    fw.layer_norm(got, w.cuda(), b.cuda(), y=got)
    assert torch.equal(got, want)
    ref = fw.layer_norm_backward(dy.cuda(), xc, w.cuda(), mean, rstd)
    for alias in ("dy", "x"):
        g, z = dy.cuda(), xc.clone()
        dx, dw, db = fw.layer_norm_backward(g, z, w.cuda(), mean, rstd, dx=g if alias == "dy" else z)
        assert all(torch.equal(a, c) for a, c in zip((dx, dw, db), ref))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,width", [(150001, 64), (70001, 136), (30001, 520), (9001, 2040), (6001, 4104),
                                        (3001, 8184)])
def test_many_rows_a_block(rows, width, dtype):
    """Blocks that take many rows, some ahead of the others, in place as well; the widths fill the last
    vectors of a row in part.  The tolerances are those above: a thread adds up a few hundred rows of
    random signs, whose roundings grow like the sums."""
    x, dy, w, b = (t.cuda() for t in make(rows, width, dtype, seed=width))
    y, mean, rstd = fw.layer_norm(x, w, b)
    dx, dw, db = fw.layer_norm_backward(dy, x, w, mean, rstd)
    assert R.rel(y, R.layer_norm(x, w, b)[0]) <= TOL[dtype]
    rdx, rdw, rdb = R.layer_norm_backward(dy, x, w)
    assert R.rel(dx, rdx) <= TOL[dtype]
    assert R.rel(dw, rdw) <= TOL[F32] and R.rel(db, rdb) <= TOL[F32]
    z = x.clone()
    fw.layer_norm(z, w, b, y=z)
    assert torch.equal(z, y)
    g, z = dy.clone(), x.clone()
    for args, buf in (((g, x), g), ((dy, z), z)):
        got = fw.layer_norm_backward(*args, w, mean, rstd, dx=buf)
        assert all(torch.equal(a, c) for a, c in zip(got, (dx, dw, db)))


def test_same_bits_on_every_run_and_in_a_graph():
    x, dy, w, b = (t.cuda() for t in make(3000, 640, BF16, seed=4))
    run = lambda: [*fw.layer_norm(x, w, b)] + [*fw.layer_norm_backward(  # noqa: E731
        dy, x, w, *fw.layer_norm(x, w, b)[1:])]
    want = run()
    for _ in range(3):
        assert all(torch.equal(a, c) for a, c in zip(run(), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(outs, want))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_norm_of_the_other_paths(dtype):
    """prefill, step, window_prefill and window_step take the same output norm."""
    w = I.WORKLOADS["falcon1_bf16"].with_shape(B=1, H=2, T=70, dtype=dtype)
    x = {k: (t.cuda() if t is not None else None) for k, t in I.prefill_inputs(w).items()}
    g = torch.Generator().manual_seed(0)
    nw, nb = torch.randn(128, generator=g).cuda(), torch.randn(128, generator=g).cuda()
    args = (x["q"], x["k"], x["v"], x["beta"], x["lam"])
    for call in (lambda **k: fw.prefill(*args, x["S0"], **k)[0],
                 lambda **k: fw.prefill(*args, x["S0"], noalloc=True, **k)[0],
                 lambda **k: fw.window_prefill(*args, 3, x["S0"], **k)[0],
                 lambda **k: fw.step(*(t[:, :, 0].contiguous() for t in args), x["S0"].clone(), **k),
                 lambda **k: fw.window_step(*(t[:, :, 0].contiguous() for t in args),
                                            x["S0"].clone(), 3, **k)[0]):
        o, y = call(), call(norm=(nw, nb), norm_eps=1e-4)
        assert R.rel(y, R.layer_norm(o, nw, nb, 1e-4)[0]) <= TOL[dtype]


def test_offsets_beyond_32_bits():
    rows, width = 2 ** 24 + 9, 128
    gen = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn(rows, width, device="cuda", dtype=BF16, generator=gen)
    dy = torch.randn(rows, width, device="cuda", dtype=BF16, generator=gen)
    w = torch.randn(width, device="cuda", generator=gen)
    y, mean, rstd = fw.layer_norm(x, w)
    dx, dw, db = fw.layer_norm_backward(dy, x, w, mean, rstd)
    tail = slice(rows - 300, rows)
    assert R.rel(y[tail], R.layer_norm(x[tail], w)[0]) <= TOL[BF16]
    assert R.rel(dx[tail], R.layer_norm_backward(dy[tail], x[tail], w)[0]) <= TOL[BF16]
    assert R.rel(mean[tail], R.layer_norm(x[tail])[1]) <= 10 * TOL[F32]   # means near zero
    # fp32 sums of 2^24 terms over 608 x 2 or more partial sums of at most 14000 terms each
    rdb = dy.double().sum(0).cpu()
    assert R.rel(db, rdb) <= 14000 ** 0.5 * 2.0 ** -24 * 4
