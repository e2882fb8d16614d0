"""Gated norm and its gradients on the GPU against the definition in 64 bits.

Tolerances (relative L2 of a whole output).  fp32: u, the product with silu (its exponential and quotient two ulp
each) and the two sums of a row (errors of random sign) are within about 16 2^-24 of their terms, and a gradient
forms such rows and sums twice: 4e-6.  Sums over rows: errors of random sign in fp32 over three levels: 4e-6.
Statistics: 4e-6; a mean may cancel, and is measured against the row's standard deviation.  bf16: a row is rounded once
(2^-8 at most): 4.1e-3 with the fast exponential's few fp32 ulp; sums over rows are of fp32 values: 4e-6.
"""
import pytest
import torch

from linear_token_mixer_gb300 import fw

import mixer_ref as R

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TOL = {F32: 4e-6, BF16: 4.1e-3}
TOL_SUM = 4e-6


def inputs(rows, width, dtype, H=None, seed=0, gate=True, residual=True, params=True):
    """Rows [rows, width], or [rows / H / 3, H, 3, width] with parameters of each head."""
    gen = torch.Generator().manual_seed(seed)

    def rn(*s):
        return torch.randn(*s, generator=gen)

    shape = (rows, width) if H is None else (rows // H // 3, H, 3, width)
    par = (width,) if H is None else (H, width)
    x = {"x": (rn(*shape) * 2 + rn(*shape[:-1], 1)).to(dtype)}
    if gate:
        x["gate"] = (2 * rn(*shape)).to(dtype)
    if residual:
        x["residual"] = (3 * rn(*shape)).to(dtype)
    if params:
        x.update(weight=1 + 0.3 * rn(*par), bias=rn(*par))
        if residual:
            x["scale"] = 0.5 + 0.3 * rn(*par)
    d = {"dy": rn(*shape).to(dtype), "dtotal": rn(*shape).to(dtype)}
    return x, d


def room(x, d, rms, after, eps, want):
    """How many times its tolerance a gradient may be off: 1, but for layer norm of two columns.  There n = (c, -c),
    c^2 = 1 - eps r^2, so that ds = r (g - mean(g) - n mean(g n)) = r (g_1 - g_2) / 2 (1 - c^2): the terms cancel to
    eps r^2 of themselves (1e-5 of a variance of one).  The tolerance is relative to the terms: the quotient
    of their norm and the result's, of each gradient that ds goes into.  One column with rms is the same: n = c,
    ds = r (g - n g n) = r g (1 - c^2)."""
    one = dict.fromkeys(want, 1.0)
    if x["x"].shape[-1] != (1 if rms else 2):
        return one
    z = {n: R.f64(t) for n, t in x.items()}
    _, u, m, r = R.gated(**z, eps=eps, rms=rms, gate_after=after)
    sg = torch.sigmoid(z["gate"])
    act, slope = z["gate"] * sg, sg * (1 + z["gate"] * (1 - sg))
    g = R.f64(d["dy"]) * z["weight"] * (act if after else 1.0)
    n = ((u if after else u * act) - m[..., None]) * r[..., None]
    terms = r[..., None] * (g.abs() + (0.0 if rms else g.mean(-1, keepdim=True).abs()) + (n * (g * n).mean(-1, keepdim=True)).abs())
    du = terms * (1.0 if after else act.abs())
    terms = {"x": du, "residual": du * z["scale"].abs(), "gate": terms * (u * slope).abs(),
             "scale": (du * z["residual"].abs()).norm(dim=0)}
    if after:
        terms.pop("gate")                          # (its gradient does not hold ds)
    return {**one, **{k: max(1.0, (t.norm() / want[k].norm()).item()) for k, t in terms.items()}}


def check(x, d, dtype, rms, after, eps=1e-5, dtotal=True):
    g = {n: t.cuda() for n, t in x.items()}
    dg = {n: t.cuda() for n, t in d.items()}
    kind = dict(gate=g.get("gate"), residual=g.get("residual"), scale=g.get("scale"), rms=rms, gate_after=after)
    w, b = g.get("weight"), g.get("bias")
    y, total, mean, rstd = fw.gated_norm(g["x"], w, b, eps=eps, **kind)
    got = fw.gated_norm_backward(dg["dy"], g["x"], w, b, mean, rstd, dtotal=dg["dtotal"] if dtotal else None, **kind)
    fw.check()
    ry, ru, rm, rr = R.gated(**{n: R.f64(t) for n, t in x.items()}, rms=rms, gate_after=after, eps=eps)
    assert y.dtype == dtype and R.rel(y, ry) <= TOL[dtype]
    assert R.rel(rstd, rr) <= 4e-6
    if rms:
        assert mean is None
    else:
        assert ((mean.cpu().double() - rm) * rr).abs().max() <= 4e-6 * 4
    if "residual" in x:
        assert total.dtype == dtype and R.rel(total, ru) <= TOL[dtype]
    else:
        assert total is None
    want = R.gated_grads(d["dy"], d["dtotal"] if dtotal else None, eps, rms=rms, gate_after=after, **x)
    dx, dweight, dbias, dgate, dresidual, dscale = got
    more = room(x, d, rms, after, eps, want)
    assert dx.dtype == dtype and R.rel(dx, want["x"]) <= TOL[dtype] * more["x"]
    if "gate" in x:
        assert R.rel(dgate, want["gate"]) <= TOL[dtype] * more["gate"]
    else:
        assert dgate is None
    if "residual" not in x:
        assert dresidual is None and dscale is None
    else:
        assert R.rel(dresidual, want["residual"]) <= TOL[dtype] * more["residual"]
        assert (dscale is None) == ("scale" not in x)
    if "weight" in x:
        assert R.rel(dweight, want["weight"]) <= TOL_SUM and R.rel(dbias, want["bias"]) <= TOL_SUM
        if "scale" in x:
            assert R.rel(dscale, want["scale"]) <= TOL_SUM * more["scale"]


WIDTHS = [2, 3, 8, 31, 32, 33, 64, 66, 68, 100, 128, 130, 200, 256, 257, 258, 300, 512, 514, 520, 1000, 1023, 1024, 1030,
          1100, 2048, 2052, 2056, 2500, 4095, 4096, 4098, 5000, 8190, 8191, 8192]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("rms,after", [(False, False), (True, False), (False, True), (True, True)])
def test_widths(width, rms, after, dtype):
    x, d = inputs(37, width, dtype, seed=width)
    check(x, d, dtype, rms, after)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate,residual,params", [(False, False, False), (False, True, True), (True, False, True),
                                                  (True, True, False), (False, True, False), (False, False, True)])
@pytest.mark.parametrize("rms,after", [(False, True), (True, False)])
def test_what_is_given(gate, residual, params, rms, after, dtype):
    for width in (96, 1500):
        x, d = inputs(11, width, dtype, seed=width, gate=gate, residual=residual, params=params)
        check(x, d, dtype, rms, after, dtotal=residual)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("H,n,width", [(2, 1, 64), (3, 7, 128), (16, 40, 65), (5, 3, 1024), (700, 1, 32)])
@pytest.mark.parametrize("after", [False, True])
def test_parameters_of_each_head(H, n, width, after, dtype):
    x, d = inputs(H * n * 3, width, dtype, H=H, seed=H)
    check(x, d, dtype, not after, after)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,width", [(1, 64), (1, 8192), (2, 1), (20000, 64), (9000, 257), (3000, 2048), (700, 8192)])
def test_rows(rows, width, dtype):
    x, d = inputs(rows, width, dtype, seed=rows)
    check(x, d, dtype, width == 1, False)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_mean_far_from_zero_and_rows_that_are_equal(dtype):
    """E[s^2] - E[s]^2 would lose the variance of these rows."""
    x, d = inputs(50, 512, F32, seed=1, gate=False, residual=False)
    x["x"] = (x["x"] + 1000.0).to(dtype)
    d = {n: t.to(dtype) for n, t in d.items()}
    y, _, mean, rstd = fw.gated_norm(x["x"].cuda(), x["weight"].cuda(), x["bias"].cuda())
    ry, _, rm, rr = R.gated(*[R.f64(x[n]) for n in ("x", "weight", "bias")])
    # the mean is within 2^-24 of 1000, 6e-5 of the rows' deviation of two or more
    assert R.rel(y, ry) <= TOL[dtype] + 1e-4 and R.rel(rstd, rr) <= 4e-6 + 1e-7
    z = torch.full((3, 640), 5.0, dtype=dtype, device="cuda")
    y, _, _, _ = fw.gated_norm(z, None, torch.ones(640, device="cuda"))
    assert (y == 1).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("width", [7, 33, 96, 130, 1023, 1024, 4097, 5000])
@pytest.mark.parametrize("after", [False, True])
@pytest.mark.parametrize("rows", [23, 1300])
def test_in_place(rows, after, width, dtype):
    x, d = inputs(rows, width, dtype, seed=2)
    g = {n: t.cuda() for n, t in {**x, **d}.items()}
    kind = dict(scale=g["scale"], rms=True, gate_after=after)
    y, total, _, rstd = fw.gated_norm(g["x"], g["weight"], g["bias"], gate=g["gate"], residual=g["residual"], **kind)
    for a, b in (("x", "residual"), ("gate", "x"), ("residual", "gate")):
        z = {n: t.clone() for n, t in g.items()}
        got = fw.gated_norm(z["x"], z["weight"], z["bias"], gate=z["gate"], residual=z["residual"], y=z[a], total=z[b], **kind)
        assert got[0] is z[a] and got[1] is z[b]
        assert torch.equal(z[a], y) and torch.equal(z[b], total) and torch.equal(got[3], rstd)
    grads = fw.gated_norm_backward(g["dy"], g["x"], g["weight"], g["bias"], None, rstd, gate=g["gate"],
                                   residual=g["residual"], dtotal=g["dtotal"], **kind)
    for names in (("dy", "gate", "residual"), ("dtotal", "x", "dy"), ("x", "dtotal", "gate")):
        z = {n: t.clone() for n, t in g.items()}
        got = fw.gated_norm_backward(z["dy"], z["x"], z["weight"], z["bias"], None, rstd, gate=z["gate"],
                                     residual=z["residual"], dtotal=z["dtotal"], dx=z[names[0]], dgate=z[names[1]],
                                     dresidual=z[names[2]], **kind)
        assert all(torch.equal(a, b) for a, b in zip(got, grads))


@pytest.mark.parametrize("after", [False, True])
def test_gates_of_any_size(after):
    """silu(z) is z, and its slope 1, for large z; both 0 for large -z."""
    x, d = inputs(6, 64, F32, seed=5, residual=False)
    x["gate"][:, ::4], x["gate"][:, 1::4] = 1e6, -1e6
    x["gate"][:, 2::4] = 50.0
    check(x, d, F32, True, after, dtotal=False)


def test_values_that_are_not_finite_stay_in_their_row():
    x, d = inputs(20, 300, F32, seed=4)
    g = {n: t.cuda() for n, t in x.items()}
    kind = dict(gate=g["gate"], residual=g["residual"], scale=g["scale"])
    y0 = fw.gated_norm(g["x"], g["weight"], g["bias"], **kind)[0]
    g["x"][7, 5] = float("inf")
    g["gate"][9, 0] = float("nan")
    y = fw.gated_norm(g["x"], g["weight"], g["bias"], **kind)[0]
    keep = [i for i in range(20) if i not in (7, 9)]
    assert torch.equal(y[keep], y0[keep]) and torch.isnan(y[9]).all()
    g["x"][7, 5] = 0.0
    g["gate"][9, 0] = -200.0                        # silu is zero there
    assert torch.isfinite(fw.gated_norm(g["x"], g["weight"], g["bias"], **kind)[0]).all()


def test_sums_repeat_to_the_bit_and_in_replays():
    x, d = inputs(5000, 384, BF16, seed=6)
    g = {n: t.cuda() for n, t in {**x, **d}.items()}

    def run():
        kind = dict(gate=g["gate"], residual=g["residual"], scale=g["scale"])
        y, total, mean, rstd = fw.gated_norm(g["x"], g["weight"], g["bias"], **kind)
        return [y, total, *fw.gated_norm_backward(g["dy"], g["x"], g["weight"], g["bias"], mean, rstd, dtotal=g["dtotal"],
                                                  **kind)]
    first = [t.clone() for t in run()]
    assert all(torch.equal(a, b) for a, b in zip(first, run()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run()
    for t in outs:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, outs))


def test_offsets_beyond_32_bits():
    rows, width = (1 << 18) + 3, 8192
    if torch.cuda.mem_get_info()[0] < (40 << 30):
        pytest.skip("needs 40 GB")
    x, d = inputs(3, width, BF16, seed=1)
    big = {n: torch.zeros(rows, width, dtype=BF16, device="cuda") for n in ("x", "gate")}
    for n in big:
        big[n][-3:] = x[n].cuda()
    w, b = x["weight"].cuda(), x["bias"].cuda()
    y, _, _, _ = fw.gated_norm(big["x"], w, b, gate=big["gate"], rms=True)
    ry = R.gated(R.f64(x["x"]), R.f64(x["weight"]), R.f64(x["bias"]), gate=R.f64(x["gate"]), rms=True)[0]
    assert R.rel(y[-3:], ry) <= TOL[BF16] and torch.equal(y[0], b.to(BF16))
