"""Calls of the selective scan, the convolution and the gated norm that their documentation allows and that are made
seldom: decays that grow, steps, queries and keys that are not finite, biases without softplus, gradients of some
arguments alone.  Against the definitions in 64 bits, with the tolerances of each operator's own tests."""
import ctypes

import pytest
import torch

from linear_token_mixer_gb300 import fw

import mixer_ref as R
import test_conv_gpu as C
import test_gated_norm_gpu as N
import test_select_gpu as S

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
both = pytest.mark.parametrize("dtype", [F32, BF16])


@both
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,total", [(128, 30.0), (150, 70.0), (2100, 2.0)])
def test_decays_that_grow(T, total, d, dtype):
    """Logs that sum to `total` in 128 tokens: states and rows of up to e^80, no chunk of them beyond it."""
    x, _ = S.inputs(1, 2, 1, T, d, dtype, seed=T, dt_type=F32)
    x["dt"] = 0.5 + torch.rand(1, 2, T, generator=torch.Generator().manual_seed(1))
    x["ld"] = torch.tensor([1.0, 0.6]) * total / 128
    g = {n: t.cuda() for n, t in x.items()}
    got = S.run(g, softplus=False)
    fw.check()
    S.check(got, S.ref(x, softplus=False), dtype)


@both
@pytest.mark.parametrize("T,at", [(500, 300), (2100, 1500)])
@pytest.mark.parametrize("name,value", [("q", float("nan")), ("k", float("inf")), ("k", float("nan")), ("dt", float("nan")),
                                        ("dt", float("inf"))])
def test_queries_keys_and_steps_that_are_not_finite(name, value, T, at, dtype):
    """One in q reaches its row alone; one in k or in a step its chunk of 128 tokens and what follows, in its own chain."""
    x, _ = S.inputs(1, 2, 2, T, 64, dtype, seed=T, rate=(0.1, 0.2), dt_type=F32)
    want, _ = S.ref(x)
    if name == "dt":
        x["dt"][0, 0, at] = value
    else:
        x[name][0, 0, at, 7] = value
    o, state = S.run({n: t.cuda() for n, t in x.items()})
    fw.check()
    hit = torch.zeros(1, 2, T, 64, dtype=torch.bool)
    hit[0, 0, at:at + 1 if name == "q" else T] = True
    may = hit.clone()
    if name != "q":
        may[0, 0, at // 128 * 128:] = True
    o = o.cpu()
    assert not torch.isfinite(o[0, 0, at]).all() and torch.isfinite(o[~may]).all()
    assert R.rel(torch.where(may, 0.0, o.double()), torch.where(may, 0.0, want)) <= S.TOL[dtype]
    assert torch.isfinite(state[0, 1]).all() and torch.isfinite(state[0, 0]).all().item() == (name == "q")


@both
def test_a_bias_of_the_steps_without_softplus(dtype):
    x, g = S.inputs(2, 4, 2, 200, 64, dtype, seed=3, dt_type=F32)
    x["bias"] = 0.02 + 0.02 * torch.rand(4, generator=torch.Generator().manual_seed(2))
    x["dt"] = x["dt"].abs() * 0.02
    g = {n: t.cuda() for n, t in x.items()}
    args = (g["q"], g["k"], g["v"], g["dt"], g["ld"])
    ref = [x[n] for n in ("q", "k", "v", "dt", "ld")]
    want = R.select(*ref, x["S0"], x["bias"], False, x["skip"], 0.5)
    S.check(fw.select_prefill(*args, g["S0"], dt_bias=g["bias"], skip=g["skip"], scale=0.5), want, dtype)
    one = [t[:, :, 0].contiguous() for t in args[:4]]
    state = g["S0"].clone()
    o = fw.select_step(*one, g["ld"], state, dt_bias=g["bias"], skip=g["skip"], scale=0.5)
    ro, rS = R.select(*[t[:, :, :1] for t in ref[:4]], x["ld"], x["S0"], x["bias"], False, x["skip"], 0.5)
    assert R.rel(o, ro[:, :, 0]) <= S.TOL[dtype] and R.rel_rows(state, rS, 2) <= S.TOL_STATE


@both
@pytest.mark.parametrize("B", [60, 70])
def test_more_rows_of_a_batch_than_are_ranked(B, dtype):
    """Padded batches on either side of the number of rows whose longest start first; states from zero."""
    H, T = 3, 150
    x, g = S.inputs(B, H, 1, T, 64, dtype, seed=B)
    lens = torch.randint(0, T + 1, (B,), generator=torch.Generator().manual_seed(3), dtype=torch.int32)
    lens[:2] = torch.tensor([0, -5])
    got = S.run(g, S0=False, lens=lens.cuda())
    S.check(got, S.ref(x, S0=False, lens=lens), dtype)
    assert not got[1][:2].any()


@both
@pytest.mark.parametrize("d", [40, 33])
def test_gradients_of_a_carried_state_alone(d, dtype):
    """dstate_out without a state before (and its gradient asked for all the same), and a state without dstate_out."""
    B, H, T, W = 5, 2, 11, 4
    x, g = C.inputs(B, H, T, d, W, dtype, seed=d)
    lens = torch.tensor([T, 0, 1, 2, 7], dtype=torch.int32)
    on = torch.zeros(B, 1, T, 1, dtype=torch.bool)
    for b, n in enumerate(lens):
        on[b, :, :n] = True
    for state, dso in ((None, "dso"), ("state", None)):
        ds = torch.full((B, H, W - 1, d), 7.0, dtype=dtype, device="cuda")
        at = lambda z, n: None if n is None else z[n]  # noqa: E731
        got = fw.conv_backward(g["dy"], g["x"], g["w"], g["b"], at(g, state), at(g, dso), lens=lens.cuda(), dstate=ds)
        want = R.conv_grads(x["dy"], x["x"], x["w"], x["b"], at(x, state), at(x, dso), True, lens)
        assert got[3] is ds and R.rel(got[0], torch.where(on, want[0], 0.0)) <= C.TOL[dtype]
        assert R.rel(got[1], want[1]) <= C.TOL_SUM and R.rel(got[2], want[2]) <= C.TOL_SUM
        assert R.rel(ds, want[3]) <= C.TOL[dtype]


def _shape(*s):
    return ctypes.byref(fw.fw_shape(*s))


@both
def test_some_gradients_of_the_convolution_alone(dtype):
    """Through the C call: dweight or dbias alone, and neither, without a workspace.  The same bits as together."""
    B, H, T, d, W = 3, 2, 70, 24, 4
    _, g = C.inputs(B, H, T, d, W, dtype, seed=1)
    full = fw.conv_backward(g["dy"], g["x"], g["w"], g["b"], g["state"])
    L, code = fw.lib(), 1 if dtype == BF16 else 0
    ws = torch.empty(L.fw_conv_workspace(_shape(B, H, T, d, d), W), dtype=torch.uint8, device="cuda")
    for want in ((False, False), (True, False), (False, True)):
        dx, dw, db = (torch.full_like(t, 7.0) for t in full[:3])
        sums = any(want)
        st = L.fw_conv_backward(g["dy"].data_ptr(), g["x"].data_ptr(), g["w"].data_ptr(), g["b"].data_ptr(),
                                g["state"].data_ptr(), None, None, dx.data_ptr(), dw.data_ptr() if want[0] else None,
                                db.data_ptr() if want[1] else None, None, _shape(B, H, T, d, d), W, code, 8,
                                ws.data_ptr() if sums else None, ws.numel() if sums else 0,
                                torch.cuda.current_stream().cuda_stream)
        assert st == 0 and torch.equal(dx, full[0])
        assert torch.equal(dw, full[1]) if want[0] else (dw == 7.0).all()
        assert torch.equal(db, full[2]) if want[1] else (db == 7.0).all()
    fw.check()


@both
@pytest.mark.parametrize("width", [96, 257, 5000])
def test_some_gradients_of_the_gated_norm_alone(width, dtype):
    """Through the C call, each output by itself: the same bits as together, and nothing else written."""
    rows = 300
    x, d = N.inputs(rows, width, dtype, seed=width)
    g = {n: t.cuda() for n, t in {**x, **d}.items()}
    kind = dict(gate=g["gate"], residual=g["residual"], scale=g["scale"])
    _, _, mean, rstd = fw.gated_norm(g["x"], g["weight"], g["bias"], **kind)
    dx, dw, db, dg, dr, ds = fw.gated_norm_backward(g["dy"], g["x"], g["weight"], g["bias"], mean, rstd, dtotal=g["dtotal"],
                                                    **kind)
    full = [dx, dg, dr, dw, db, ds]
    L, code = fw.lib(), 1 if dtype == BF16 else 0
    ws = torch.empty(L.fw_gated_norm_workspace(rows, width, 1, code), dtype=torch.uint8, device="cuda")
    args = fw.fw_gated(g["gate"].data_ptr(), g["residual"].data_ptr(), g["scale"].data_ptr(), g["weight"].data_ptr(),
                       g["bias"].data_ptr(), 1, rows, 0.0, 0, 0)
    for i in range(6):
        outs = [torch.full_like(t, 7.0) for t in full]
        ptr = [t.data_ptr() if j == i else None for j, t in enumerate(outs)]
        st = L.fw_gated_norm_backward(g["dy"].data_ptr(), g["dtotal"].data_ptr(), g["x"].data_ptr(), ctypes.byref(args),
                                      mean.data_ptr(), rstd.data_ptr(), *ptr, rows, width, code,
                                      ws.data_ptr() if i >= 3 else None, ws.numel() if i >= 3 else 0,
                                      torch.cuda.current_stream().cuda_stream)
        assert st == 0
        for j, (t, want) in enumerate(zip(outs, full)):
            assert torch.equal(t, want) if j == i else (t == 7.0).all()
    fw.check()


@both
@pytest.mark.parametrize("residual", [False, True])
def test_gradients_of_the_sum_with_and_without_a_residual(residual, dtype):
    """dtotal without a residual (total is a copy of x then), and a residual without dtotal or scale."""
    x, d = N.inputs(40, 130, dtype, seed=2, residual=residual)
    x.pop("scale", None)
    g = {n: t.cuda() for n, t in {**x, **d}.items()}
    kind = dict(gate=g["gate"], residual=g.get("residual"), rms=True)
    total = torch.empty_like(g["x"])
    y, out, _, rstd = fw.gated_norm(g["x"], g["weight"], g["bias"], total=total, **kind)
    _, ru, _, _ = R.gated(**{n: R.f64(t) for n, t in x.items()}, rms=True)
    assert out is total and R.rel(total, ru) <= N.TOL[dtype]
    dtotal = None if residual else g["dtotal"]
    got = fw.gated_norm_backward(g["dy"], g["x"], g["weight"], g["bias"], None, rstd, dtotal=dtotal, **kind)
    want = R.gated_grads(d["dy"], None if residual else d["dtotal"], rms=True, gate_after=False, **x)
    assert R.rel(got[0], want["x"]) <= N.TOL[dtype] and R.rel(got[3], want["gate"]) <= N.TOL[dtype]
    assert (got[4] is got[0] and got[5] is None) if residual else got[4] is None
    own = torch.empty_like(g["x"])
    if residual:
        again = fw.gated_norm_backward(g["dy"], g["x"], g["weight"], g["bias"], None, rstd, dresidual=own, **kind)
        assert again[4] is own and torch.equal(own, got[0])


@both
def test_a_row_by_itself(dtype):
    """x of one axis: statistics of none."""
    x, d = N.inputs(1, 200, dtype, seed=9, gate=False)
    g = {n: t[0].cuda() if t.dim() == 2 else t.cuda() for n, t in {**x, **d}.items()}
    kind = dict(residual=g["residual"], scale=g["scale"])
    y, total, mean, rstd = fw.gated_norm(g["x"], g["weight"], g["bias"], **kind)
    ry, ru, rm, rr = R.gated(**{n: R.f64(t) for n, t in x.items()})
    assert mean.shape == rstd.shape == () and R.rel(y, ry[0]) <= N.TOL[dtype] and R.rel(total, ru[0]) <= N.TOL[dtype]
    got = fw.gated_norm_backward(g["dy"], g["x"], g["weight"], g["bias"], mean, rstd, dtotal=g["dtotal"], **kind)
    want = R.gated_grads(d["dy"], d["dtotal"], rms=False, gate_after=False, **x)
    assert R.rel(got[0], want["x"][0]) <= N.TOL[dtype] and R.rel(got[1], want["weight"]) <= N.TOL_SUM
