"""Short causal convolution and its gradients on the GPU against the definition in 64 bits.

Tolerances (relative L2).  Rows in fp32: at most W + 8 rounded operations of 2^-24 each, the exponential and the
quotient of silu among them with two ulp: 16 2^-24 = 9.5e-7, and a gradient row sums W such: 4e-6.
dweight, dbias: sums of n terms in fp32 over four levels (a thread's rows, lanes, warps, blocks), errors of random
sign: sqrt(n) 2^-24 of a sum that grows as sqrt(n) itself, and each term as off as a row: 4e-6.  bf16 rows are
rounded once (2^-8 at most): 4.1e-3 with the fast exponential's few fp32 ulp.  A row in W or fewer tokens of
cancelling taps costs no more: errors are relative to the terms, and an output of many rows has its terms' size.
"""
import pytest
import torch

from linear_token_mixer_gb300 import fw

import mixer_ref as R

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TOL = {F32: 4e-6, BF16: 4.1e-3}
TOL_SUM = 4e-6


def inputs(B, H, T, d, W, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed)

    def rn(*s):
        return torch.randn(*s, generator=gen)

    x = {"x": rn(B, H, T, d).to(dtype), "w": rn(H, d, W) * W ** -0.5, "b": rn(H, d) * 0.3,
         "state": rn(B, H, W - 1, d).to(dtype), "dy": rn(B, H, T, d).to(dtype), "dso": rn(B, H, W - 1, d).to(dtype)}
    return x, {n: t.cuda() for n, t in x.items()}


def check(x, g, dtype, silu=True, bias=True, state=True, lens=None):
    b, s, dso = ("b" if bias else None), ("state" if state else None), ("dso" if state else None)
    at = lambda z, n: None if n is None else z[n]  # noqa: E731
    lg = None if lens is None else lens.cuda()
    y, so = fw.conv_prefill(g["x"], g["w"], at(g, b), at(g, s), silu=silu, lens=lg)
    grads = fw.conv_backward(g["dy"], g["x"], g["w"], at(g, b), at(g, s), at(g, dso), silu=silu, lens=lg)
    fw.check()
    clean = {n: t.clone() for n, t in x.items()}
    ry, rso = R.conv(*[R.f64(at(clean, n)) for n in ("x", "w", b, s)], silu, lens)
    rg = R.conv_grads(clean["dy"], clean["x"], clean["w"], at(clean, b), at(clean, s), at(clean, dso), silu, lens)
    assert y.dtype == dtype and R.rel(y, ry) <= TOL[dtype]
    assert torch.equal(so.cpu().double(), rso)
    B, H, T, d = x["x"].shape
    for i, n in enumerate(R.ends(lens, B, T)):
        rg[0][i, :, n:] = 0
    assert grads[0].dtype == dtype and R.rel(grads[0], rg[0]) <= TOL[dtype]
    assert grads[1].dtype == F32 and R.rel(grads[1], rg[1]) <= TOL_SUM
    assert R.rel(grads[2], rg[2]) <= TOL_SUM
    if state:
        assert grads[3].dtype == dtype and R.rel(grads[3], rg[3]) <= TOL[dtype]
    else:
        assert grads[3] is None


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("W", [2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("d", [1, 3, 6, 8, 12, 64, 65, 136])
def test_widths_and_taps(d, W, dtype):
    x, g = inputs(2, 3, 37, d, W, dtype, seed=d + W)
    check(x, g, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,H,T,d", [(1, 1, 1, 64), (3, 2, 2, 64), (1, 1, 3, 5), (2, 1, 8, 16), (1, 2, 65, 128),
                                     (2, 2, 700, 40), (1, 1, 2000, 257), (5, 40, 3, 8)])
@pytest.mark.parametrize("silu,bias,state", [(True, False, False), (False, True, True), (False, False, False)])
def test_lengths(B, H, T, d, silu, bias, state, dtype):
    x, g = inputs(B, H, T, d, 4, dtype, seed=T)
    check(x, g, dtype, silu, bias, state)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [1, 3, 9, 200])
@pytest.mark.parametrize("d", [24, 33])
@pytest.mark.parametrize("state", [False, True])
def test_padded_batch(state, d, T, dtype):
    B, H, W = 6, 2, 4
    x, g = inputs(B, H, T, d, W, dtype, seed=T)
    lens = torch.tensor([T, 0, 1, 2, T // 2, T + 5], dtype=torch.int32)
    for b, n in enumerate(R.ends(lens, B, T)):     # what lies behind a row's end is never used
        for name in ("x", "dy"):
            g[name][b, :, n:] = float("nan")
    check(x, g, dtype, lens=lens, state=state)
    y, dx = (torch.full((B, H, T, d), 7.0, dtype=dtype, device="cuda") for _ in range(2))
    past = g["state"] if state else None
    fw.conv_prefill(g["x"], g["w"], g["b"], past, lens=lens.cuda(), y=y)
    fw.conv_backward(g["dy"], g["x"], g["w"], g["b"], past, lens=lens.cuda(), dx=dx)
    for b, n in enumerate(R.ends(lens, B, T)):
        assert (y[b, :, n:] == 7.0).all() and (dx[b, :, n:] == 7.0).all()
        assert torch.isfinite(y[b]).all() and torch.isfinite(dx[b]).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("W,d", [(2, 64), (4, 128), (4, 7), (8, 130)])
def test_parts_and_tokens_continue_one_another(W, d, dtype):
    """A prompt in parts, then token by token, the state moved on in place: the bits of the whole prompt."""
    B, H, T = 2, 3, 40
    x, g = inputs(B, H, T, d, W, dtype, seed=W)
    whole, end = fw.conv_prefill(g["x"], g["w"], g["b"], g["state"])
    state = g["state"].clone()
    rows = []
    for a, b in ((0, 1), (1, 3), (3, 30)):
        y, s = fw.conv_prefill(g["x"][:, :, a:b].contiguous(), g["w"], g["b"], state, state_out=state)
        assert s is state
        rows.append(y)
    for t in range(30, T):
        rows.append(fw.conv_step(g["x"][:, :, t].contiguous(), g["w"], g["b"], state).unsqueeze(2))
    assert torch.equal(torch.cat(rows, 2), whole) and torch.equal(state, end)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_values_that_are_not_finite_reach_their_taps_only(dtype):
    B, H, T, d, W = 1, 2, 100, 16, 4
    x, g = inputs(B, H, T, d, W, dtype, seed=1)
    want, _ = R.conv(*[R.f64(x[n]) for n in ("x", "w", "b", "state")])
    g["x"][0, 1, 50, 3] = float("nan")
    y, _ = fw.conv_prefill(g["x"], g["w"], g["b"], g["state"])
    hit = torch.zeros(B, H, T, d, dtype=torch.bool)
    hit[0, 1, 50:50 + W, 3] = True
    assert torch.isnan(y.cpu()[hit]).all() and R.rel(torch.where(hit, 0.0, y.cpu().double()), torch.where(hit, 0.0, want)) <= TOL[dtype]
    g["x"][0, 1, 50, 3] = 1e4                       # (silu of a large negative value is zero, of a large one itself)
    y, _ = fw.conv_prefill(-g["x"].abs(), g["w"].abs(), g["b"], None)
    assert torch.isfinite(y).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_slopes_of_large_values(dtype):
    """silu'(a) is 1 for large a and 0 for large -a, of any size."""
    a = torch.tensor([60.0, 3e4, 1e7, 2.0 ** 30, 1e30, -60.0, -3e4, -2.0 ** 30, -1e30]).to(dtype)
    x = a.view(1, 1, 1, -1).cuda()
    w = torch.zeros(1, 9, 2, device="cuda")
    w[:, :, 1] = 1.0
    dx, _, _, _ = fw.conv_backward(torch.ones_like(x), x, w)
    y, _ = fw.conv_prefill(x, w)
    r = a.double()
    sig = 1 / (1 + torch.exp(-r))
    # (what is below 2^-126 may be zero)
    for got, want in ((dx, sig * (1 + r * (1 - sig))), (y, r * sig)):
        assert ((got.cpu().double().view(-1) - want).abs() <= TOL[dtype] * want.abs() + 2.0 ** -126).all()


def test_gradients_repeat_to_the_bit():
    x, g = inputs(8, 4, 300, 96, 4, BF16, seed=3)
    first = [t.clone() for t in fw.conv_backward(g["dy"], g["x"], g["w"], g["b"], g["state"])]
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, fw.conv_backward(g["dy"], g["x"], g["w"], g["b"], g["state"])))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_replayed_with_other_inputs(dtype):
    def run(z):
        y = fw.conv_prefill(z["x"], z["w"], z["b"], z["state"], lens=z["lens"])
        return [*y, *fw.conv_backward(z["dy"], z["x"], z["w"], z["b"], z["state"], z["dso"], lens=z["lens"])]
    _, z = inputs(3, 2, 120, 48, 4, dtype, 1)
    z["lens"] = torch.tensor([120, 3, 60], dtype=torch.int32, device="cuda")
    run(z)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run(z)
    for seed in (2, 3):
        _, y = inputs(3, 2, 120, 48, 4, dtype, seed)
        y["lens"] = torch.tensor([0, 120, 7 * seed], dtype=torch.int32, device="cuda")
        want = [t.clone() for t in run(y)]
        for n in z:
            z[n].copy_(y[n])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_offsets_beyond_32_bits():
    B, H, T, d, W = 3, 2, 1 << 18, 2048, 4
    if torch.cuda.mem_get_info()[0] < (60 << 30):
        pytest.skip("needs 60 GB")
    x, g = inputs(1, 1, 300, d, W, BF16, seed=1)
    big, dy = (torch.zeros(B, H, T, d, dtype=BF16, device="cuda") for _ in range(2))
    big[-1, -1, -300:], dy[-1, -1, -300:] = g["x"][0, 0], g["dy"][0, 0]
    w, b = g["w"].expand(H, d, W).contiguous(), torch.zeros(H, d, device="cuda")
    y, _ = fw.conv_prefill(big, w, b)
    ry, _ = R.conv(R.f64(x["x"]), R.f64(x["w"]))
    assert R.rel(y[-1:, -1:, -300:], ry) <= TOL[BF16] and not y[0].any()
    del y
    dx, dw, _, _ = fw.conv_backward(dy, big, w, b)
    rg = R.conv_grads(x["dy"], x["x"], x["w"])
    assert R.rel(dx[-1:, -1:, -300:], rg[0]) <= TOL[BF16] and not dx[0].any()
    assert R.rel(dw[-1:], rg[1]) <= TOL_SUM
