"""Decayed linear attention on the GPU against the 64-bit token recurrence.

Tolerances (relative L2 of a whole output, and of every chain).  fp32: each of a row's sums has
at most d + C + 3 rounded operations of relative size 2^-24 on terms whose signs are random, so
the relative L2 error is about sqrt(400) 2^-24 = 1.2e-6, and cancellation in one chain of few
tokens costs a small factor more: 1e-5.  bf16 inputs: the state is kept in fp32 (S_T, dS0: its
operands carry 16 bits or more, 2^-17 each: 1e-5 like fp32); an output row is rounded once
(at most 2^-8 relative) and its matrix operands, the masked products and the carried state, once
each, all of random sign: sqrt(3) 2^-8 / sqrt(3) = 3.9e-3 as an upper estimate of the relative
L2, with two more such roundings' room for one chain of few rows: 8e-3.
"""
import pytest
import torch

from linear_token_mixer_gb300 import fw

import decay_ref as R

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TOL = {F32: 1e-5, BF16: 8e-3}
TOL_STATE = 1e-5


def decays(H, kind="mixed"):
    h = torch.arange(H, dtype=torch.float64)
    if kind == "none":
        return torch.zeros(H)
    if kind == "slow":
        return torch.log1p(-torch.exp2(-5.0 - h)).float()
    return (-torch.exp2(1.0 - 2.0 * h)).float()          # from g = 0.14 on


def inputs(B, H, T, d, dtype, seed=0, kind="mixed"):
    g = torch.Generator().manual_seed(seed)
    def rn(*s):
        return torch.randn(*s, generator=g)
    x = {n: rn(B, H, T, d).to(dtype) for n in ("q", "k", "v", "do")}
    x.update(ld=decays(H, kind), S0=rn(B, H, d, d) * 3, dS=rn(B, H, d, d))
    return x, {n: t.cuda() for n, t in x.items()}


def check_state(got, ref):
    assert got.dtype == F32
    assert R.rel_rows(got, ref, 2) <= TOL_STATE


def check_rows(got, ref, dtype):
    assert got.dtype == dtype
    assert R.rel(got, ref) <= TOL[dtype]
    assert R.rel_rows(got, ref, 2) <= TOL[dtype]


SIZES = [(1, 1, 1), (2, 2, 2), (1, 3, 63), (1, 2, 64), (2, 1, 65), (1, 2, 127), (1, 1, 128),
         (1, 2, 129), (1, 2, 257), (2, 3, 400)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,T", SIZES)
@pytest.mark.parametrize("s0", [False, True])
def test_prefill(B, H, T, d, dtype, s0):
    x, g = inputs(B, H, T, d, dtype, seed=T)
    S0 = x["S0"] if s0 else None
    o, S = fw.decay_prefill(g["q"], g["k"], g["v"], g["ld"], g["S0"] if s0 else None, scale=0.25)
    fw.check()
    ro, rS, _ = R.forward(x["q"], x["k"], x["v"], x["ld"], S0, 0.25)
    check_rows(o, ro, dtype)
    check_state(S, rS)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,T", SIZES)
@pytest.mark.parametrize("s0", [False, True])
def test_backward(B, H, T, d, dtype, s0):
    x, g = inputs(B, H, T, d, dtype, seed=T + 1)
    got = fw.decay_backward(g["q"], g["k"], g["v"], g["ld"], g["do"], g["S0"] if s0 else None,
                            g["dS"] if s0 else None, scale=0.25)
    fw.check()
    ref = R.backward(x["q"], x["k"], x["v"], x["ld"], x["do"], x["S0"] if s0 else None,
                     x["dS"] if s0 else None, 0.25)
    for a, b in zip(got[:3], ref[:3]):
        check_rows(a, b, dtype)
    if s0:
        check_state(got[3], ref[3])
    else:
        assert got[3] is None


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", ["none", "slow"])
def test_decay_extremes(kind, dtype):
    x, g = inputs(1, 3, 300, 64, dtype, seed=9, kind=kind)
    o, S = fw.decay_prefill(g["q"], g["k"], g["v"], g["ld"], g["S0"])
    ro, rS, _ = R.forward(x["q"], x["k"], x["v"], x["ld"], x["S0"])
    check_rows(o, ro, dtype)
    check_state(S, rS)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_no_memory_at_all(dtype):
    """g = 0 (log_decay = -inf): every token sees itself only."""
    x, g = inputs(1, 2, 200, 64, dtype, seed=4)
    ld = torch.full((2,), float("-inf"))
    o, S = fw.decay_prefill(g["q"], g["k"], g["v"], ld.cuda(), g["S0"])
    q, k, v = (x[n].double() for n in "qkv")
    check_rows(o, (q * k).sum(-1, keepdim=True) * v, dtype)
    check_state(S, k[:, :, -1, :, None] * v[:, :, -1, None, :])
    dq, dk, dv, dS0 = fw.decay_backward(g["q"], g["k"], g["v"], ld.cuda(), g["do"], g["S0"], g["dS"])
    do = x["do"].double()
    check_rows(dq, (v * do).sum(-1, keepdim=True) * k, dtype)
    assert float(dS0.abs().max()) == 0.0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128])
def test_growing_decay_is_computed_literally(d, dtype):
    x, g = inputs(1, 2, 150, d, dtype, seed=8)
    ld = torch.tensor([0.02, 0.0])
    o, S = fw.decay_prefill(g["q"], g["k"], g["v"], ld.cuda())
    ro, rS, _ = R.forward(x["q"], x["k"], x["v"], ld)
    check_rows(o, ro, dtype)
    check_state(S, rS)


LENS = [(0, 1, 300), (300, 64, 65), (128, 127, 129), (-5, 999, 256)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", LENS)
def test_padded_batch(lens, d, dtype):
    """Rows behind the end hold NaN and infinities, which must not reach anything; the outputs'
    rows there stay as they were."""
    B, H, T = 3, 2, 300
    x, g = inputs(B, H, T, d, dtype, seed=sum(lens))
    ln = torch.tensor(lens, dtype=torch.int32)
    n = ln.clamp(0, T)
    behind = torch.arange(T).view(1, 1, T, 1) >= n.view(B, 1, 1, 1)
    bad = {}
    for name in ("q", "k", "v", "do"):
        fill = torch.full_like(x[name], float("nan"))
        fill[..., ::2] = float("inf")
        bad[name] = torch.where(behind, fill, x[name]).cuda()
    mark = -7.0
    o = torch.full((B, H, T, d), mark, device="cuda", dtype=dtype)
    o, S = fw.decay_prefill(bad["q"], bad["k"], bad["v"], g["ld"], g["S0"], scale=0.5,
                            lens=ln.cuda(), o=o)
    outs = [torch.full((B, H, T, d), mark, device="cuda", dtype=dtype) for _ in range(3)]
    dq, dk, dv, dS0 = fw.decay_backward(bad["q"], bad["k"], bad["v"], g["ld"], bad["do"], g["S0"],
                                        g["dS"], scale=0.5, lens=ln.cuda(), dq=outs[0],
                                        dk=outs[1], dv=outs[2])
    fw.check()
    ro, rS, _ = R.forward(x["q"], x["k"], x["v"], x["ld"], x["S0"], 0.5, ln)
    ref = R.backward(x["q"], x["k"], x["v"], x["ld"], x["do"], x["S0"], x["dS"], 0.5, ln)
    for got, want in zip((o, dq, dk, dv), (ro,) + ref[:3]):
        got = got.cpu()
        assert (got[behind.expand_as(got)] == mark).all()
        check_rows(torch.where(behind, torch.zeros((), dtype=dtype), got), want, dtype)
    check_state(S, rS)
    check_state(dS0, ref[3])
    # allocated there, they are zero
    o2, _ = fw.decay_prefill(bad["q"], bad["k"], bad["v"], g["ld"], g["S0"], scale=0.5, lens=ln.cuda())
    new = fw.decay_backward(bad["q"], bad["k"], bad["v"], g["ld"], bad["do"], g["S0"], g["dS"],
                            scale=0.5, lens=ln.cuda())
    mixed = fw.decay_backward(bad["q"], bad["k"], bad["v"], g["ld"], bad["do"], g["S0"], g["dS"],
                              scale=0.5, lens=ln.cuda(), dk=torch.full_like(bad["k"], mark))
    for z, was in zip((o2, *new[:3], *mixed[:3]), (o, dq, dk, dv, dq, dk, dv)):
        want = mark if z is mixed[1] else 0.0
        assert (z.cpu()[behind.expand_as(z)] == want).all()
        assert torch.equal(z.cpu()[~behind.expand_as(z)], was.cpu()[~behind.expand_as(z)])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128])
def test_non_finite_values_stay_in_their_chain_and_time(d, dtype):
    x, g = inputs(1, 2, 200, d, dtype, seed=2)
    k = g["k"].clone()
    k[0, 0, 150] = float("nan")
    o, S = fw.decay_prefill(g["q"], k, g["v"], g["ld"])
    ro, rS, _ = R.forward(x["q"], x["k"], x["v"], x["ld"])
    check_rows(o[:, 1:], ro[:, 1:], dtype)
    check_state(S[:, 1:], rS[:, 1:])
    assert torch.isnan(o[0, 0, 150:]).all() and torch.isnan(S[0, 0]).all()
    # the causal mask: earlier rows of the same chunk see nothing of it
    check_rows(o[:, :1, :128], ro[:, :1, :128], dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("affine", [(True, True), (True, False), (False, False)])
def test_fused_norm(affine, d, dtype):
    x, g = inputs(2, 2, 140, d, dtype, seed=6)
    gen = torch.Generator().manual_seed(1)
    w = torch.randn(d, generator=gen) if affine[0] else None
    b = torch.randn(d, generator=gen) if affine[1] else None
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    ln = torch.tensor([140, 77], dtype=torch.int32)
    o, S = fw.decay_prefill(g["q"], g["k"], g["v"], g["ld"], g["S0"], scale=0.1, lens=ln.cuda(),
                            norm=(dev(w), dev(b)), norm_eps=1e-3)
    ro, rS, _ = R.forward(x["q"], x["k"], x["v"], x["ld"], x["S0"], 0.1, ln)
    on = (torch.arange(140).view(1, 1, -1, 1) < ln.view(-1, 1, 1, 1)).double()
    check_rows(o, R.layer_norm(ro, w, b, 1e-3)[0] * on, dtype)
    check_state(S, rS)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,norm", [(1, 1, False), (2, 5, True), (3, 70, False), (40, 8, True)])
def test_step(B, H, d, norm, dtype):
    x, g = inputs(B, H, 1, d, dtype, seed=B)
    gen = torch.Generator().manual_seed(1)
    w, b = torch.randn(d, generator=gen), torch.randn(d, generator=gen)
    S = g["S0"].clone()
    o = fw.decay_step(g["q"][:, :, 0], g["k"][:, :, 0], g["v"][:, :, 0], g["ld"], S, scale=0.3,
                      norm=(w.cuda(), b.cuda()) if norm else None)
    ro, rS, _ = R.forward(x["q"], x["k"], x["v"], x["ld"], x["S0"], 0.3)
    if norm:
        ro = R.layer_norm(ro, w, b)[0]
    check_rows(o[:, :, None], ro, dtype)
    check_state(S, rS)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_run_as_it_is_used(dtype):
    """Serving: a padded batch of prompts, then tokens one by one, each through the output norm;
    and the prompt's training step through the norm's gradient.  One reference for all of it."""
    B, H, T, d, n_new = 2, 3, 170, 64, 3
    x, g = inputs(B, H, T + n_new, d, dtype, seed=12)
    gen = torch.Generator().manual_seed(2)
    w, b = (1 + 0.2 * torch.randn(d, generator=gen)).cuda(), torch.randn(d, generator=gen).cuda()
    part = lambda n, a, e: g[n][:, :, a:e].contiguous()  # noqa: E731
    y, S = fw.decay_prefill(part("q", 0, T), part("k", 0, T), part("v", 0, T), g["ld"], scale=0.2,
                            norm=(w, b))
    ys = [y]
    for t in range(T, T + n_new):
        one = [g[n][:, :, t].contiguous() for n in "qkv"]
        ys.append(fw.decay_step(*one, g["ld"], S, scale=0.2, norm=(w, b))[:, :, None])
    ro, rS, _ = R.forward(x["q"], x["k"], x["v"], x["ld"], None, 0.2)
    check_rows(torch.cat(ys, 2), R.layer_norm(ro, w, b)[0], dtype)
    check_state(S, rS)
    # a training step of the whole length
    o, _ = fw.decay_prefill(g["q"], g["k"], g["v"], g["ld"], scale=0.2)
    y, mean, rstd = fw.layer_norm(o, w, b)
    do, dw, db = fw.layer_norm_backward(g["do"], o, w, mean, rstd)
    dq, dk, dv, _ = fw.decay_backward(g["q"], g["k"], g["v"], g["ld"], do, scale=0.2)
    rdo, rdw, rdb = R.layer_norm_backward(x["do"], ro, w)
    ref = R.backward(x["q"], x["k"], x["v"], x["ld"], rdo, None, None, 0.2)
    # the chain rounds o and do once more each to the tensors' type
    tol = 2 * TOL[dtype]
    for a, r in zip((dq, dk, dv), ref[:3]):
        assert R.rel(a, r) <= tol
    assert R.rel(dw, rdw) <= tol and R.rel(db, rdb) <= tol


def test_prefill_in_two_parts_is_the_whole():
    x, g = inputs(1, 3, 333, 128, F32, seed=3)
    a = [g[n][:, :, :200].contiguous() for n in "qkv"]
    b = [g[n][:, :, 200:].contiguous() for n in "qkv"]
    o1, S = fw.decay_prefill(*a, g["ld"])
    o2, S2 = fw.decay_prefill(*b, g["ld"], S, S_T=S)          # S_T may be S0
    assert S2 is S
    ro, rS, _ = R.forward(x["q"], x["k"], x["v"], x["ld"])
    check_rows(torch.cat([o1, o2], 2), ro, F32)
    check_state(S, rS)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_in_place_state_of_long_chains(dtype):
    """S_T = S0 where a chain is split over the GPU: every part reads S0 before it is written."""
    x, g = inputs(1, 2, 2500, 128, dtype, seed=5, kind="slow")
    S = g["S0"].clone()
    o, _ = fw.decay_prefill(g["q"], g["k"], g["v"], g["ld"], S, S_T=S)
    ro, rS, _ = R.forward(x["q"], x["k"], x["v"], x["ld"], x["S0"])
    check_rows(o, ro, dtype)
    check_state(S, rS)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,H,T,d", [(1, 2, 3000, 128), (1, 5, 2049, 64), (2, 80, 700, 128)])
def test_long_and_many_chains(B, H, T, d, dtype):
    """Against the definition in 64 bits on the GPU (tensor products in place of einsum loops)."""
    x, g = inputs(B, H, T, d, dtype, seed=B + H, kind="slow" if H < 10 else "mixed")
    ln = torch.randint(0, T + 1, (B,), generator=torch.Generator().manual_seed(H)).int()
    o, S = fw.decay_prefill(g["q"], g["k"], g["v"], g["ld"], g["S0"], scale=0.1, lens=ln.cuda())
    got = fw.decay_backward(g["q"], g["k"], g["v"], g["ld"], g["do"], g["S0"], g["dS"], scale=0.1,
                            lens=ln.cuda())
    ro, rS, ref = _reference_on_gpu(g, ln, 0.1)
    check_rows(o, ro, dtype)
    check_state(S, rS)
    for a, r in zip(got[:3], ref[:3]):
        check_rows(a, r, dtype)
    check_state(got[3], ref[3])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,T", [(1, 32, 1300), (2, 13, 900), (3, 1, 5000), (1, 60, 1500)])
def test_backward_of_few_chains(B, H, T, d):
    """All three scans at once in one piece, or one after the other in segments, with a workspace of
    exactly the size that is asked for."""
    x, g = inputs(B, H, T, d, BF16, seed=T, kind="slow" if H < 10 else "mixed")
    ln = torch.tensor([T, T - 77, 3][:B], dtype=torch.int32)
    n = fw.decay_workspace(B, H, T, d, backward=True)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    for _ in range(2):
        got = fw.decay_backward(g["q"], g["k"], g["v"], g["ld"], g["do"], g["S0"], g["dS"], scale=0.1,
                                lens=ln.cuda(), workspace=ws)
    fw.check()
    _, _, ref = _reference_on_gpu(g, ln, 0.1)
    for a, r in zip(got[:3], ref[:3]):
        check_rows(a, r, BF16)
    check_state(got[3], ref[3])


def _reference_on_gpu(g, ln, scale):
    q, k, v, do = (g[n].double() for n in ("q", "k", "v", "do"))
    B, H, T, d = q.shape
    on = (torch.arange(T).view(1, T) < ln.view(B, 1)).cuda()
    ga = torch.exp(g["ld"].double()).view(1, H, 1, 1)
    S, D = g["S0"].double(), g["dS"].double()
    o, dq, dk, dv = (torch.zeros_like(q) for _ in range(4))
    for t in range(T):
        m = on[:, t].view(B, 1, 1, 1).double()
        S = S * (1 + m * (ga - 1)) + m * k[:, :, t, :, None] * v[:, :, t, None, :]
        o[:, :, t] = scale * (q[:, :, t, None, :] @ S)[:, :, 0] * m[..., 0]
        dq[:, :, t] = scale * (S @ do[:, :, t, :, None])[..., 0] * m[..., 0]
    for t in reversed(range(T)):
        m = on[:, t].view(B, 1, 1, 1).double()
        D = D + scale * m * q[:, :, t, :, None] * do[:, :, t, None, :]
        dk[:, :, t] = (D @ v[:, :, t, :, None])[..., 0] * m[..., 0]
        dv[:, :, t] = (k[:, :, t, None, :] @ D)[:, :, 0] * m[..., 0]
        D = D * (1 + m * (ga - 1))
    return o.cpu(), S.cpu(), [t.cpu() for t in (dq, dk, dv, D)]


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_same_bits_every_time_and_on_another_stream(dtype):
    x, g = inputs(2, 4, 500, 128, dtype, seed=7, kind="slow")
    def both(stream=None):
        o, S = fw.decay_prefill(g["q"], g["k"], g["v"], g["ld"], g["S0"], stream=stream)
        return [o, S, *fw.decay_backward(g["q"], g["k"], g["v"], g["ld"], g["do"], g["S0"],
                                         g["dS"], stream=stream)]
    first = both()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    a, b = both(s1), both(s2)                      # at once
    torch.cuda.synchronize()
    for r in (a, b, both()):
        assert all(torch.equal(x, y) for x, y in zip(first, r))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_captured_and_replayed(dtype):
    x, g = inputs(1, 4, 300, 64, dtype, seed=21)
    y, h = inputs(1, 4, 300, 64, dtype, seed=22)
    run = lambda z: [*fw.decay_prefill(z["q"], z["k"], z["v"], z["ld"], z["S0"]),  # noqa: E731
                     *fw.decay_backward(z["q"], z["k"], z["v"], z["ld"], z["do"], z["S0"], z["dS"])]
    want = [t.clone() for t in run(h)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run(g)
    for n in g:
        g[n].copy_(h[n])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_two_captured_graphs_with_workspaces_of_their_own():
    x, g = inputs(1, 6, 900, 64, F32, seed=23)
    y, h = inputs(1, 6, 900, 64, F32, seed=24)
    want = [fw.decay_prefill(z["q"], z["k"], z["v"], z["ld"])[0].clone() for z in (g, h)]
    graphs, outs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for z in (g, h):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(fw.decay_prefill(z["q"], z["k"], z["v"], z["ld"])[0])
        graphs.append(gr)
    torch.cuda.synchronize()
    for _ in range(10):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_binding_refusals_on_the_gpu():
    x, g = inputs(1, 2, 20, 64, BF16)
    with pytest.raises(ValueError, match="contiguous"):
        fw.decay_prefill(g["q"].transpose(1, 2).contiguous().transpose(1, 2), g["k"], g["v"], g["ld"])
    with pytest.raises(fw.FwError, match="ARG"):
        fw.decay_prefill(g["q"], g["k"], g["v"], g["ld"], o=g["q"])
    with pytest.raises(fw.FwError, match="DTYPE"):
        h = [g[n].half() for n in "qkv"]
        fw.decay_prefill(*h, g["ld"])
    with pytest.raises(fw.FwError, match="SHAPE"):
        z = torch.zeros(1, 2, 0, 64, device="cuda", dtype=BF16)
        fw.decay_prefill(z, z, z, g["ld"])
    with pytest.raises(fw.FwError, match="ALIGN"):
        flat = torch.zeros(1 * 2 * 20 * 64 + 1, device="cuda", dtype=BF16)
        fw.decay_prefill(flat[1:].view(1, 2, 20, 64), g["k"], g["v"], g["ld"])
    with pytest.raises(ValueError, match="norm_eps"):
        fw.decay_prefill(g["q"], g["k"], g["v"], g["ld"], norm=(None, None), norm_eps=-1.0)
    with pytest.raises(fw.FwError, match="SCRATCH"):
        f = [g[n].float().repeat(1, 1, 20, 1) for n in "qkv"]
        fw.decay_prefill(*f, g["ld"], workspace=torch.empty(16, device="cuda", dtype=torch.uint8))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", ["slow", "mixed"])
def test_padded_batch_of_more_chains_than_fit_at_once(kind, dtype):
    """13 x 13 chains of very different lengths (the longest start first)."""
    B, H, T, d = 13, 13, 420, 64
    x, g = inputs(B, H, T, d, dtype, seed=77, kind=kind)
    ln = torch.tensor([0, 420, 1, 300, 300, 128, 127, 5, 420, 64, 256, 17, 399], dtype=torch.int32)
    o, S = fw.decay_prefill(g["q"], g["k"], g["v"], g["ld"], g["S0"], lens=ln.cuda())
    got = fw.decay_backward(g["q"], g["k"], g["v"], g["ld"], g["do"], g["S0"], g["dS"],
                            lens=ln.cuda())
    fw.check()
    ro, rS, ref = _reference_on_gpu(g, ln, 1.0)
    check_rows(o, ro, dtype)
    check_state(S, rS)
    for a, r in zip(got[:3], ref[:3]):
        check_rows(a, r, dtype)
    check_state(got[3], ref[3])


@pytest.mark.parametrize("ld", [-0.46, -0.48, -3.0, -20.0, 0.46, 2.0])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_decays_on_both_sides_of_what_may_be_divided_by(ld, dtype):
    """Heads whose decay over 128 tokens is e^-60 and around it, forward and backward, where a
    chunk's end and a sequence's end fall together or not.  (Growing ones only for a few tokens:
    e^0.46 a token passes fp32 after 190.)"""
    T = 300 if ld < 0 else (100 if ld < 1 else 20)
    x, g = inputs(1, 1, T, 64, dtype, seed=31)
    l = torch.tensor([ld])
    o, S = fw.decay_prefill(g["q"], g["k"], g["v"], l.cuda())
    got = fw.decay_backward(g["q"], g["k"], g["v"], l.cuda(), g["do"])
    ro, rS, _ = R.forward(x["q"], x["k"], x["v"], l)
    ref = R.backward(x["q"], x["k"], x["v"], l, x["do"])
    check_rows(o, ro, dtype)
    check_state(S, rS)
    for a, r in zip(got[:3], ref[:3]):
        check_rows(a, r, dtype)


@pytest.mark.parametrize("ld", [-0.46, -0.2, -0.185, 0.0])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_large_values_do_not_overflow_inside_a_chunk(ld, dtype):
    """Rows of 1e4: scores of 1e9, outputs of 1e13 to 1e15, which no quotient of decays may carry
    past the largest fp32.  Scaling every input scales the outputs and their errors alike."""
    x, _ = inputs(1, 1, 300, 128, dtype, seed=57)
    x = {n: (t if n == "ld" else (t.double() * 1e4).to(t.dtype)) for n, t in x.items()}
    g = {n: t.cuda() for n, t in x.items()}
    l = torch.tensor([ld])
    o, S = fw.decay_prefill(g["q"], g["k"], g["v"], l.cuda(), g["S0"])
    got = fw.decay_backward(g["q"], g["k"], g["v"], l.cuda(), g["do"], g["S0"], g["dS"])
    fw.check()
    ro, rS, _ = R.forward(x["q"], x["k"], x["v"], l, x["S0"])
    ref = R.backward(x["q"], x["k"], x["v"], l, x["do"], x["S0"], x["dS"])
    check_rows(o, ro, dtype)
    check_state(S, rS)
    for a, r in zip(got[:3], ref[:3]):
        check_rows(a, r, dtype)
    check_state(got[3], ref[3])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_non_finite_values_stay_behind_their_chunk(dtype):
    x, g = inputs(1, 2, 300, 64, dtype, seed=2)
    v = g["v"].clone()
    v[0, 1, 200, 3] = float("inf")
    o, S = fw.decay_prefill(g["q"], g["k"], v, g["ld"])
    ro, rS, _ = R.forward(x["q"], x["k"], x["v"], x["ld"])
    check_rows(o[:, :1], ro[:, :1], dtype)
    check_rows(o[:, 1:, :128], ro[:, 1:, :128], dtype)
    assert not torch.isfinite(o[0, 1, 200:, 3]).any() and not torch.isfinite(S[0, 1, :, 3]).any()


@pytest.mark.parametrize("d", [64, 128])
def test_a_bounded_wait_reports_and_recovers(d):
    """A wait that nothing ends runs out: fw_check reports it, and the next call is right."""
    L = fw.lib()
    x, g = inputs(1, 2, 700, d, BF16, seed=1)
    L.fw_set_wait_limit_us(2000)
    L.fw_debug_force_timeout(1)
    try:
        fw.decay_prefill(g["q"], g["k"], g["v"], g["ld"])
        with pytest.raises(fw.FwError) as ei:
            fw.check()
        assert ei.value.status == -7
    finally:
        L.fw_debug_force_timeout(0)
        L.fw_set_wait_limit_us(0)
    fw.check()
    o, S = fw.decay_prefill(g["q"], g["k"], g["v"], g["ld"])
    ro, rS, _ = R.forward(x["q"], x["k"], x["v"], x["ld"])
    check_rows(o, ro, BF16)
    check_state(S, rS)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_offsets_beyond_32_bits(dtype):
    """One chain of 2^24 + 300 tokens: 2^31 + 38400 elements.  With g = e^-0.5 a row depends on the
    500 tokens before it alone (e^-250 of the rest is left)."""
    T, d, n = 2 ** 24 + 300, 128, 700
    gen = torch.Generator(device="cuda").manual_seed(3)
    t = [torch.randn(1, 1, T, d, device="cuda", dtype=dtype, generator=gen) for _ in range(3)]
    ld = torch.tensor([-0.5])
    o, S = fw.decay_prefill(*t, ld.cuda())
    fw.check()
    cut = [z[:, :, -n:].clone() for z in t]
    ro, rS, _ = R.forward(*cut, ld)
    check_rows(o[:, :, -200:], ro[:, :, -200:], dtype)
    check_state(S, rS)
    first = R.forward(*[z[:, :, :200].clone() for z in t], ld)[0]
    check_rows(o[:, :, :200], first, dtype)
    if dtype == BF16:
        do = torch.randn(1, 1, T, d, device="cuda", dtype=dtype, generator=gen)
        got = fw.decay_backward(*t, ld.cuda(), do)
        fw.check()
        ref = R.backward(*cut, ld, do[:, :, -n:].clone())
        for a, r in zip(got[:3], ref[:3]):
            check_rows(a[:, :, -200:], r[:, :, -200:], dtype)


def test_step_offsets_beyond_32_bits():
    B, H, d = 2 ** 13 + 1, 16, 128            # 2^31 + 2^18 state elements
    gen = torch.Generator(device="cuda").manual_seed(5)
    S = torch.randn(B, H, d, d, device="cuda", generator=gen)
    q, k, v = (torch.randn(B, H, d, device="cuda", generator=gen) for _ in range(3))
    ld = decays(H).cuda()
    before = S[-1:].clone()
    o = fw.decay_step(q, k, v, ld, S)
    ro, rS, _ = R.forward(*(z[-1:, :, None] for z in (q, k, v)), ld, before)
    check_rows(o[-1:, :, None], ro, F32)
    check_state(S[-1:], rS)
