"""The calls of a mixer layer together, as they are used: convolutions of q, k, v, the scan, the gated norm, and the
residual norm before the next block; prompts, tokens behind them, and a training step through the decayed scan.

Tolerances.  Each stage rounds its rows to the type once (bf16: 2^-8 at most) and is otherwise as near as its own test
says; an error made before a stage reaches its output through it.  A convolution's taps and silu pass a relative
error of their rows on with about its size (weights of norm one, silu's slope at most 1.1), the scan's product of three
rows (q, k, v) with about the sum of the three, the norm with its size: in all about 1 + 3 + 1 + 1 + 1 roundings of
random sign against the 64-bit layer, sqrt(7) 2^-8 / sqrt(3), with the scan's own two: 7e-3, and three times that for
one row of few: 2e-2.  fp32: the same count of 1e-5 (the scan's) and 4e-6: 4e-5.
"""
import pytest
import torch

from linear_token_mixer_gb300 import fw

import mixer_ref as R

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TOL = {F32: 4e-5, BF16: 2e-2}


def layer(B, H, G, T, d, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed)

    def rn(*s, std=1.0):
        return torch.randn(*s, generator=gen) * std

    p = {"cw" + n: rn(h, d, 4, std=0.5) for n, h in (("q", G), ("k", G), ("v", H))}
    p.update({"cb" + n: rn(h, d, std=0.1) for n, h in (("q", G), ("k", G), ("v", H))})
    p.update(ld=-(1 + 7 * torch.rand(H, generator=gen)), bias=-3 + rn(H), skip=1 + rn(H, std=0.2), nw=1 + rn(H, d, std=0.2),
             rw=1 + rn(H * d, std=0.2), rs=rn(H * d, std=0.3))
    x = {n: rn(B, h, T, d).to(dtype) for n, h in (("q", G), ("k", G), ("v", H), ("z", H))}
    x["dt"] = rn(B, H, T).to(dtype)
    x["stream"] = rn(B, T, H * d).to(dtype)
    return p, x


def forward(p, x, scale, state=None, lens=None):
    """(y, stream) of a prompt and the states behind it: three convolutions' and the scan's."""
    state = state or {}
    c = {}
    for n in "qkv":
        c[n], state[n] = fw.conv_prefill(x[n], p["cw" + n], p["cb" + n], state.get(n), lens=lens)
    o, state["S"] = fw.select_prefill(c["q"], c["k"], c["v"], x["dt"], p["ld"], state.get("S"), dt_bias=p["bias"],
                                      softplus=True, skip=p["skip"], scale=scale, lens=lens)
    y, _, _, _ = fw.gated_norm(o, p["nw"], gate=x["z"], rms=True, stats=False)
    B, H, T, d = y.shape
    rows = y.transpose(1, 2).reshape(B, T, H * d)
    out, stream, _, _ = fw.gated_norm(x["stream"], p["rw"], residual=rows, scale=p["rs"], rms=True, stats=False)
    return out, stream, state


def token(p, x, t, scale, state):
    one = {n: x[n][:, :, t].contiguous() for n in ("q", "k", "v", "z", "dt")}
    c = {n: fw.conv_step(one[n], p["cw" + n], p["cb" + n], state[n]) for n in "qkv"}
    o = fw.select_step(c["q"], c["k"], c["v"], one["dt"], p["ld"], state["S"], dt_bias=p["bias"], softplus=True,
                       skip=p["skip"], scale=scale)
    B, H, d = o.shape
    y, _, _, _ = fw.gated_norm(o.view(B, H, 1, d), p["nw"], gate=one["z"].view(B, H, 1, d), rms=True, stats=False)
    out, stream, _, _ = fw.gated_norm(x["stream"][:, t].contiguous(), p["rw"], residual=y.view(B, H * d), scale=p["rs"],
                                      rms=True, stats=False)
    return out, stream


def exact(p, x, scale, lens=None):
    p, x = ({n: R.f64(t) for n, t in z.items()} for z in (p, x))
    c = {n: R.conv(x[n], p["cw" + n], p["cb" + n], None, True, lens)[0] for n in "qkv"}
    o, S = R.select(c["q"], c["k"], c["v"], x["dt"], p["ld"], None, p["bias"], True, p["skip"], scale, lens)
    y = R.gated(o, p["nw"], gate=x["z"], rms=True)[0]
    B, H, T, d = y.shape
    out, stream, _, _ = R.gated(x["stream"], p["rw"], residual=y.transpose(1, 2).reshape(B, T, H * d), scale=p["rs"], rms=True)
    return out, stream, S


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,H,G,T,d", [(2, 4, 2, 150, 64), (1, 3, 1, 300, 128)])
def test_a_prompt_and_tokens_behind_it(B, H, G, T, d, dtype):
    p, x = layer(B, H, G, T, d, dtype, seed=T)
    scale, cut = d ** -0.5, T - 9
    want, ws, wS = exact(p, x, scale)
    pg, xg = ({n: t.cuda() for n, t in z.items()} for z in (p, x))
    out, stream, _ = forward(pg, xg, scale)
    assert R.rel(out, want) <= TOL[dtype] and R.rel(stream, ws) <= TOL[dtype]
    head = {n: (t[:, :cut] if n == "stream" else t[:, :, :cut]).contiguous() for n, t in xg.items()}
    o1, s1, state = forward(pg, head, scale)
    rows = [o1]
    for t in range(cut, T):
        rows.append(token(pg, xg, t, scale, state)[0].unsqueeze(1))
    fw.check()
    assert R.rel(torch.cat(rows, 1), want) <= TOL[dtype]
    # the state: k and v rounded once more than their tests', 2^-8 each
    assert R.rel_rows(state["S"], wS, 2) <= TOL[dtype]


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_padded_batch_of_prompts(dtype):
    B, H, G, T, d = 4, 4, 1, 200, 64
    p, x = layer(B, H, G, T, d, dtype, seed=1)
    lens = torch.tensor([200, 0, 3, 131], dtype=torch.int32)
    want, _, wS = exact(p, x, 0.125, lens)
    for b, n in enumerate(lens.tolist()):
        for name in ("q", "k", "v", "dt"):
            x[name][b, :, n:] = float("nan")
    pg, xg = ({n: t.cuda() for n, t in z.items()} for z in (p, x))
    out, _, state = forward(pg, xg, 0.125, lens=lens.cuda())
    for b, n in enumerate(lens.tolist()):
        if n:
            assert R.rel(out[b, :n], want[b, :n]) <= TOL[dtype]
    assert torch.isfinite(out).all() and R.rel_rows(state["S"], wS, 2) <= TOL[dtype]


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_training_step_through_the_decayed_scan(dtype):
    """conv -> decayed scan -> gated norm, and back: every gradient against the 64-bit layer's."""
    B, H, T, d = 2, 3, 200, 64
    p, x = layer(B, H, H, T, d, dtype, seed=3)
    ld, scale = -torch.tensor([0.01, 0.2, 1.5]), 0.125
    dy = torch.randn(B, H, T, d, generator=torch.Generator().manual_seed(9)).to(dtype)
    pg, xg = ({n: t.cuda() for n, t in z.items()} for z in (p, x))
    c = {n: fw.conv_prefill(xg[n], pg["cw" + n], pg["cb" + n])[0] for n in "qkv"}
    o, _ = fw.decay_prefill(c["q"], c["k"], c["v"], ld.cuda(), scale=scale)
    y, _, _, rstd = fw.gated_norm(o, pg["nw"], gate=xg["z"], rms=True)
    do, dnw, _, dz, _, _ = fw.gated_norm_backward(dy.cuda(), o, pg["nw"], None, None, rstd, gate=xg["z"], rms=True)
    dc = dict(zip("qkv", fw.decay_backward(c["q"], c["k"], c["v"], ld.cuda(), do, scale=scale)))
    got = {"nw": dnw, "z": dz}
    for n in "qkv":
        got[n], got["cw" + n], got["cb" + n], _ = fw.conv_backward(dc[n], xg[n], pg["cw" + n], pg["cb" + n])
    fw.check()
    leaf = {n: R.f64(t).requires_grad_() for n, t in {**p, **x}.items()}
    r = {n: R.conv(leaf[n], leaf["cw" + n], leaf["cb" + n])[0] for n in "qkv"}
    lag = torch.arange(T).view(T, 1) - torch.arange(T).view(1, T)
    decay = torch.exp(ld.double().view(H, 1, 1) * lag.clamp_min(0)) * (lag >= 0)
    ro = scale * torch.einsum("bhts,bhsd->bhtd", torch.einsum("bhtd,bhsd->bhts", r["q"], r["k"]) * decay, r["v"])
    ry = R.gated(ro, leaf["nw"], gate=leaf["z"], rms=True)[0]
    assert R.rel(y, ry.detach()) <= TOL[dtype]
    want = dict(zip(got, torch.autograd.grad((ry * R.f64(dy)).sum(), [leaf[n] for n in got])))
    for n in got:
        assert R.rel(got[n], want[n]) <= 2 * TOL[dtype], n   # (twice the layer's stages)


def _calls():
    g = torch.Generator().manual_seed(1)
    rn = lambda *s, dtype=BF16: torch.randn(*s, generator=g).to(dtype).cuda()  # noqa: E731
    B, H, G, T, d = 2, 4, 2, 300, 64
    q, k, v, dt = rn(B, G, T, d), rn(B, G, T, d), rn(B, H, T, d), rn(B, H, T)
    ld, bias, skip, S = -rn(H, dtype=F32).abs(), rn(H, dtype=F32), rn(H, dtype=F32), rn(B, H, d, d, dtype=F32)
    kw = dict(softplus=True)
    yield "select_prefill", [q, k, v, dt, ld, S, bias, skip], lambda q, k, v, dt, l, s, b, sk, **o: fw.select_prefill(
        q, k, v, dt, l, s, dt_bias=b, skip=sk, **kw, **o)
    yield "select_step", [t[:, :, 0].contiguous() for t in (q, k, v, dt)] + [ld, S, bias, skip], \
        lambda q, k, v, dt, l, s, b, sk, **o: (fw.select_step(q, k, v, dt, l, s, dt_bias=b, skip=sk, **kw, **o),)
    w, cb, st, dy, ds = rn(H, d, 4, dtype=F32), rn(H, d, dtype=F32), rn(B, H, 3, d), rn(B, H, T, d), rn(B, H, 3, d)
    yield "conv_prefill", [v, w, cb, st], lambda *a, **o: fw.conv_prefill(*a, **o)
    yield "conv_backward", [dy, v, w, cb, st, ds], lambda *a, **o: fw.conv_backward(*a, **o)
    yield "conv_step", [v[:, :, 0].contiguous(), w, cb, st], lambda *a, **o: (fw.conv_step(*a, **o),)
    x, z, r = rn(900, 256), rn(900, 256), rn(900, 256)
    nw, nb, sc = rn(256, dtype=F32), rn(256, dtype=F32), rn(256, dtype=F32)
    mean, rstd = rn(900, dtype=F32), rn(900, dtype=F32)
    yield "gated_norm", [x, nw, nb, z, r, sc], lambda x, w, b, z, r, s, **o: fw.gated_norm(
        x, w, b, gate=z, residual=r, scale=s, **o)
    yield "gated_norm_backward", [x, x.flip(0), nw, nb, mean, rstd, z, r, sc], lambda dy, x, w, b, m, rs, z, r, s, **o: \
        fw.gated_norm_backward(dy, x, w, b, m, rs, gate=z, residual=r, scale=s, **o)


NAMES = ["select_prefill", "select_step", "conv_prefill", "conv_backward", "conv_step", "gated_norm",
         "gated_norm_backward"]


@pytest.mark.parametrize("name", NAMES)
def test_temporaries_of_a_call_on_another_stream(name):
    """The memory of what a caller gives back is not handed out again while the kernels still wait to read it."""
    _, args, call = next(c for c in _calls() if c[0] == name)
    want = [t for t in call(*[a.clone() for a in args]) if t is not None]
    s = torch.cuda.Stream()
    call(*[a.clone() for a in args], stream=s)     # (what a first use loads is loaded)
    torch.full_like(args[0], 0.0)
    with torch.cuda.stream(s):
        torch.cuda._sleep(1000)
    torch.cuda.synchronize()
    tmp = [a.clone() for a in args]
    at = {t.data_ptr() for t in tmp}
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)             # about 100 ms: the call's kernels wait behind it
    got = call(*tmp, stream=s)
    del tmp
    new = [torch.full_like(a, float("nan")) for a in args for _ in range(2)]
    assert not s.query()                           # still waiting
    assert not at & {t.data_ptr() for t in new}
    torch.cuda.synchronize()
    fw.check()
    for a, b in zip((t for t in got if t is not None), want):
        assert torch.equal(a, b)


def _leave(value):
    """Kernels whose tiles, states and products stay behind in the shared and tensor memory of every SM."""
    x = torch.full((19, 16, 256, 128), value, device="cuda", dtype=BF16)
    fw.decay_prefill(x, x, x, torch.zeros(16, device="cuda"))
    fw.gated_norm(torch.full((2000, 8192), value, device="cuda"), gate=torch.full((2000, 8192), value, device="cuda"))
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [1, 2, 63, 65, 130, 257])
def test_behind_kernels_that_leave_nan(T, d, dtype):
    """The same bits behind kernels that left NaN everywhere as behind kernels that left zeros."""
    gen = torch.Generator().manual_seed(T)
    rn = lambda *s, t=dtype: torch.randn(*s, generator=gen).to(t).cuda()  # noqa: E731
    B, H, G = 2, 4, 2
    q, k, v, dt, S = rn(B, G, T, d), rn(B, G, T, d), rn(B, H, T, d), rn(B, H, T), rn(B, H, d, d, t=F32)
    ld, skip = -8 * torch.rand(H, generator=gen).cuda(), rn(H, t=F32)
    w, dy, nw = rn(H, d, 4, t=F32), rn(B, H, T, d), rn(H, d, t=F32)
    lens = torch.tensor([T, T // 2], dtype=torch.int32).cuda()
    got = []
    for value in (float("nan"), 0.0):
        _leave(value)
        a = [*fw.select_prefill(q, k, v, dt, ld, S, softplus=True, skip=skip, lens=lens)]
        _leave(value)
        a += [*fw.conv_prefill(v, w, lens=lens), *fw.conv_backward(dy, v, w, lens=lens)[:3]]
        _leave(value)
        y, _, mean, rstd = fw.gated_norm(v, nw, gate=dy)
        a += [y, *fw.gated_norm_backward(dy, v, nw, None, mean, rstd, gate=dy)[:4]]
        got.append([t.clone() for t in a])
    fw.check()
    for a, b in zip(*got):
        assert torch.isfinite(a).all() and torch.equal(a, b)


def test_one_workspace_for_calls_in_turn():
    """A workspace holds nothing that the next call needs, of whichever call it was."""
    gen = torch.Generator().manual_seed(2)
    rn = lambda *s, t=BF16: torch.randn(*s, generator=gen).to(t).cuda()  # noqa: E731
    B, H, T, d = 2, 2, 700, 64
    q, v, dt, ld = rn(B, H, T, d), rn(B, H, T, d), rn(B, H, T), -torch.rand(H, generator=gen).cuda()
    w, nw = rn(H, d, 4, t=F32), rn(d, t=F32)
    rstd = torch.rand(B, H, T, generator=gen).cuda()
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")

    def run(**kw):
        return [*fw.select_prefill(q, q, v, dt, ld, softplus=True, **kw), *fw.conv_backward(q, v, w, **kw)[:3],
                *fw.gated_norm_backward(q, v, nw, None, None, rstd, rms=True, **kw)[:3],
                *fw.decay_backward(q, q, v, ld, v, **kw)[:3]]
    want = run()
    for _ in range(2):
        assert all(torch.equal(a, b) for a, b in zip(run(workspace=ws), want))
