"""Selective scan on the GPU against the 64-bit token recurrence.

Tolerances (relative L2 of a whole output, and of every chain), as those of the decayed scans, whose sums these
are.  fp32: sums of up to d + C + 3 rounded operations of relative size 2^-24 on terms of random sign, and
decays whose exponents are sums in 64 bits, each exponential two ulp off: 1e-5.  S_T: its operands carry 22 bits or
more: 1e-5.  bf16 rows are rounded once, and the masked scores and the carried state once each (at most 2^-8
relative): 3.9e-3 as an upper estimate of the relative L2, and as much again for one chain of few rows: 8e-3.
"""
import pytest
import torch

from linear_token_mixer_gb300 import fw

import mixer_ref as R

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TOL = {F32: 1e-5, BF16: 8e-3}
TOL_STATE = 1e-5


def inputs(B, H, G, T, d, dtype, seed=0, rate=(1.0, 16.0), dt_type=None, mean=-4.0):
    """Steps of about softplus(mean), log decays of -rate a step."""
    gen = torch.Generator().manual_seed(seed)

    def rn(*s):
        return torch.randn(*s, generator=gen)

    x = {"q": rn(B, G, T, d).to(dtype), "k": rn(B, G, T, d).to(dtype), "v": rn(B, H, T, d).to(dtype),
         "dt": (rn(B, H, T)).to(dt_type or dtype), "ld": -(rate[0] + (rate[1] - rate[0]) * torch.rand(H, generator=gen)),
         "S0": rn(B, H, d, d), "bias": mean + rn(H), "skip": 1 + 0.3 * rn(H)}
    return x, {n: t.cuda() for n, t in x.items()}


def run(z, S0=True, skip=True, softplus=True, **kw):
    return fw.select_prefill(z["q"], z["k"], z["v"], z["dt"], z["ld"], z["S0"] if S0 else None,
                             dt_bias=z["bias"] if softplus else None, softplus=softplus,
                             skip=z["skip"] if skip else None, **kw)


def ref(z, S0=True, skip=True, softplus=True, **kw):
    return R.select(z["q"], z["k"], z["v"], z["dt"], z["ld"], z["S0"] if S0 else None,
                    z["bias"] if softplus else None, softplus, z["skip"] if skip else None, **kw)


def check(got, want, dtype):
    (o, S), (ro, rS) = got, want
    assert o.dtype == dtype and S.dtype == F32
    assert R.rel(o, ro) <= TOL[dtype] and R.rel_rows(o, ro, 2) <= TOL[dtype]
    assert R.rel_rows(S, rS, 2) <= TOL_STATE


SIZES = [(1, 1, 1, 1), (2, 2, 1, 2), (1, 3, 3, 63), (1, 2, 1, 64), (2, 6, 2, 65), (1, 2, 2, 127), (1, 1, 1, 128),
         (1, 2, 1, 129), (1, 4, 2, 257), (2, 3, 1, 400)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,G,T", SIZES)
@pytest.mark.parametrize("full", [False, True])
def test_prefill(B, H, G, T, d, dtype, full):
    x, g = inputs(B, H, G, T, d, dtype, seed=T)
    kw = dict(S0=full, skip=full, scale=0.25)
    got = run(g, **kw)
    fw.check()
    check(got, ref(x, **kw), dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rate,mean", [((0.0, 0.0), -1.0), ((0.01, 0.1), -3.0), ((1.0, 2.0), 0.0), ((5.0, 9.0), 1.0),
                                       ((16.0, 16.0), 2.0), ((200.0, 300.0), 1.0), ((15.0, 30.0), -5.0)])
def test_decays_from_none_to_all(rate, mean, d, dtype):
    """Chunks from no decay at all over those on either side of e^-24 to tokens that keep nothing."""
    x, g = inputs(1, 4, 2, 390, d, dtype, seed=3, rate=rate, mean=mean)
    got = run(g)
    fw.check()
    check(got, ref(x), dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dt_type", [F32, BF16])
def test_steps_of_either_type_as_they_are(dt_type, dtype):
    """Without softplus, fp32 steps beside bf16 rows; most of them zero: such a token changes nothing.  bf16 steps
    beside fp32 rows are refused."""
    x, _ = inputs(2, 4, 4, 200, 64, dtype, seed=5, dt_type=dt_type)
    if dtype == F32 and dt_type == BF16:
        with pytest.raises(ValueError):
            run({n: t.cuda() for n, t in x.items()}, softplus=False)
        return
    x["dt"] = (x["dt"].float().abs() * 0.1 * (x["dt"].float() > 0.8)).to(dt_type)
    g = {n: t.cuda() for n, t in x.items()}
    got = run(g, softplus=False)
    check(got, ref(x, softplus=False), dtype)
    x["dt"] = torch.zeros_like(x["dt"])
    g["dt"] = x["dt"].cuda()
    o, S = run(g, softplus=False, skip=False)
    assert torch.equal(S.cpu(), x["S0"])
    check((o, S), ref(x, softplus=False, skip=False), dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("scale", [0.0, -3.0, 1e-6])
def test_scales(scale, dtype):
    """A scale of zero leaves skip v alone; a small one makes skip v almost all of a row."""
    x, g = inputs(1, 3, 1, 300, 64, dtype, seed=7)
    check(run(g, scale=scale), ref(x, scale=scale), dtype)
    if scale:
        check(run(g, scale=scale, skip=False), ref(x, scale=scale, skip=False), dtype)
    else:
        assert not run(g, scale=scale, skip=False)[0].any()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("every", [1, 3, 40, 128])
def test_states_that_start_afresh(every, dtype):
    """Steps so long that their decay is zero, between mild ones: sequences packed in one row."""
    x, _ = inputs(1, 2, 1, 300, 64, dtype, seed=6, dt_type=F32, rate=(1.0, 2.0))
    x["dt"] = x["dt"].abs() * 0.02
    x["dt"][:, :, ::every] = 400.0
    x["k"][:, :, ::every] *= 2.0 ** -12            # (their writes are as large as the others')
    g = {n: t.cuda() for n, t in x.items()}
    got = run(g, softplus=False)
    check(got, ref(x, softplus=False), dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [1, 70, 300])
def test_padded_batch(T, d, dtype):
    B, H, G = 5, 4, 2
    x, _ = inputs(B, H, G, T, d, dtype, seed=T)
    lens = torch.tensor([T, 0, 1, T // 2, T + 9], dtype=torch.int32)
    want = ref(x, lens=lens)
    for b, n in enumerate(R.ends(lens, B, T)):     # what lies behind a row's end is never used
        for name in "qkv":
            x[name][b, :, n:] = float("nan")
        x["dt"][b, :, n:] = float("inf")
    g = {n: t.cuda() for n, t in x.items()}
    lg = lens.cuda()
    check(run(g, lens=lg), want, dtype)
    o = torch.full((B, H, T, d), 7.0, dtype=dtype, device="cuda")
    S = g["S0"].clone()
    g["S0"] = S
    got = run(g, lens=lg, o=o, S_T=S)              # in place, rows behind the ends as they were
    assert got[0] is o and got[1] is S
    kept = o.cpu()
    for b, n in enumerate(R.ends(lens, B, T)):
        assert (kept[b, :, n:] == 7.0).all()
        kept[b, :, n:] = 0
    check((kept, S), want, dtype)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,G,T,ragged", [(1, 1, 1, 2100, False), (1, 3, 1, 1500, True), (2, 2, 2, 1999, True),
                                            (1, 40, 5, 900, False)])
@pytest.mark.parametrize("rate", [(0.01, 0.02), (1.0, 16.0)])
def test_chains_in_segments(B, H, G, T, ragged, d, rate):
    x, g = inputs(B, H, G, T, d, BF16, seed=T, rate=rate)
    lens = torch.tensor([T - 131, 700][:B], dtype=torch.int32) if ragged else None
    want = ref(x, lens=lens)
    lg = None if lens is None else lens.cuda()
    check(run(g, lens=lg), want, BF16)
    S = g["S0"]
    check(run(g, lens=lg, S_T=S), want, BF16)


@pytest.mark.parametrize("d", [64, 128])
def test_chains_of_many_chunks(d):
    """More chunks in one piece than a CTA has warps to form their tables."""
    x, g = inputs(1, 80, 1, 3700, d, BF16, seed=5, rate=(0.05, 16.0))
    check(run(g), ref(x), BF16)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_more_chains_than_multiprocessors(dtype):
    B, H, G, T, d = 40, 8, 4, 140, 64
    x, g = inputs(B, H, G, T, d, dtype, seed=8)
    lens = torch.randint(0, T + 1, (B,), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    check(run(g, lens=lens.cuda()), ref(x, lens=lens), dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128])
def test_a_prompt_in_parts_and_token_by_token(d, dtype):
    B, H, G, T = 2, 6, 2, 150
    x, g = inputs(B, H, G, T, d, dtype, seed=2)
    ro, rS = ref(x)
    cut = lambda z, a, b: {n: (t[:, :, a:b].contiguous() if n in ("q", "k", "v", "dt") else t) for n, t in z.items()}  # noqa: E731
    z = cut(g, 0, 131)
    o1, S = run(z)
    rows = [o1]
    for t in range(131, T):
        z = {n: (y[:, :, t].contiguous() if n in ("q", "k", "v", "dt") else y) for n, y in g.items()}
        o = fw.select_step(z["q"], z["k"], z["v"], z["dt"], z["ld"], S, dt_bias=z["bias"], softplus=True, skip=z["skip"])
        rows.append(o.unsqueeze(2))
    check((torch.cat(rows, 2), S), (ro, rS), dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("softplus", [False, True])
def test_step_alone(softplus, dtype):
    for B, H, G, d in ((1, 1, 1, 64), (3, 6, 2, 128), (64, 8, 8, 128)):
        x, g = inputs(B, H, G, 1, d, dtype, seed=B, dt_type=F32)
        one = {n: (t[:, :, 0].contiguous() if n in ("q", "k", "v", "dt") else t) for n, t in g.items()}
        S = one["S0"].clone()
        o = fw.select_step(one["q"], one["k"], one["v"], one["dt"], one["ld"], S,
                           dt_bias=one["bias"] if softplus else None, softplus=softplus, scale=0.5)
        ro, rS = ref(x, skip=False, softplus=softplus, scale=0.5)
        assert R.rel(o, ro[:, :, 0]) <= TOL[dtype] and R.rel_rows(S, rS, 2) <= TOL_STATE
        # A chain here is one row, whose sum over the state's rows may cancel: where little of the state is kept
        # o = scale dt (q.k) v, and q.k of one of 512 chains is 1e-3 for terms of 64.  Each term is rounded at most 32 times
        # on its way (16 rows of a thread, 8 or 16 threads, products, decay and scale): 32 2^-24 of the terms' sum.
        terms = 0.5 * torch.einsum("bhi,bhij->bhj", R.f64(x["q"][:, :, 0]).abs().repeat_interleave(H // G, 1), rS.abs())
        off = (o.cpu().double() - ro[:, :, 0]).norm(dim=-1)
        assert (off <= TOL[dtype] * ro[:, :, 0].norm(dim=-1) + 32 * 2.0 ** -24 * terms.norm(dim=-1)).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,H,T", [(1, 2, 300), (1, 1, 2100)])
def test_values_that_are_not_finite(B, H, T, dtype):
    """An infinity or NaN in v reaches the rows that depend on it: its own column, from its token on."""
    d, bad = 64, [(0, 0, 140, 5, float("inf")), (0, H - 1, T - 3, 63, float("nan"))]
    x, _ = inputs(B, H, 1, T, d, dtype, seed=4, rate=(0.1, 0.2))
    want, _ = ref(x)
    for b, h, t, c, value in bad:
        x["v"][b, h, t, c] = value
    o, S = run({n: y.cuda() for n, y in x.items()})
    hit = torch.zeros(B, H, T, d, dtype=torch.bool)
    for b, h, t, c, _ in bad:
        hit[b, h, t:, c] = True
    o = o.cpu()
    assert not torch.isfinite(o[hit]).any()
    assert torch.isfinite(o[~hit]).all()
    assert R.rel(torch.where(hit, 0.0, o.double()), torch.where(hit, 0.0, want)) <= TOL[dtype]
    assert not torch.isfinite(S[0, 0, :, 5]).any() and torch.isfinite(S[0, 0, :, 6]).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_offsets_beyond_32_bits(dtype):
    """The last chain of rows of which v alone holds more than 2^31 elements."""
    d, T, B, H = 128, 1100, 128, 128
    if torch.cuda.mem_get_info()[0] < (90 << 30):
        pytest.skip("needs 90 GB")
    x, _ = inputs(1, 1, 1, T, d, dtype, seed=1)
    v = torch.zeros(B, H, T, d, dtype=dtype, device="cuda")
    v[-1, -1] = x["v"][0, 0].cuda()
    q, k = (x[n].cuda().expand(B, 1, T, d).contiguous() for n in "qk")
    dt = x["dt"].cuda().expand(B, H, T).contiguous()
    ld, bias, skip = (x[n].cuda().expand(H).contiguous() for n in ("ld", "bias", "skip"))
    o, S = fw.select_prefill(q, k, v, dt, ld, dt_bias=bias, softplus=True, skip=skip)
    fw.check()
    check((o[-1:, -1:], S[-1:, -1:]), ref(x, S0=False), dtype)
    assert not o[0, 0].any() and not S[5, 7].any()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,H,G,T,d", [(3, 4, 2, 300, 64), (1, 2, 1, 2100, 128), (14, 12, 3, 150, 64), (2, 3, 3, 50, 128)])
def test_replayed_with_other_inputs(B, H, G, T, d, dtype):
    _, z = inputs(B, H, G, T, d, dtype, 1)
    z["lens"] = torch.full((B,), T, dtype=torch.int32, device="cuda")
    run(z, lens=z["lens"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run(z, lens=z["lens"])
    for seed in (2, 3):
        _, y = inputs(B, H, G, T, d, dtype, seed, rate=(0.01, 3.0 * seed))
        y["lens"] = torch.randint(0, T + 1, (B,), generator=torch.Generator().manual_seed(seed), dtype=torch.int32).cuda()
        want = [t.clone() for t in run(y, lens=y["lens"])]
        for n in z:
            z[n].copy_(y[n])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    fw.check()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,T", [(1, 2, 300), (1, 1, 3000)])
def test_a_wait_that_runs_out_is_reported(B, H, T, d):
    x, g = inputs(B, H, 1, T, d, BF16, seed=1)
    L = fw.lib()
    L.fw_set_wait_limit_us(2000)
    L.fw_debug_force_timeout(1)
    try:
        run(g)
        with pytest.raises(fw.FwError, match="TIMEOUT"):
            fw.check()
    finally:
        L.fw_debug_force_timeout(0)
        L.fw_set_wait_limit_us(0)
    got = run(g)
    fw.check()
    check(got, ref(x), BF16)


def test_two_calls_at_once_with_a_workspace_each():
    zs = [inputs(1, 3, 1, 700, 64, BF16, seed=s)[1] for s in (1, 2)]
    want = [[t.clone() for t in run(z)] for z in zs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in zs]
    for _ in range(5):
        got = [run(z, stream=s) for z, s in zip(zs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(u, v) for u, v in zip(a, b))
