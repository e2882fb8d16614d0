"""Decayed scans of rows that hold infinities and NaN: the causal mask keeps them from every row that does not
depend on them.

Tolerances of the rows that they do not reach, element by element relative to the recurrence over
absolute values: fp32 1e-5 (6.2e-6: a product of split operands leaves out 2^-22 three times over, in two
products, and the sums take 40 additions of at most 2^-23), bf16 8e-3 (7.83e-3: an operand and the row
rounded, 2^-8 each); rows behind an output norm relative L2, 8e-3 and 1e-5, as without such values.
"""
import pytest
import torch

from linear_token_mixer_gb300 import fw

import decay_ref as R

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TOL = {F32: 1e-5, BF16: 8e-3}


def inputs(B, H, T, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = {n: torch.randn(B, H, T, d, generator=g).to(dtype) for n in ("q", "k", "v", "do")}
    x.update(S0=torch.randn(B, H, d, d, generator=g), dS=torch.randn(B, H, d, d, generator=g))
    return x, {n: t.cuda() for n, t in x.items()}


def check_rows(got, ref, size, where, dtype):
    got = got.cpu().double()[where]
    assert torch.isfinite(got).all()
    assert ((got - ref[where]).abs() <= TOL[dtype] * size[where]).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ld", [-0.05, -0.5])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("T,t", [(300, 200), (300, 0), (128, 127), (40, 17), (1300, 700)])
def test_non_finite_values_reach_no_row_before_them(T, t, value, ld, d, dtype):
    """A value that is not finite reaches its own column of its own row and of later ones, and of the
    state, and nothing else, also within the tokens that are worked on together (T = 1300: chains
    split over the GPU)."""
    B, H, c = 1, 2, 5
    x, g = inputs(B, H, T, d, dtype, seed=11)
    y = {n: z.abs() for n, z in x.items()}
    l = torch.tensor([ld, ld])
    at = torch.arange(T)
    v = g["v"].clone()
    v[0, 1, t, c] = value
    o, S = fw.decay_prefill(g["q"], g["k"], v, l.cuda(), g["S0"])
    in_place = g["S0"].clone()
    o2, _ = fw.decay_prefill(g["q"], g["k"], v, l.cuda(), in_place, S_T=in_place)
    _, wS = fw.decay_prefill(g["q"], g["k"], g["v"], l.cuda(), g["S0"])
    fw.check()
    hit = torch.zeros(B, H, T, d, dtype=torch.bool)
    hit[0, 1, t:, c] = True
    ref, size = (R.forward(z["q"], z["k"], z["v"], l, z["S0"])[0] for z in (x, y))
    for a in (o, o2):
        check_rows(a, ref, size, ~hit, dtype)
        assert not torch.isfinite(a.cpu()[hit]).any()
    for a in (S, in_place):
        assert not torch.isfinite(a[0, 1, :, c]).any()
        a[0, 1, :, c] = wS[0, 1, :, c]
        assert torch.equal(a, wS)
    # dv_t and dk_t know the tokens from t on, dq_t those up to t: the same for a row of q, do or k
    ref, size = (R.backward(z["q"], z["k"], z["v"], l, z["do"], z["S0"], z["dS"]) for z in (x, y))
    for name in ("k", "q", "do"):
        bad = {n: (z.clone() if n == name else z) for n, z in g.items()}
        bad[name][0, 1, t, c] = value
        got = fw.decay_backward(bad["q"], bad["k"], bad["v"], l.cuda(), bad["do"], bad["S0"], bad["dS"])
        fw.check()
        clean = {"k": (at < t, at >= 0, at != t), "q": (at >= 0, at > t, at > t),
                 "do": (at != t, at > t, at > t)}[name]
        for a, r, s, rows in zip(got[:3], ref[:3], size[:3], clean):
            where = torch.ones(B, H, T, d, dtype=torch.bool)
            where[0, 1] = rows.view(T, 1)
            check_rows(a, r, s, where, dtype)
        if name == "do":
            assert not torch.isfinite(got[0][0, 1, t]).any()
            assert not torch.isfinite(got[2][0, 1, :t + 1, c]).any()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,t", [(128, 0), (128, 127), (256, 128), (70, 69), (1500, 700)])
def test_whole_rows_that_are_not_finite(T, t, d, dtype):
    """A row of v that is all NaN, with and without an output norm, at the borders of a chunk and in a chain
    that is split over the GPU; a padded batch whose other rows are as they would be."""
    x, g = inputs(2, 3, T, d, dtype, seed=T + t)
    l = torch.tensor([-0.01, -0.3, 0.0])
    ln = torch.tensor([T, max(T - 30, 1)], dtype=torch.int32)
    gen = torch.Generator().manual_seed(5)
    w, b = torch.randn(d, generator=gen), torch.randn(d, generator=gen)
    v = g["v"].clone()
    v[0, :, t] = float("nan")
    v[0, 1, T - 1, 3] = float("inf")
    ro = R.forward(x["q"], x["k"], x["v"], l, x["S0"], 1.0, ln)[0]
    for norm in (None, (w.cuda(), b.cuda())):
        o, S = fw.decay_prefill(g["q"], g["k"], v, l.cuda(), g["S0"], norm=norm, lens=ln.cuda())
        fw.check()
        r = ro if norm is None else R.layer_norm(ro, w, b)[0]
        if t > 0:
            assert R.rel_rows(o[:1, :, :t], r[:1, :, :t], 2) <= TOL[dtype]
        assert R.rel_rows(o[1:, :, :ln[1]], r[1:, :, :ln[1]], 2) <= TOL[dtype]
        assert (o[1, :, ln[1]:] == 0).all() and torch.isfinite(S[1]).all()
        assert not torch.isfinite(o[0, :, t:]).any() and not torch.isfinite(S[0]).any()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128])
def test_padded_batch_of_more_chains_than_fit_at_once(d, dtype):
    """13 x 13 chains of different lengths, the longest first, NaN behind every end and one value inside some
    chains: rows before it (after it, for dk and dv) are those of the call without it, up to the two calls'
    roundings (twice the tolerance, relative L2 of a chain's rows), and so is every other chain."""
    B, H, T, t = 13, 13, 420, 60
    x, g = inputs(B, H, T, d, dtype, seed=d)
    ln = torch.tensor([0, 420, 1, 300, 300, 128, 127, 5, 420, 64, 256, 17, 399], dtype=torch.int32)
    n = ln.view(B, 1, 1, 1)
    behind = torch.arange(T).view(1, 1, T, 1) >= n
    nan = torch.full((), float("nan"), dtype=dtype)
    clean = {k: torch.where(behind, nan, x[k]).cuda() for k in ("q", "k", "v", "do")}
    l = (-torch.rand(H, generator=torch.Generator().manual_seed(1)) * 0.2).cuda()
    hit = [(1, 0), (1, 12), (3, 5), (8, 7), (9, 2), (12, 12)]

    def run(bad_name=None):
        z = {k: (v.clone() if k == bad_name else v) for k, v in clean.items()}
        if bad_name:
            for b, h in hit:
                z[bad_name][b, h, t, 7] = float("inf") if h == 12 else float("nan")
        o, S = fw.decay_prefill(z["q"], z["k"], z["v"], l, g["S0"], lens=ln.cuda(), norm=None)
        dq, dk, dv, dS0 = fw.decay_backward(z["q"], z["k"], z["v"], l, z["do"], g["S0"], g["dS"], lens=ln.cuda())
        fw.check()
        return o, dq, dk, dv, S, dS0

    want = run()
    assert all(torch.isfinite(a).all() for a in want)
    # rows of a hit chain that do not depend on token t: before it (-1), after it (1), all (0)
    # (o, dq, dk, dv), or that may be anything (None)
    side = {"v": (-1, -1, None, 0), "k": (-1, -1, 0, None), "do": (0, None, 1, 1), "q": (None, 0, 1, 1)}
    for name, sides in side.items():
        got = run(name)
        for a, r, s in zip(got[:4], want[:4], sides):
            for b in range(B):
                for h in range(H):
                    rows = slice(None)
                    if (b, h) in hit:
                        if s is None:
                            continue
                        rows = slice(0, t) if s < 0 else slice(t + 1, None) if s > 0 else rows
                    num, den = (a[b, h, rows] - r[b, h, rows]).double().norm(), r[b, h, rows].double().norm()
                    assert torch.isfinite(a[b, h, rows]).all() and num <= 2 * TOL[dtype] * den
        for a, r in zip(got[4:], want[4:]):
            ok = torch.ones(B, H, dtype=torch.bool)
            ok[tuple(zip(*hit))] = False
            assert torch.equal(a[ok.cuda()], r[ok.cuda()])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("t", [3, 1700, 3999])
def test_backward_of_few_long_chains(t, d):
    """Chains whose reverse scans are split over the GPU too: rows that do not depend on token t are those of the
    call without it, up to the two calls' roundings."""
    B, H, T = 1, 2, 4000
    _, g = inputs(B, H, T, d, BF16, seed=t)
    l = torch.tensor([-0.002, -0.1]).cuda()
    n = fw.decay_workspace(B, H, T, d, BF16, backward=True)
    assert n > fw.decay_workspace(B, H, T, d, BF16) > 0     # segments in both directions

    def run(name=None):
        z = {k: (v.clone() if k == name else v) for k, v in g.items()}
        if name:
            z[name][0, 1, t, 9] = float("nan")
        got = fw.decay_backward(z["q"], z["k"], z["v"], l, z["do"], z["S0"], z["dS"])
        fw.check()
        return got

    want = run()
    for name, sides in {"v": (-1, None, 0), "k": (-1, 0, None), "do": (None, 1, 1), "q": (0, 1, 1)}.items():
        got = run(name)
        for a, r, s in zip(got[:3], want[:3], sides):
            assert torch.equal(a[0, 0], r[0, 0])
            rows = slice(0, t) if s == -1 else slice(t + 1, None) if s == 1 else slice(None)
            if s is None:
                rows = torch.arange(T, device="cuda") != t
            x, y = a[0, 1, rows].double(), r[0, 1, rows].double()
            assert torch.isfinite(x).all() and (x - y).norm() <= 2 * TOL[BF16] * y.norm()
        assert torch.equal(got[3][0, 0], want[3][0, 0])
