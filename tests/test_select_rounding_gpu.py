"""What the bf16 selective scan rounds, and where: a row's own value `skip v` beside the scan.

Tolerances: bf16 rows are rounded once, by half of the type's step at most, 2^-8 relative.  fp32 rows: 2^-24.
"""
import pytest
import torch

from linear_token_mixer_gb300 import fw

import mixer_ref as R

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
# mild chunks, steep ones, and blocks of 32 tokens whose decays multiply to less than e^-40
RATES = [(0.05, 0.2), (4.0, 16.0), (60.0, 200.0)]


def inputs(B, H, G, T, d, dtype, rate, seed=0):
    gen = torch.Generator().manual_seed(seed)

    def rn(*s):
        return torch.randn(*s, generator=gen)

    x = {"q": rn(B, G, T, d).to(dtype), "k": rn(B, G, T, d).to(dtype), "v": rn(B, H, T, d).to(dtype),
         "dt": 0.05 + 0.1 * torch.rand(B, H, T, generator=gen),
         "ld": -(rate[0] + (rate[1] - rate[0]) * torch.rand(H, generator=gen)), "S0": rn(B, H, d, d), "skip": 1 + 0.3 * rn(H)}
    return x, {n: t.cuda() for n, t in x.items()}


def run(z, **kw):
    o, S = fw.select_prefill(z["q"], z["k"], z["v"], z["dt"], z["ld"], z["S0"], skip=z["skip"], **kw)
    fw.check()
    return o.cpu(), S


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rate", RATES)
@pytest.mark.parametrize("B,H,G,T,lens", [(2, 3, 1, 300, None), (2, 2, 2, 300, (171, 0)), (1, 1, 1, 2100, None)])
def test_a_row_of_its_own_value_alone_is_rounded_once(B, H, G, T, lens, rate, d, dtype):
    """With queries of zero a row is skip v: one product in fp32, one rounding to the rows' type."""
    x, g = inputs(B, H, G, T, d, dtype, rate, seed=T)
    g["q"].zero_()
    o, _ = run(g, scale=0.25, lens=None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda())
    want = (x["skip"].view(1, H, 1, 1) * x["v"].float()).to(dtype)
    for b, n in enumerate(R.ends(None if lens is None else torch.tensor(lens), B, T)):
        want[b, :, n:] = 0
    assert torch.equal(o, want)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rate", RATES)
@pytest.mark.parametrize("scale", [1e-6, -1e-12, 1e-30, 0.0])
def test_skip_beside_a_scale_of_any_size(scale, rate, d, dtype):
    """skip v does not pass through the scan's factors: neither skip / scale nor its product with a decay can overflow.
    The scan's own share of a row is below 1e-6 times 2^12 (sums of 300 terms of dt q.k v and a state of one) here: rounded to
    2^-7 of itself, it is off by 1e-4 of 1e-2 at most, and by 2^-20 of it in fp32 rows."""
    B, H, G, T = 1, 3, 1, 300
    x, g = inputs(B, H, G, T, d, dtype, rate, seed=5)
    o, S = run(g, scale=scale)
    want, rS = R.select(x["q"], x["k"], x["v"], x["dt"], x["ld"], x["S0"], skip=x["skip"], scale=scale)
    part = (want - R.f64(x["skip"]).view(1, H, 1, 1) * R.f64(x["v"])).abs().max()
    half, inner = (2.0 ** -24, 2.0 ** -18) if dtype == F32 else (2.0 ** -8, 2.0 ** -7)
    assert torch.isfinite(o).all()
    assert ((o.double() - want).abs() <= (half + 2.0 ** -23) * want.abs() + inner * part + 2.0 ** -126).all()
    assert R.rel_rows(S, rS, 2) <= 1e-5


@pytest.mark.parametrize("first,written,tol", [(96, False, 3.3e-4), (96, True, 1.1e-3), (112, False, 4.6e-4)])
def test_decays_behind_tokens_that_keep_nothing(first, written, tol):
    """The first 96 or 112 tokens of a chunk keep nothing (their logs are 104 or more each); those behind them keep almost all of
    it, and their decays are as exact as in a chunk of their own, or, where 16 of their block of 32 keep nothing, off by a unit of
    a sum of 1664, 1.3e-4.  The factor by which all chains' rows of a token are off is the
    decays' common error and the mean of roundings of random sign: those of P (2^-8 at most, 1.6e-3 in the mean square of a value)
    and of the rows (64 x 64 of them, 2.5e-5).  Where the first tokens write nothing, a row is a sum of eight terms or more in 64
    chains, sum_j P_ij v_j: 1.6e-3 / sqrt(8 x 64) = 7e-5, with sums that vary from chain to chain 1.1e-4, and three times that
    3.3e-4.  Where they write, with steps of 400 beside 0.0003, a row is one term, the last such token's, in 64 chains, 2.1e-4,
    and the largest of 24 rows five times that."""
    B, H, T, d = 8, 8, 128, 64
    x, _ = inputs(B, H, H, T, d, BF16, (1.0, 1.0), seed=9)
    x["q"], x["k"] = x["q"].float().abs().bfloat16(), x["k"].float().abs().bfloat16()
    x["dt"][:] = 0.0003
    x["dt"][:, :, :first] = 400.0
    if not written:
        x["k"][:, :, :first] = 0.0
    x["skip"].zero_()
    o, _ = run({n: t.cuda() for n, t in x.items()}, scale=100.0)
    want, _ = R.select(x["q"], x["k"], x["v"], x["dt"], x["ld"], x["S0"], scale=100.0)
    o, want = (t.double()[:, :, first + 8:] for t in (o, want))
    assert ((o * want).sum((0, 1, 3)) / (want * want).sum((0, 1, 3)) - 1).abs().max().item() <= tol
