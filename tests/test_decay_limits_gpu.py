"""Decayed scans where their forms change: the largest decay whose powers a bf16 chunk divides by, and
the states of chains whose last tokens write nothing.

Tolerances.  Rows, element by element, relative to the same recurrence over absolute values (a row of
one token is a score times v, and no bound holds relative to a score that cancels).  fp32: a product of
split operands leaves out 2^-22 three times over, and the sums of a score (d), of a chunk (64) and of
the state's read (d) take 16 + 8 + 16 additions of at most 2^-23: 3 x 2^-22 twice and 40 x 2^-23 =
6.2e-6 with d = 128, 1e-5.  bf16: an operand of each product is rounded once (at most 2^-8) and the row
once: 2 x 2^-8 + 2^-16 = 7.83e-3, 8e-3.  States: an fp32 state's
operands are split into terms that hold 22 bits (fp32 rows) or 24 (bf16), at most 2^-22 = 2.4e-7 lost;
a chunk's sum takes up to 24 additions on the tensor cores, which cut towards zero, at most 2^-23 of the
running sum each: 24 x 2^-23 = 2.9e-6 together.  What carries a state on is an fp32 FMA a chunk.  3.2e-6.
"""
import pytest
import torch

from linear_token_mixer_gb300 import fw

import decay_ref as R

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TOL = {F32: 1e-5, BF16: 8e-3}
TOL_STATE = 3.2e-6


def inputs(B, H, T, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = {n: torch.randn(B, H, T, d, generator=g).to(dtype) for n in ("q", "k", "v", "do")}
    x.update(S0=torch.randn(B, H, d, d, generator=g), dS=torch.randn(B, H, d, d, generator=g))
    return x, {n: t.cuda() for n, t in x.items()}


def check_rows(got, ref, size, dtype):
    got = got.cpu().double()
    assert torch.isfinite(got).all()
    assert ((got - ref).abs() <= TOL[dtype] * size).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [(260, 135), (256, 1), (129, 0)])
@pytest.mark.parametrize("ld", [-0.186, -0.189, 0.186, 0.189, -3.0, -20.0])
def test_decays_around_the_dividing_bound(ld, lens, d, dtype):
    """128 |log g| = 24 is where the bf16 scans begin to divide by a chunk's decay: shrinking and growing
    heads on both sides of it, one of each bound's neighbours in one call, rows of the batch that end inside
    a chunk, with it, and before it."""
    B, H, T = 2, 2, 260
    x, g = inputs(B, H, T, d, dtype, seed=int(1000 * abs(ld)) + d)
    l = torch.tensor([ld, ld / 2])
    ln = torch.tensor(lens, dtype=torch.int32)
    o, S = fw.decay_prefill(g["q"], g["k"], g["v"], l.cuda(), g["S0"], scale=0.25, lens=ln.cuda())
    got = fw.decay_backward(g["q"], g["k"], g["v"], l.cuda(), g["do"], g["S0"], g["dS"], scale=0.25,
                            lens=ln.cuda())
    fw.check()
    ro, rS, _ = R.forward(x["q"], x["k"], x["v"], l, x["S0"], 0.25, ln)
    ref = R.backward(x["q"], x["k"], x["v"], l, x["do"], x["S0"], x["dS"], 0.25, ln)
    y = {n: t.abs() for n, t in x.items()}
    size = [R.forward(y["q"], y["k"], y["v"], l, y["S0"], 0.25, ln)[0],
            *R.backward(y["q"], y["k"], y["v"], l, y["do"], y["S0"], y["dS"], 0.25, ln)[:3]]
    for a, r, s in zip((o, *got[:3]), (ro, *ref[:3]), size):
        check_rows(a, r, s, dtype)
    assert R.rel_rows(S, rS, 2) <= TOL_STATE
    assert R.rel_rows(got[3], ref[3], 2) <= TOL_STATE


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,written", [(700, 140), (2600, 300)])
@pytest.mark.parametrize("quiet", [0.0, 2.0 ** -20])
def test_states_whose_last_tokens_write_little(quiet, T, written, d, dtype):
    """Tokens whose keys are zero (or all but zero) at the end: the returned state is what the first chunks
    wrote, however much it has decayed since, and is as exact as any other; in reverse, the gradient of the
    first state from the last tokens alone.  (T = 2600: chains in segments.)"""
    x, _ = inputs(1, 2, T, d, dtype, seed=T)
    ld = torch.tensor([-0.02, -0.004])
    x["k"][:, :, written:] *= quiet
    x["q"][:, :, :T - written] *= quiet
    g = {n: t.cuda() for n, t in x.items()}
    _, S = fw.decay_prefill(g["q"], g["k"], g["v"], ld.cuda())
    zero = torch.zeros_like(g["S0"])
    *_, dS0 = fw.decay_backward(g["q"], g["k"], g["v"], ld.cuda(), g["do"], dS0=zero)
    fw.check()
    _, rS, _ = R.forward(x["q"], x["k"], x["v"], ld)
    *_, rdS0 = R.backward(x["q"], x["k"], x["v"], ld, x["do"])
    assert R.rel_rows(S, rS, 2) <= TOL_STATE
    assert R.rel_rows(dS0, rdS0, 2) <= TOL_STATE
