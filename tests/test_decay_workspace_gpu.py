"""Decayed calls in a workspace of exactly the size that is asked for, between guards, and chains of one chunk
whose state is updated in place without any.  Tolerances as for the other decayed tests (relative L2 of a chain:
fp32 rows and states 1e-5, bf16 rows 8e-3)."""
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
    x.update(S0=torch.randn(B, H, d, d, generator=g), dS=torch.randn(B, H, d, d, generator=g),
             ld=-torch.rand(H, generator=g) * 0.1)
    return x, {n: t.cuda() for n, t in x.items()}


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,H,T,d", [(1, 2, 700, 64), (2, 3, 130, 128), (1, 1, 1300, 128), (1, 5, 40, 64)])
def test_exactly_the_size_that_is_asked_for(B, H, T, d, dtype):
    x, g = inputs(B, H, T, d, dtype, seed=T)
    guard = 4096
    for backward in (False, True):
        n = fw.decay_workspace(B, H, T, d, dtype, backward=backward)
        room = torch.full((n + 2 * guard,), 0x5a, dtype=torch.uint8, device="cuda")
        ws = room[guard:guard + n] if n else None
        if backward:
            got = fw.decay_backward(g["q"], g["k"], g["v"], g["ld"], g["do"], g["S0"], g["dS"], workspace=ws)
            ref = R.backward(x["q"], x["k"], x["v"], x["ld"], x["do"], x["S0"], x["dS"])
            rows, state = got[:3], got[3]
        else:
            o, state = fw.decay_prefill(g["q"], g["k"], g["v"], g["ld"], g["S0"], workspace=ws)
            ref = R.forward(x["q"], x["k"], x["v"], x["ld"], x["S0"])[:2]
            rows = (o,)
        fw.check()
        for a, r in zip(rows, ref):
            assert R.rel_rows(a, r, 2) <= TOL[dtype]
        assert R.rel_rows(state, ref[-1], 2) <= 1e-5
        assert (room[:guard] == 0x5a).all() and (room[guard + n:] == 0x5a).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,lens", [(1, None), (64, None), (33, (0, 33)), (64, (7, 64))])
def test_one_chunk_in_place(T, lens, d, dtype):
    B, H = 2, 3
    x, g = inputs(B, H, T, d, dtype, seed=d + T)
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    S = g["S0"].clone()
    o, _ = fw.decay_prefill(g["q"], g["k"], g["v"], g["ld"], S, lens=None if ln is None else ln.cuda(), S_T=S)
    ro, rS, _ = R.forward(x["q"], x["k"], x["v"], x["ld"], x["S0"], 1.0, ln)
    assert R.rel_rows(o, ro, 2) <= TOL[dtype] and R.rel_rows(S, rS, 2) <= 1e-5
