"""Captured decayed calls replayed with other inputs, lengths among them; a decode step replayed token by token.
Replays give the bits of the plain calls."""
import pytest
import torch

from linear_token_mixer_gb300 import fw

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def inputs(B, H, T, d, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    z = {n: torch.randn(B, H, T, d, generator=gen).to(dtype).cuda() for n in ("q", "k", "v", "do")}
    z.update(S0=torch.randn(B, H, d, d, generator=gen).cuda(), dS=torch.randn(B, H, d, d, generator=gen).cuda(),
             ld=(-torch.rand(H, generator=gen)).cuda(), w=torch.randn(d, generator=gen).cuda(),
             lens=torch.randint(0, T + 1, (B,), generator=gen, dtype=torch.int32).cuda())
    return z


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,H,T,d", [(3, 4, 300, 64), (1, 2, 2100, 128), (14, 12, 150, 64), (2, 3, 50, 128)])
def test_replayed_with_other_lengths(B, H, T, d, dtype):
    def run(z):
        return [*fw.decay_prefill(z["q"], z["k"], z["v"], z["ld"], z["S0"], lens=z["lens"], norm=(z["w"], None)),
                *fw.decay_backward(z["q"], z["k"], z["v"], z["ld"], z["do"], z["S0"], z["dS"], lens=z["lens"])]
    z = inputs(B, H, T, d, dtype, 1)
    run(z)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run(z)
    for seed in (2, 3):
        y = inputs(B, H, T, d, dtype, seed)
        want = [t.clone() for t in run(y)]
        for n in z:
            z[n].copy_(y[n])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    fw.check()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_decode_loop(dtype):
    B, H, d, n = 3, 5, 128, 6
    z = inputs(B, H, n, d, dtype, 4)
    tok = [z[x][:, :, 0].contiguous() for x in "qkv"]
    S, S2 = z["S0"].clone(), z["S0"].clone()
    fw.decay_step(*tok, z["ld"], S.clone(), norm=(z["w"], None))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = fw.decay_step(*tok, z["ld"], S, norm=(z["w"], None))
    for t in range(n):
        now = [z[x][:, :, t].contiguous() for x in "qkv"]
        for a, b in zip(tok, now):
            a.copy_(b)
        graph.replay()
        want = fw.decay_step(*now, z["ld"], S2, norm=(z["w"], None))
        assert torch.equal(o, want) and torch.equal(S, S2)
