"""Shared and tensor memory hold what the kernel before left there.  Every call, at sizes that leave parts of its
tiles unloaded, gives the same bits behind kernels that left NaN everywhere as behind kernels that left zeros."""
import pytest
import torch

from linear_token_mixer_gb300 import fw
from linear_token_mixer_gb300 import inputs as I

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def leave(value):
    """A decayed prefill of 304 chains of rows of `value`: its tiles, states and products stay behind in the
    shared and tensor memory of every SM."""
    x = torch.full((19, 16, 256, 128), value, device="cuda", dtype=BF16)
    fw.decay_prefill(x, x, x, torch.zeros(16, device="cuda"))
    fw.layer_norm(torch.full((2000, 8192), value, device="cuda"))
    torch.cuda.synchronize()


def same(call):
    got = []
    for value in (float("nan"), 0.0):
        leave(value)
        got.append([t.clone() for t in call()])
    fw.check()
    for a, b in zip(*got):
        assert torch.isfinite(a).all() and torch.equal(a, b)


def inputs(mode, dtype, T, d=128, B=2, H=3):
    w = I.WORKLOADS["falcon2_bf16" if mode.startswith("falcon2") else "falcon1_bf16"].with_shape(
        B=B, H=H, T=T, dtype=dtype, mode=mode, d=d)
    x = {k: (t.cuda() if t is not None else None) for k, t in I.prefill_inputs(w, seed=T).items()}
    gen = torch.Generator().manual_seed(T)
    return x, torch.randn(B, H, d, d, generator=gen).cuda()


TS = [1, 2, 63, 65, 130, 257]


@pytest.mark.parametrize("T", TS)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("mode", ["falcon1", "falcon1a", "falcon2", "falcon2a", "linattn"])
@pytest.mark.parametrize("algo", ["auto", "recurrent"])
def test_prefill(algo, mode, dtype, T):
    x, S = inputs(mode, dtype, T)
    for kw in ({}, {"rbw": True, "same_pair": True}):
        same(lambda: fw.prefill(x["q"], x["k"], x["v"], x["beta"], x["lam"], S, mode=mode, algo=algo, **kw))


@pytest.mark.parametrize("T", [70, 700])
def test_prefill_in_two_segments(T):
    x, S = inputs("falcon1", BF16, T, B=1, H=2)
    L = fw.lib()
    L.fw_debug_segment_split(1)
    try:
        same(lambda: fw.prefill(x["q"], x["k"], x["v"], x["beta"], x["lam"], S))
    finally:
        L.fw_debug_segment_split(0)


@pytest.mark.parametrize("T", TS)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("mode", ["falcon3", "falcon3a"])
@pytest.mark.parametrize("window", [1, 3, 8])
def test_window_prefill(window, mode, dtype, T):
    x, S = inputs("falcon1", dtype, T)

    def call():
        o, S_T, win = fw.window_prefill(x["q"], x["k"], x["v"], x["beta"], x["lam"], window, S, mode=mode)
        return o, S_T, *win
    same(call)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128])
def test_steps(d, dtype):
    for mode in ("falcon1", "falcon1a", "falcon2", "falcon2a", "linattn", "falcon3", "falcon3a"):
        x, S = inputs(mode if mode.startswith("falcon2") else "falcon1", dtype, 1, d=d)
        one = [x[n][:, :, 0].contiguous() for n in ("q", "k", "v", "beta", "lam")]

        def call():
            s = S.clone()
            if mode.startswith("falcon3"):
                o, win = fw.window_step(*one, s, 3, mode=mode)
                return o, s, *win
            return fw.step(*one, s, mode=mode), s
        same(call)


@pytest.mark.parametrize("T", TS + [1300])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128])
def test_decayed(d, dtype, T):
    gen = torch.Generator().manual_seed(T)
    B, H = 2, 3
    q, k, v, do = (torch.randn(B, H, T, d, generator=gen).to(dtype).cuda() for _ in range(4))
    S0, dS = (torch.randn(B, H, d, d, generator=gen).cuda() for _ in range(2))
    ld = torch.tensor([-0.01, -0.1, -2.0]).cuda()
    w, b = torch.randn(d, generator=gen).cuda(), torch.randn(d, generator=gen).cuda()
    for lens in (None, torch.tensor([T, T // 2], dtype=torch.int32).cuda()):
        same(lambda: fw.decay_prefill(q, k, v, ld, S0, lens=lens, norm=(w, b)))
        same(lambda: fw.decay_prefill(q, k, v, ld, lens=lens))
        same(lambda: fw.decay_backward(q, k, v, ld, do, S0, dS, lens=lens))

    def step():
        s = S0.clone()
        return fw.decay_step(*(t[:, :, 0].contiguous() for t in (q, k, v)), ld, s, norm=(w, b)), s
    same(step)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,width", [(1, 1), (3, 7), (37, 100), (700, 77), (2000, 130), (2000, 520), (1500, 2056),
                                        (1100, 4104), (37, 8184), (1100, 16392), (3, 33000)])
def test_layer_norm(rows, width, dtype):
    gen = torch.Generator(device="cuda").manual_seed(width)
    x, dy = (torch.randn(rows, width, device="cuda", generator=gen).to(dtype) for _ in range(2))
    w, b = (torch.randn(width, device="cuda", generator=gen) for _ in range(2))

    def call():
        y, mean, rstd = fw.layer_norm(x, w, b)
        return y, mean, rstd, *fw.layer_norm_backward(dy, x, w, mean, rstd)
    same(call)
