"""Calls on a stream of their own whose inputs are temporaries: the memory of what a caller gives back is
not handed out again while the kernels still wait to read it."""
import pytest
import torch

from linear_token_mixer_gb300 import fw
from linear_token_mixer_gb300 import inputs as I

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def _calls():
    g = torch.Generator().manual_seed(1)
    rn = lambda *s, dtype=BF16: torch.randn(*s, generator=g).to(dtype).cuda()  # noqa: E731
    B, H, T, d = 2, 4, 300, 64
    rows, one = [rn(B, H, T, d) for _ in range(4)], [rn(B, H, d) for _ in range(3)]
    ld, S = -torch.rand(H, generator=g).cuda(), rn(B, H, d, d, dtype=torch.float32)
    nw, nb = rn(d, dtype=torch.float32), rn(d, dtype=torch.float32)
    x, dy, w, b = rn(900, 256), rn(900, 256), rn(256, dtype=torch.float32), rn(256, dtype=torch.float32)
    mean, rstd = rn(900, dtype=torch.float32), rn(900, dtype=torch.float32)
    f = I.WORKLOADS["falcon1_bf16"].with_shape(B=1, H=2, T=70, dtype=BF16)
    f = {k: t.cuda() for k, t in I.prefill_inputs(f).items() if t is not None}
    fx = [f[k] for k in ("q", "k", "v", "beta", "lam")]
    f1 = [t[:, :, 0].contiguous() for t in fx]
    fS = rn(1, 2, fx[0].shape[-1], fx[0].shape[-1], dtype=torch.float32)
    fn = [rn(fx[0].shape[-1], dtype=torch.float32) for _ in range(2)]
    yield "decay_prefill", [*rows[:3], ld, S, nw, nb], lambda q, k, v, l, s, w, b, **kw: fw.decay_prefill(
        q, k, v, l, s, norm=(w, b), **kw)
    yield "decay_backward", [*rows[:3], ld, rows[3], S], lambda *a, **kw: fw.decay_backward(*a, **kw)
    yield "decay_step", [*one, ld, S, nw, nb], lambda q, k, v, l, s, w, b, **kw: (
        fw.decay_step(q, k, v, l, s, norm=(w, b), **kw),)
    yield "layer_norm", [x, w, b], lambda *a, **kw: fw.layer_norm(*a, **kw)
    yield "layer_norm_backward", [dy, x, w, mean, rstd], lambda *a, **kw: fw.layer_norm_backward(*a, **kw)
    yield "prefill", [*fx, fS, *fn], lambda *a, **kw: fw.prefill(*a[:6], norm=a[6:], **kw)
    yield "step", [*f1, fS, *fn], lambda *a, **kw: (fw.step(*a[:6], norm=a[6:], **kw),)
    yield "window_prefill", [*fx, fS, *fn], lambda *a, **kw: fw.window_prefill(
        *a[:5], 3, a[5], norm=a[6:], **kw)[:2]
    yield "window_step", [*f1, fS, *fn], lambda *a, **kw: (fw.window_step(*a[:6], 3, norm=a[6:], **kw)[0],)


NAMES = ["decay_prefill", "decay_backward", "decay_step", "layer_norm", "layer_norm_backward", "prefill",
         "step", "window_prefill", "window_step"]


@pytest.mark.parametrize("name", NAMES)
def test_temporaries_of_a_call_on_another_stream(name):
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
