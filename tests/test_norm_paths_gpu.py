"""The output norm of the paths that update a state: a call that cannot be made is refused before the
state moves."""
import pytest
import torch

from linear_token_mixer_gb300 import fw
from linear_token_mixer_gb300 import inputs as I

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def calls(x, S, **kw):
    args = (x["q"], x["k"], x["v"], x["beta"], x["lam"])
    one = [t[:, :, 0].contiguous() for t in args]
    yield lambda **k: fw.prefill(*args, S, S_T=S, **kw, **k)
    yield lambda **k: fw.prefill(*args, S, S_T=S, noalloc=True, **kw, **k)
    yield lambda **k: fw.step(*one, S, **kw, **k)
    yield lambda **k: fw.window_prefill(*args, 3, S, S_T=S, **kw, **k)
    yield lambda **k: fw.window_step(*one, S, 3, **kw, **k)


def flat(n, skip=0, dtype=torch.float32):
    return torch.ones(n + skip, device="cuda", dtype=dtype)[skip:]


@pytest.mark.parametrize("bad", ["misaligned weight", "misaligned bias", "eps above fp32", "eps not finite",
                                 "weight too short", "weight of bf16", "o of another type",
                                 "o too short", "weight is o"])
def test_a_norm_that_is_refused_leaves_the_state_alone(bad):
    w = I.WORKLOADS["falcon1_bf16"].with_shape(B=1, H=2, T=70, dtype=BF16)
    x = {k: (t.cuda() if t is not None else None) for k, t in I.prefill_inputs(w).items()}
    d = x["q"].shape[-1]
    start = torch.randn(1, 2, d, d, device="cuda")
    S = start.clone()
    for i, call in enumerate(calls(x, S)):
        shape = x["q"].shape if i in (0, 1, 3) else x["q"][:, :, 0].shape
        o = torch.empty(shape, device="cuda", dtype=BF16)
        kw = {"misaligned weight": dict(norm=(flat(d, 1), None)),
              "misaligned bias": dict(norm=(flat(d), flat(d, 1))),
              "eps above fp32": dict(norm=(flat(d), None), norm_eps=1e39),
              "eps not finite": dict(norm=(None, None), norm_eps=float("nan")),
              "weight too short": dict(norm=(flat(d - 4), None)),
              "weight of bf16": dict(norm=(flat(d, dtype=BF16), None)),
              "o of another type": dict(norm=(None, None), o=o.float()),
              "o too short": dict(norm=(None, None), o=o[:, :1].contiguous()),
              "weight is o": dict(norm=(o.view(torch.float32).flatten()[:d], None), o=o)}[bad]
        with pytest.raises((ValueError, fw.FwError)):
            call(**kw)
        assert torch.equal(S, start)
