"""Decayed linear attention and layer norm without a GPU: the 64-bit references against
differences, the chunk form of the scans against the token form, and the C ABI's refusals."""
import ctypes

import pytest
import torch

from linear_token_mixer_gb300 import build as B_
from linear_token_mixer_gb300 import fw

import decay_ref as R


@pytest.fixture(scope="module")
def L():
    B_.build()
    return fw.lib()


def _inputs(B=2, H=2, T=7, d=4, seed=0):
    g = torch.Generator().manual_seed(seed)
    def rn(*s):
        return torch.randn(*s, generator=g, dtype=torch.float64)
    return (rn(B, H, T, d), rn(B, H, T, d), rn(B, H, T, d),
            -torch.rand(H, generator=g, dtype=torch.float64), rn(B, H, d, d), rn(B, H, T, d),
            rn(B, H, d, d))


@pytest.mark.parametrize("lens", [None, (7, 3), (0, 5)])
def test_reference_gradients_against_differences(lens):
    q, k, v, ld, S0, do, dS = _inputs()
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    grads = R.backward(q, k, v, ld, do, S0, dS, scale=0.7, lens=ln)
    g = torch.Generator().manual_seed(5)

    def loss(q, k, v, S0):
        o, S, _ = R.forward(q, k, v, ld, S0, 0.7, ln)
        return float((o * do).sum() + (S * dS).sum())

    args = [q, k, v, S0]
    for i, grad in enumerate(grads):
        for _ in range(3):
            u = torch.randn(args[i].shape, generator=g, dtype=torch.float64)
            h = 1e-5
            hi = [a + h * u if j == i else a for j, a in enumerate(args)]
            lo = [a - h * u if j == i else a for j, a in enumerate(args)]
            num = (loss(*hi) - loss(*lo)) / (2 * h)
            assert abs(num - float((grad * u).sum())) <= 1e-7 * max(1.0, abs(num))


def test_reference_norm_gradients_against_differences():
    g = torch.Generator().manual_seed(3)
    x, dy = (torch.randn(5, 9, generator=g, dtype=torch.float64) for _ in range(2))
    w, b = (torch.randn(9, generator=g, dtype=torch.float64) for _ in range(2))
    grads = R.layer_norm_backward(dy, x, w)

    def loss(x, w, b):
        return float((R.layer_norm(x, w, b)[0] * dy).sum())

    args = [x, w, b]
    for i, grad in enumerate(grads):
        u = torch.randn(args[i].shape, generator=g, dtype=torch.float64)
        h = 1e-6
        hi = [a + h * u if j == i else a for j, a in enumerate(args)]
        lo = [a - h * u if j == i else a for j, a in enumerate(args)]
        num = (loss(*hi) - loss(*lo)) / (2 * h)
        assert abs(num - float((grad * u).sum())) <= 1e-7 * max(1.0, abs(num))


def _scan(a, b, c, ld, X, C, rev, in_scale=1.0, out_scale=1.0):
    """The scans' chunk form (one chain set, no lens), as the kernels compute it."""
    T = a.shape[2]
    out = torch.zeros_like(a)
    g = lambda n: torch.exp(ld.view(1, -1, 1) * n)  # noqa: E731
    starts = list(range(0, T, C))
    for c0 in reversed(starts) if rev else starts:
        n = min(C, T - c0)
        i = torch.arange(n, dtype=torch.float64)
        A, Bt, Ct = (t[:, :, c0:c0 + n] for t in (a, b, c))
        lag = (i.view(-1, 1) - i.view(1, -1)) * (-1 if rev else 1)
        P = torch.where(lag >= 0, torch.einsum("bhid,bhjd->bhij", A, Bt)
                        * torch.exp(ld.view(1, -1, 1, 1) * lag.clamp(min=0)), torch.zeros(()).double())
        rd = g(n - 1 - i if rev else i + 1)
        wr = g(i + 1 if rev else n - 1 - i) * in_scale
        out[:, :, c0:c0 + n] = out_scale * (in_scale * P @ Ct + rd[..., None] * (A @ X))
        X = g(torch.tensor(float(n)))[..., None] * X + (Bt * wr[..., None]).transpose(-1, -2) @ Ct
    return out, X


@pytest.mark.parametrize("T,C", [(1, 4), (7, 4), (8, 4), (13, 64), (9, 3)])
def test_scan_form_is_the_recurrence_and_its_gradient(T, C):
    q, k, v, ld, S0, do, dS = _inputs(T=T, seed=T)
    s = 0.3
    o, S, _ = R.forward(q, k, v, ld, S0, s)
    tr = lambda x: x.transpose(-1, -2)  # noqa: E731
    o2, S2 = _scan(q, k, v, ld, S0, C, False, out_scale=s)
    dq, dk, dv, dS0 = R.backward(q, k, v, ld, do, S0, dS, s)
    dq2, _ = _scan(do, v, k, ld, tr(S0), C, False, out_scale=s)
    dv2, dS02 = _scan(k, q, do, ld, dS, C, True, in_scale=s)
    dk2, dk_end = _scan(v, do, q, ld, tr(dS), C, True, in_scale=s)
    for x, y in ((o, o2), (S, S2), (dq, dq2), (dv, dv2), (dk, dk2), (dS0, dS02), (dS0, tr(dk_end))):
        assert torch.allclose(x, y, rtol=1e-12, atol=1e-12)


# ---- refusals (fake addresses, never dereferenced) -----------------------------

no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                            reason="fake-pointer validation checks run only without a GPU")
P = [0x10000000 + 0x1000000 * i for i in range(24)]
WS = 1 << 40


def _shape(s):
    return ctypes.byref(fw.fw_shape(*s)) if s is not None else None


def _prefill(L, q=P[0], k=P[1], v=P[2], ld=P[3], S0=None, lens=None, norm=None, o=P[4], S_T=P[5],
             shape=(1, 2, 8, 64, 64), dtype=1, scale=1.0, flags=0, ws=P[6], nws=WS):
    n = None if norm is None else ctypes.byref(fw.fw_norm(*norm))
    return L.fw_decay_prefill(q, k, v, ld, S0, lens, n, o, S_T, _shape(shape), dtype, scale,
                              flags, ws, nws, None)


COMMON = [
    (dict(shape=None), -1), (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1),
    (dict(ld=None), -1), (dict(o=None), -1),
    (dict(shape=(0, 2, 8, 64, 64)), -2), (dict(shape=(1, 0, 8, 64, 64)), -2),
    (dict(shape=(1, 2, 0, 64, 64)), -2), (dict(shape=(1, 2, 8, 96, 96)), -2),
    (dict(shape=(1, 2, 8, 64, 128)), -2), (dict(shape=(1, 2, 2**31 - 100, 64, 64)), -2),
    (dict(shape=(2**20, 2**10, 2**17, 64, 64)), -2),
    (dict(dtype=5), -3), (dict(scale=float("nan")), -9), (dict(scale=float("inf")), -9),
    (dict(q=P[0] + 8), -4), (dict(ld=P[3] + 4), -4), (dict(o=P[4] + 2), -4),
    (dict(flags=1), -5), (dict(flags=8), -5),
]


@no_gpu
@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(S_T=None), -1), (dict(lens=P[7] + 4), -4), (dict(S0=P[8] + 4), -4),
    (dict(ws=P[6] + 4), -4), (dict(o=P[0]), -9), (dict(S_T=P[1]), -9), (dict(S_T=P[4]), -9),
    (dict(S0=P[5] + 16), -9), (dict(o=P[3]), -9), (dict(S0=P[4]), -9), (dict(lens=P[5]), -9),
    (dict(norm=(P[9] + 4, None, 1e-5)), -4), (dict(norm=(P[9], P[10], -1.0)), -9),
    (dict(norm=(P[9], None, float("nan"))), -9), (dict(norm=(P[4], None, 1e-5)), -9),
    (dict(norm=(None, P[5], 1e-5)), -9)])
def test_prefill_refusals(L, kw, code):
    assert _prefill(L, **kw) == code


def _backward(L, q=P[0], k=P[1], v=P[2], ld=P[3], S0=None, lens=None, do=P[4], dS_T=None, dq=P[5],
              dk=P[6], dv=P[7], dS0=None, shape=(1, 2, 8, 64, 64), dtype=1, scale=1.0, flags=0,
              ws=P[8], nws=WS):
    return L.fw_decay_backward(q, k, v, ld, S0, lens, do, dS_T, dq, dk, dv, dS0, _shape(shape),
                               dtype, scale, flags, ws, nws, None)


@no_gpu
@pytest.mark.parametrize("kw,code", [(({**kw, "do": kw["o"]} if "o" in kw else dict(kw)), c)
                                     for kw, c in COMMON] + [
    (dict(dq=None), -1), (dict(dk=None), -1), (dict(dv=None), -1), (dict(dq=P[0]), -9),
    (dict(dk=P[5]), -9), (dict(dv=P[4]), -9), (dict(dS0=P[9], dS_T=P[9]), -9),
    (dict(dS0=P[9], S0=P[9]), -9), (dict(dS0=P[5]), -9), (dict(dS_T=P[9] + 8), -4)])
def test_backward_refusals(L, kw, code):
    kw = dict(kw)
    kw.pop("o", None)
    assert _backward(L, **kw) == code


def _step(L, q=P[0], k=P[1], v=P[2], ld=P[3], S=P[4], norm=None, o=P[5], shape=(1, 2, 1, 64, 64),
          dtype=1, scale=1.0):
    n = None if norm is None else ctypes.byref(fw.fw_norm(*norm))
    return L.fw_decay_step(q, k, v, ld, S, n, o, _shape(shape), dtype, scale, None)


@no_gpu
@pytest.mark.parametrize("kw,code", [
    (dict(shape=None), -1), (dict(q=None), -1), (dict(S=None), -1), (dict(o=None), -1),
    (dict(ld=None), -1), (dict(shape=(1, 2, 2, 64, 64)), -2), (dict(shape=(1, 2, 1, 32, 32)), -2),
    (dict(dtype=2), -3), (dict(S=P[4] + 4), -4), (dict(o=P[0]), -9), (dict(S=P[1]), -9),
    (dict(o=P[4]), -9), (dict(scale=float("inf")), -9), (dict(norm=(P[6], None, -2.0)), -9),
    (dict(norm=(P[5], None, 0.0)), -9), (dict(norm=(None, P[6] + 2, 0.0)), -4)])
def test_step_refusals(L, kw, code):
    assert _step(L, **kw) == code


def _norm(L, x=P[0], w=P[1], b=P[2], y=P[3], mean=P[4], rstd=P[5], rows=4, width=64, dtype=1,
          eps=1e-5):
    return L.fw_layer_norm(x, w, b, y, mean, rstd, rows, width, dtype, eps, None)


@no_gpu
@pytest.mark.parametrize("kw,code", [
    (dict(x=None), -1), (dict(y=None), -1), (dict(rows=0), -2), (dict(width=0), -2),
    (dict(rows=-3), -2), (dict(rows=2**31), -2), (dict(width=2**24 + 1), -2), (dict(dtype=2), -3),
    (dict(x=P[0] + 2), -4), (dict(w=P[1] + 4), -4), (dict(mean=P[4] + 4), -4), (dict(eps=-1.0), -9),
    (dict(eps=float("nan")), -9), (dict(y=P[0] + 16), -9), (dict(y=P[1]), -9), (dict(mean=P[0]), -9),
    (dict(rstd=P[4]), -9), (dict(mean=P[3]), -9)])
def test_layer_norm_refusals(L, kw, code):
    assert _norm(L, **kw) == code


def _norm_bwd(L, dy=P[0], x=P[1], w=P[2], mean=P[3], rstd=P[4], dx=P[5], dw=P[6], db=P[7], rows=4,
              width=64, dtype=1, ws=P[8], nws=WS):
    return L.fw_layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db, rows, width, dtype, ws, nws,
                                    None)


@no_gpu
@pytest.mark.parametrize("kw,code", [
    (dict(dy=None), -1), (dict(x=None), -1), (dict(mean=None), -1), (dict(rstd=None), -1),
    (dict(dx=None), -1), (dict(ws=None), -1), (dict(rows=0), -2), (dict(dtype=9), -3),
    (dict(dx=P[5] + 8), -4), (dict(dw=P[6] + 4), -4), (dict(nws=16), -11), (dict(dx=P[0] + 16), -9),
    (dict(dw=P[0]), -9), (dict(db=P[6]), -9), (dict(ws=P[5]), -9), (dict(dx=P[2]), -9),
    (dict(dw=P[3]), -9)])
def test_layer_norm_backward_refusals(L, kw, code):
    assert _norm_bwd(L, **kw) == code


def test_workspace_queries(L):
    assert fw.decay_workspace(1, 2, 1, 64, torch.float32) >= 0
    assert fw.decay_workspace(2, 3, 500, 128, torch.float32, backward=True) >= \
        fw.decay_workspace(2, 3, 500, 128, torch.float32)
    with pytest.raises(fw.FwError):
        fw.decay_workspace(1, 1, 8, 96)
    assert L.fw_layer_norm_workspace(0, 4) == -2
    assert L.fw_layer_norm_workspace(5, 4) > 0


@no_gpu
def test_a_small_workspace_is_refused(L):
    n = fw.decay_workspace(1, 2, 300, 64, torch.float32)
    assert n > 0
    kw = dict(shape=(1, 2, 300, 64, 64), dtype=0)
    assert _prefill(L, nws=n - 1, **kw) == -11
    assert _prefill(L, ws=None, nws=0, **kw) == -1
    assert _backward(L, nws=fw.decay_workspace(1, 2, 300, 64, torch.float32, backward=True) - 1,
                     **kw) == -11


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(1, 2, 3, 64)
    ld = torch.zeros(2)
    with pytest.raises(ValueError, match="CUDA"):
        fw.decay_prefill(x, x, x, ld)
    with pytest.raises(ValueError, match="CUDA"):
        fw.layer_norm(x)


@pytest.mark.parametrize("bad", ["k", "ld", "S0", "lens", "do"])
def test_binding_checks_shapes_and_types_first(bad):
    x = torch.zeros(1, 2, 3, 64)
    kw = dict(q=x, k=x, v=x, log_decay=torch.zeros(2), S0=None, lens=None, do=x)
    kw.update({"k": dict(k=x.bfloat16()), "ld": dict(log_decay=torch.zeros(3)),
               "S0": dict(S0=torch.zeros(1, 2, 64, 32)), "lens": dict(lens=torch.zeros(1).long()),
               "do": dict(do=x[:, :1])}[bad])
    with pytest.raises(ValueError, match="must be"):
        fw.decay_backward(**kw)
