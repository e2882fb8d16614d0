"""Selective scan, short convolution and gated norm without a GPU: the 64-bit references against the
calls they reduce to and against differences, and the refusals of the C ABI and of the binding."""
import ctypes

import pytest
import torch

from linear_token_mixer_gb300 import build as B_
from linear_token_mixer_gb300 import fw

import decay_ref
import mixer_ref as R


@pytest.fixture(scope="module")
def L():
    B_.build()
    return fw.lib()


no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses")


def rn(*s, seed=0):
    return torch.randn(*s, generator=torch.Generator().manual_seed(seed + sum(s)), dtype=torch.float64)


def test_select_reference_is_the_decayed_recurrence_for_steps_of_one():
    q, k, v = (rn(2, 3, 9, 4, seed=i) for i in range(3))
    ld, S0, lens = -rn(3).abs(), rn(2, 3, 4, 4), torch.tensor([9, 4])
    o, S = R.select(q, k, v, torch.ones(2, 3, 9), ld, S0, scale=0.3, lens=lens)
    ro, rS, _ = decay_ref.forward(q, k, v, ld, S0, 0.3, lens)
    assert (o - ro).abs().max() < 1e-12 and (S - rS).abs().max() < 1e-12


def test_select_reference_against_the_masked_quadratic_form():
    B, H, G, T, d = 2, 4, 2, 11, 3
    q, k, v = rn(B, G, T, d), rn(B, G, T, d, seed=1), rn(B, H, T, d, seed=2)
    raw, bias, ld, skip = rn(B, H, T), rn(H, seed=4), -rn(H).abs(), rn(H, seed=9)
    o, _ = R.select(q, k, v, raw, ld, None, bias, True, skip, 0.5)
    dt = torch.nn.functional.softplus(raw + bias.view(1, H, 1))
    c = torch.cumsum(dt * ld.view(1, H, 1), -1)
    P = torch.exp(c[..., :, None] - c[..., None, :]).tril() * dt[..., None, :]
    qk = torch.einsum("bgtd,bgsd->bgts", q, k).repeat_interleave(2, 1)
    assert (o - (0.5 * torch.einsum("bhts,bhsd->bhtd", P * qk, v) + skip.view(1, H, 1, 1) * v)).abs().max() < 1e-12


def test_conv_reference_against_conv1d_and_calls_in_turn():
    B, H, T, d, W = 2, 3, 12, 5, 4
    x, w, b = rn(B, H, T, d), rn(H, d, W), rn(H, d)
    y, s = R.conv(x, w, b, None, False)
    z = torch.nn.functional.conv1d(torch.nn.functional.pad(x.permute(0, 1, 3, 2).reshape(B, H * d, T), (W - 1, 0)),
                                   w.reshape(H * d, 1, W), b.reshape(-1), groups=H * d)
    assert (y - z.view(B, H, d, T).permute(0, 1, 3, 2)).abs().max() < 1e-12
    y1, s1 = R.conv(x[:, :, :5], w, b, None)
    y2, s2 = R.conv(x[:, :, 5:], w, b, s1)
    whole, end = R.conv(x, w, b, None)
    assert (torch.cat([y1, y2], 2) - whole).abs().max() < 1e-12 and torch.equal(s2, end) and torch.equal(s, end)


@pytest.mark.parametrize("lens", [None, (7, 2), (0, 5)])
@pytest.mark.parametrize("silu", [False, True])
def test_conv_reference_gradients_against_differences(silu, lens):
    B, H, T, d, W = 2, 2, 7, 3, 4
    args = [rn(B, H, T, d), rn(H, d, W), rn(H, d), rn(B, H, W - 1, d, seed=3)]
    dy, ds = rn(B, H, T, d, seed=5), rn(B, H, W - 1, d, seed=6)
    ln = None if lens is None else torch.tensor(lens)
    grads = R.conv_grads(dy, *args, ds, silu, ln)

    def loss(*a):
        y, s = R.conv(*a, silu, ln)
        return float((y * dy).sum() + (s * ds).sum())

    for i, g in enumerate(grads):
        u, h = rn(*args[i].shape, seed=11), 1e-5
        num = (loss(*[a + h * u if j == i else a for j, a in enumerate(args)])
               - loss(*[a - h * u if j == i else a for j, a in enumerate(args)])) / (2 * h)
        assert abs(num - float((g * u).sum())) <= 1e-7 * max(1.0, abs(num))


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("after", [False, True])
def test_gated_reference_against_layer_norm_and_differences(rms, after):
    H, T, w = 2, 3, 6
    given = dict(x=rn(H, T, w), gate=rn(H, T, w, seed=1), residual=rn(H, T, w, seed=2), weight=rn(H, w),
                 bias=rn(H, w, seed=1), scale=rn(H, w, seed=2))
    dy, dt = rn(H, T, w, seed=7), rn(H, T, w, seed=8)
    if not rms:
        y = R.gated(given["x"], given["weight"][0], given["bias"][0])[0]
        assert (y - decay_ref.layer_norm(given["x"], given["weight"][0], given["bias"][0])[0]).abs().max() < 1e-12
    grads = R.gated_grads(dy, dt, rms=rms, gate_after=after, **given)

    def loss(g):
        y, u, _, _ = R.gated(rms=rms, gate_after=after, **g)
        return float((y * dy).sum() + (u * dt).sum())

    for name, g in grads.items():
        v, h = rn(*g.shape, seed=13), 1e-5
        num = (loss({**given, name: given[name] + h * v}) - loss({**given, name: given[name] - h * v})) / (2 * h)
        assert abs(num - float((g * v).sum())) <= 1e-7 * max(1.0, abs(num))


# ---- refusals of the C ABI: before anything is launched, so that made-up addresses do -----------

P = [0x10000000 + 0x1000000 * i for i in range(20)]
WS = 1 << 40
SHAPE = (1, 4, 8, 64, 64)


def _shape(s):
    return None if s is None else ctypes.byref(fw.fw_shape(*s))


def _gates(dt=P[10], dt_type=1, ld=P[11], bias=None, skip=None, groups=2):
    return ctypes.byref(fw.fw_gates(dt, dt_type, ld, bias, skip, groups))


def _select(L, q=P[0], k=P[1], v=P[2], gates=True, S0=None, lens=None, o=P[4], S_T=P[5], shape=SHAPE, dtype=1,
            scale=1.0, flags=0, ws=P[6], nws=WS, **g):
    return L.fw_select_prefill(q, k, v, _gates(**g) if gates else None, S0, lens, o, S_T, _shape(shape), dtype,
                               scale, flags, ws, nws, None)


def _select_step(L, q=P[0], k=P[1], v=P[2], gates=True, S=P[5], o=P[4], shape=(1, 4, 1, 64, 64), dtype=1, scale=1.0,
                 flags=0, **g):
    return L.fw_select_step(q, k, v, _gates(**g) if gates else None, S, o, _shape(shape), dtype, scale, flags, None)


BOTH = [
    (dict(shape=None), -1), (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(o=None), -1),
    (dict(gates=False), -1), (dict(dt=None), -1), (dict(ld=None), -1), (dict(groups=0), -2), (dict(groups=3), -2),
    (dict(groups=8), -2), (dict(dtype=4), -3), (dict(dt_type=7), -3), (dict(dt_type=1, dtype=0), -3),
    (dict(scale=float("nan")), -9), (dict(q=P[0] + 8), -4), (dict(dt=P[10] + 4), -4), (dict(bias=P[12] + 4), -4),
    (dict(skip=P[13] + 8), -4), (dict(flags=1), -5), (dict(flags=8), -5), (dict(o=P[0]), -9), (dict(o=P[2]), -9),
    (dict(o=P[10]), -9), (dict(skip=P[4]), -9), (dict(bias=P[5]), -9), (dict(ld=P[5]), -9)]


@no_gpu
@pytest.mark.parametrize("kw,code", BOTH + [
    (dict(S_T=None), -1), (dict(ws=None), -1), (dict(nws=0), -11), (dict(shape=(0, 4, 8, 64, 64)), -2),
    (dict(shape=(1, 4, 0, 64, 64)), -2), (dict(shape=(1, 4, 8, 96, 96)), -2), (dict(shape=(1, 4, 8, 64, 128)), -2),
    (dict(shape=(1, 4, 2**31 - 64, 64, 64)), -2), (dict(S0=P[5] + 16), -9), (dict(S0=P[4]), -9), (dict(lens=P[5]), -9),
    (dict(S_T=P[4]), -9), (dict(S_T=P[1]), -9), (dict(ws=P[2]), -9), (dict(lens=P[7] + 4), -4)])
def test_select_refusals(L, kw, code):
    assert _select(L, **kw) == code


@no_gpu
@pytest.mark.parametrize("kw,code", BOTH + [
    (dict(S=None), -1), (dict(shape=(1, 4, 2, 64, 64)), -2), (dict(flags=4), -5), (dict(S=P[1]), -9),
    (dict(S=P[4]), -9)])
def test_select_step_refusals(L, kw, code):
    assert _select_step(L, **kw) == code


@no_gpu
def test_a_small_workspace_is_refused(L):
    assert fw.select_workspace(1, 4, 64, 64, torch.float32) == 0       # one chunk: none
    for T, dt in ((1, 1), (300, 1), (65, 0), (300, 0)):
        n = fw.select_workspace(1, 4, T, 64, torch.bfloat16 if dt else torch.float32)
        assert n > 0 and _select(L, shape=(1, 4, T, 64, 64), dtype=dt, dt_type=0, nws=n - 1) == -11
    n = L.fw_conv_workspace(_shape((2, 4, 8, 5, 5)), 3)
    assert n > 0 and _conv_bwd(L, nws=n - 1) == -11 and _conv_bwd(L, ws=None) == -1
    n = L.fw_gated_norm_workspace(12, 64, 2, 1)
    assert n > 0 and _gated_bwd(L, nws=n - 1) == -11 and _gated_bwd(L, ws=None) == -1
    assert L.fw_select_workspace(_shape((1, 1, 1, 32, 32)), 1) == -2 and L.fw_conv_workspace(_shape(SHAPE), 9) == -2
    assert L.fw_gated_norm_workspace(12, 64, 5, 1) == -2 and L.fw_gated_norm_workspace(12, 64, 2, 3) == -3


def _conv(L, x=P[0], w=P[1], b=P[2], state=P[3], lens=P[4], y=P[5], so=P[6], shape=(2, 4, 8, 5, 5), width=3, dtype=1,
          flags=8):
    return L.fw_conv_prefill(x, w, b, state, lens, y, so, _shape(shape), width, dtype, flags, None)


CONV = [(dict(shape=None), -1), (dict(x=None), -1), (dict(w=None), -1), (dict(shape=(0, 4, 8, 5, 5)), -2),
        (dict(shape=(2, 4, 8, 0, 0)), -2), (dict(shape=(2, 4, 8, 5, 6)), -2), (dict(width=1), -2), (dict(width=9), -2),
        (dict(shape=(2**20, 2**10, 2**17, 64, 64)), -2), (dict(shape=(1, 70000, 1, 4, 4)), -2), (dict(dtype=2), -3),
        (dict(x=P[0] + 2), -4), (dict(w=P[1] + 4), -4), (dict(state=P[3] + 8), -4), (dict(flags=1), -5),
        (dict(flags=16), -5)]


@no_gpu
@pytest.mark.parametrize("kw,code", CONV + [
    (dict(y=None), -1), (dict(y=P[0]), -9), (dict(y=P[3]), -9), (dict(y=P[1]), -9), (dict(so=P[5]), -9),
    (dict(so=P[0]), -9), (dict(so=P[3] + 16), -9), (dict(lens=P[4] + 4), -4), (dict(shape=(2, 4, 0, 5, 5)), -2)])
def test_conv_refusals(L, kw, code):
    assert _conv(L, **kw) == code


def _conv_bwd(L, dy=P[7], x=P[0], w=P[1], b=P[2], state=P[3], lens=P[4], dso=P[8], dx=P[5], dw=P[9], db=P[10],
              ds=P[11], shape=(2, 4, 8, 5, 5), width=3, dtype=1, flags=8, ws=P[12], nws=WS):
    return L.fw_conv_backward(dy, x, w, b, state, lens, dso, dx, dw, db, ds, _shape(shape), width, dtype, flags, ws,
                              nws, None)


@no_gpu
@pytest.mark.parametrize("kw,code", CONV + [
    (dict(dy=None), -1), (dict(dx=None), -1), (dict(dx=P[0]), -9), (dict(dx=P[7]), -9), (dict(dw=P[1]), -9),
    (dict(db=P[9]), -9), (dict(ds=P[3]), -9), (dict(ds=P[8]), -9), (dict(ws=P[5]), -9), (dict(dx=P[5] + 2), -4)])
def test_conv_backward_refusals(L, kw, code):
    assert _conv_bwd(L, **kw) == code


def _conv_step(L, x=P[0], w=P[1], b=P[2], state=P[3], y=P[5], shape=(2, 4, 1, 5, 5), width=3, dtype=1, flags=8):
    return L.fw_conv_step(x, w, b, state, y, _shape(shape), width, dtype, flags, None)


@no_gpu
@pytest.mark.parametrize("kw,code", CONV + [
    (dict(y=None), -1), (dict(state=None), -1), (dict(shape=(2, 4, 2, 5, 5)), -2), (dict(flags=4), -5),
    (dict(y=P[0]), -9), (dict(y=P[3]), -9), (dict(state=P[1]), -9), (dict(state=P[0]), -9)])
def test_conv_step_refusals(L, kw, code):
    assert _conv_step(L, **kw) == code


def _args(gate=P[1], res=P[2], scale=P[3], w=P[4], b=P[5], groups=2, inner=3, eps=1e-5, rms=0, after=0):
    return ctypes.byref(fw.fw_gated(gate, res, scale, w, b, groups, inner, eps, rms, after))


def _gated(L, x=P[0], args=True, y=P[6], total=P[7], mean=P[8], rstd=P[9], rows=12, width=64, dtype=1, **kw):
    return L.fw_gated_norm(x, _args(**kw) if args else None, y, total, mean, rstd, rows, width, dtype, None)


def _gated_bwd(L, dy=P[10], dt=P[11], x=P[0], args=True, mean=P[8], rstd=P[9], dx=P[12], dg=P[13], dr=P[14],
               dw=P[15], db=P[16], dsc=P[17], rows=12, width=64, dtype=1, ws=P[18], nws=WS, **kw):
    return L.fw_gated_norm_backward(dy, dt, x, _args(**kw) if args else None, mean, rstd, dx, dg, dr, dw, db, dsc,
                                    rows, width, dtype, ws, nws, None)


GATED = [(dict(x=None), -1), (dict(args=False), -1), (dict(rows=0), -2), (dict(rows=13), -2), (dict(width=0), -2),
         (dict(width=8193), -2), (dict(groups=0), -2), (dict(inner=0), -2), (dict(inner=4), -2), (dict(inner=7), -2),
         (dict(dtype=2), -3), (dict(x=P[0] + 2), -4), (dict(gate=P[1] + 8), -4), (dict(scale=P[3] + 4), -4),
         (dict(eps=-1.0), -9), (dict(eps=float("nan")), -9), (dict(rms=2), -5), (dict(after=-1), -5)]


@no_gpu
@pytest.mark.parametrize("kw,code", GATED + [
    (dict(y=None), -1), (dict(res=None), -9), (dict(y=P[0] + 16), -9), (dict(total=P[6]), -9), (dict(total=P[2] + 32), -9),
    (dict(y=P[4]), -9), (dict(mean=P[0]), -9), (dict(rstd=P[8]), -9), (dict(mean=P[3]), -9), (dict(y=P[6] + 4), -4)])
def test_gated_refusals(L, kw, code):
    assert _gated(L, **kw) == code


@no_gpu
@pytest.mark.parametrize("kw,code", GATED + [
    (dict(dy=None), -1), (dict(rstd=None), -1), (dict(mean=None), -1), (dict(gate=None), -9), (dict(res=None), -9),
    (dict(res=None, dr=None), -9), (dict(dx=P[10] + 16), -9), (dict(dg=P[12]), -9), (dict(dw=P[10]), -9),
    (dict(db=P[15]), -9), (dict(dsc=P[3]), -9), (dict(dx=P[8]), -9), (dict(ws=P[12]), -9), (dict(dx=P[12] + 8), -4)])
def test_gated_backward_refusals(L, kw, code):
    assert _gated_bwd(L, **kw) == code


def test_binding_refuses_cpu_tensors():
    x, w = torch.zeros(1, 2, 3, 64), torch.zeros(2, 64, 4)
    for call in (lambda: fw.select_prefill(x, x, x, torch.zeros(1, 2, 3), torch.zeros(2)),
                 lambda: fw.select_step(x[:, :, 0].clone(), x[:, :, 0].clone(), x[:, :, 0].clone(), torch.zeros(1, 2),
                                        torch.zeros(2), torch.zeros(1, 2, 64, 64)),
                 lambda: fw.conv_prefill(x, w), lambda: fw.conv_backward(x, x, w),
                 lambda: fw.conv_step(x[:, :, 0].clone(), w, None, torch.zeros(1, 2, 3, 64)),
                 lambda: fw.gated_norm(x), lambda: fw.gated_norm_backward(x, x, None, None, x[..., 0].clone(),
                                                                          x[..., 0].clone())):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_binding_checks_shapes_and_types_first():
    x, dt, ld, w = torch.zeros(1, 2, 3, 64), torch.zeros(1, 2, 3), torch.zeros(2), torch.zeros(2, 64, 4)
    for call in (lambda: fw.select_prefill(x, x[:, :1].clone(), x, dt, ld), lambda: fw.select_prefill(x, x, x, dt[:, :1], ld),
                 lambda: fw.select_prefill(x, x, x, dt.double(), ld), lambda: fw.select_prefill(x, x, x, dt, ld.double()),
                 lambda: fw.select_prefill(x, x, x, dt, ld, skip=dt), lambda: fw.select_prefill(x, x, x.bfloat16(), dt, ld),
                 lambda: fw.conv_prefill(x, w[:, :3].clone()), lambda: fw.conv_prefill(x, w, state=x[:, :, :2]),
                 lambda: fw.conv_prefill(x, w, torch.zeros(64)), lambda: fw.conv_backward(x.bfloat16(), x, w),
                 lambda: fw.gated_norm(x, torch.zeros(63)), lambda: fw.gated_norm(x, torch.zeros(3, 64)),
                 lambda: fw.gated_norm(x, torch.zeros(2, 64), torch.zeros(64)), lambda: fw.gated_norm(x, gate=x[:, :1]),
                 lambda: fw.gated_norm_backward(x, x, None, None, x, x)):
        with pytest.raises(ValueError, match="must be"):
            call()
    with pytest.raises(ValueError, match="eps"):
        fw.gated_norm(x, eps=-1.0)
