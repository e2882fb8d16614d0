"""Selective scan, short causal convolution and gated norm in 64 bits, from their definitions.  Gradients
come from differentiating them."""
import torch

from decay_ref import rel, rel_rows  # noqa: F401


def f64(t):
    return None if t is None else t.detach().cpu().double()


def ends(lens, B, T):
    return [T] * B if lens is None else [min(max(int(n), 0), T) for n in lens.cpu()]


def steps(dt, dt_bias, softplus, heads_at=1):
    x = f64(dt)
    if dt_bias is not None:
        x = x + f64(dt_bias).view([-1 if i == heads_at else 1 for i in range(x.dim())])
    return torch.log1p(torch.exp(-x.abs())) + x.clamp_min(0) if softplus else x


def select(q, k, v, dt, log_decay, S0=None, dt_bias=None, softplus=False, skip=None, scale=1.0, lens=None):
    """(o, S_T), token by token; o is zero behind lens, and nothing there is touched."""
    B, H, T, d = v.shape
    G = q.shape[1]
    q, k = (f64(t).repeat_interleave(H // G, 1) for t in (q, k))
    v, dt, A = f64(v), steps(dt, dt_bias, softplus), f64(log_decay)
    sk = torch.zeros(H, dtype=torch.float64) if skip is None else f64(skip)
    S = torch.zeros(B, H, d, d, dtype=torch.float64) if S0 is None else f64(S0).clone()
    o = torch.zeros_like(v)
    for b, n in enumerate(ends(lens, B, T)):
        for t in range(n):
            g = torch.exp(A * dt[b, :, t]).view(H, 1, 1)
            S[b] = g * S[b] + (dt[b, :, t, None] * k[b, :, t]).unsqueeze(-1) * v[b, :, t].unsqueeze(-2)
            o[b, :, t] = scale * torch.einsum("hi,hij->hj", q[b, :, t], S[b]) + sk[:, None] * v[b, :, t]
    return o, S


def conv(x, weight, bias=None, state=None, silu=True, lens=None):
    """(y, state_out) of 64-bit tensors (leaves of a graph, or not)."""
    B, H, T, d = x.shape
    W = weight.shape[2]
    past = torch.zeros(B, H, W - 1, d, dtype=torch.float64) if state is None else state
    ys, so = [], []
    for b, n in enumerate(ends(lens, B, T)):
        r = torch.cat([past[b], x[b, :, :n]], 1)
        a = torch.zeros(H, n, d, dtype=torch.float64) if bias is None else bias[:, None].expand(H, n, d)
        for w in range(W):
            a = a + weight[:, None, :, w] * r[:, w:w + n]
        y = a / (1 + torch.exp(-a)) if silu else a
        ys.append(torch.cat([y, torch.zeros(H, T - n, d, dtype=torch.float64)], 1))
        so.append(r[:, n:n + W - 1])
    return torch.stack(ys), torch.stack(so)


def conv_grads(dy, x, weight, bias=None, state=None, dstate_out=None, silu=True, lens=None):
    """(dx, dweight, dbias, dstate)."""
    B, H, T, d = x.shape
    W = weight.shape[2]
    bias = torch.zeros(H, d) if bias is None else bias
    state = torch.zeros(B, H, W - 1, d) if state is None else state
    leaf = [f64(t).requires_grad_() for t in (x, weight, bias, state)]
    y, so = conv(*leaf, silu, lens)
    on = torch.zeros(B, 1, T, 1, dtype=torch.bool)
    for b, n in enumerate(ends(lens, B, T)):
        on[b, :, :n] = True
    loss = (y * torch.where(on, f64(dy), 0.0)).sum()
    if dstate_out is not None:
        loss = loss + (so * f64(dstate_out)).sum()
    got = torch.autograd.grad(loss, leaf, allow_unused=True)
    return [torch.zeros_like(t) if g is None else g for g, t in zip(got, leaf)]


def _wide(p):
    """[width], or [H, width] against [.., H, T, width]."""
    return p if p is None or p.dim() == 1 else p.unsqueeze(1)


def gated(x, weight=None, bias=None, gate=None, residual=None, scale=None, rms=False, gate_after=False, eps=1e-5):
    """(y, u, mean, rstd) of 64-bit tensors (leaves of a graph, or not)."""
    u = x
    if residual is not None:
        u = x + (residual if scale is None else _wide(scale) * residual)
    act = None if gate is None else gate * torch.sigmoid(gate)   # (whose derivative is finite for any gate)
    s = u if act is None or gate_after else u * act
    m = torch.zeros_like(s[..., :1]) if rms else s.mean(-1, keepdim=True)
    r = 1 / torch.sqrt(((s - m) ** 2).mean(-1, keepdim=True) + eps)
    y = (s - m) * r
    if weight is not None:
        y = y * _wide(weight)
    if bias is not None:
        y = y + _wide(bias)
    if act is not None and gate_after:
        y = y * act
    return y, u, m[..., 0], r[..., 0]


def gated_grads(dy, dtotal=None, eps=1e-5, **given):
    """Gradients by name, of the tensors given."""
    leaf = {n: f64(t).requires_grad_() for n, t in given.items() if isinstance(t, torch.Tensor)}
    rest = {n: t for n, t in given.items() if not isinstance(t, torch.Tensor)}
    y, u, _, _ = gated(eps=eps, **leaf, **rest)
    loss = (y * f64(dy)).sum()
    if dtotal is not None:
        loss = loss + (u * f64(dtotal)).sum()
    return dict(zip(leaf, torch.autograd.grad(loss, list(leaf.values()))))
