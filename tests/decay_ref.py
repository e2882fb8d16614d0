"""Decayed linear attention and layer norm in 64 bits, token by token from the definition."""
import torch


def _lens(lens, B, T):
    return torch.full((B,), T) if lens is None else lens.cpu().long().clamp(0, T)


def forward(q, k, v, log_decay, S0=None, scale=1.0, lens=None):
    """(o, S_T, states after every token) on the CPU in fp64; o is zero behind lens."""
    q, k, v = (t.detach().cpu().double() for t in (q, k, v))
    B, H, T, d = q.shape
    g = torch.exp(log_decay.detach().cpu().double()).view(1, H, 1, 1)
    S = torch.zeros(B, H, d, d, dtype=torch.float64) if S0 is None else S0.detach().cpu().double().clone()
    n = _lens(lens, B, T)
    o, hist = torch.zeros_like(q), []
    for t in range(T):
        on = (t < n).view(B, 1, 1, 1)
        # no arithmetic on rows behind the end: they may hold anything
        S = torch.where(on, g * S + k[:, :, t, :, None] * v[:, :, t, None, :], S)
        r = scale * torch.einsum("bhi,bhij->bhj", q[:, :, t], S)
        o[:, :, t] = torch.where(on[..., 0], r, torch.zeros_like(r))
        hist.append(S)
    return o, S, hist


def backward(q, k, v, log_decay, do, S0=None, dS_T=None, scale=1.0, lens=None):
    """(dq, dk, dv, dS0) by the gradient's formula."""
    _, _, hist = forward(q, k, v, log_decay, S0, scale, lens)
    q, k, v, do = (t.detach().cpu().double() for t in (q, k, v, do))
    B, H, T, d = q.shape
    g = torch.exp(log_decay.detach().cpu().double()).view(1, H, 1, 1)
    D = torch.zeros(B, H, d, d, dtype=torch.float64) if dS_T is None else dS_T.detach().cpu().double()
    n = _lens(lens, B, T)
    dq, dk, dv = (torch.zeros_like(q) for _ in range(3))
    for t in reversed(range(T)):
        on = (t < n).view(B, 1, 1, 1)
        Dt = D + scale * q[:, :, t, :, None] * do[:, :, t, None, :]

        def put(dst, x):
            dst[:, :, t] = torch.where(on[..., 0], x, torch.zeros_like(x))

        put(dq, scale * torch.einsum("bhij,bhj->bhi", hist[t], do[:, :, t]))
        put(dk, torch.einsum("bhij,bhj->bhi", Dt, v[:, :, t]))
        put(dv, torch.einsum("bhij,bhi->bhj", Dt, k[:, :, t]))
        D = torch.where(on, g * Dt, D)
    return dq, dk, dv, D


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    x = x.detach().cpu().double()
    m = x.mean(-1, keepdim=True)
    r = 1 / torch.sqrt(((x - m) ** 2).mean(-1, keepdim=True) + eps)
    y = (x - m) * r
    if weight is not None:
        y = y * weight.detach().cpu().double()
    if bias is not None:
        y = y + bias.detach().cpu().double()
    return y, m[..., 0], r[..., 0]


def layer_norm_backward(dy, x, weight=None, eps=1e-5):
    _, m, r = layer_norm(x, eps=eps)
    x, dy = x.detach().cpu().double(), dy.detach().cpu().double()
    xh = (x - m[..., None]) * r[..., None]
    g = dy if weight is None else dy * weight.detach().cpu().double()
    dx = r[..., None] * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    lead = tuple(range(x.dim() - 1))
    return dx, (dy * xh).sum(lead), dy.sum(lead)


def rel(got, ref):
    got, ref = got.detach().cpu().double(), ref.double()
    assert got.shape == ref.shape
    assert torch.isfinite(got).all()
    n = ref.norm().item()
    return (got - ref).norm().item() / n if n else (got - ref).norm().item()


def rel_rows(got, ref, lead):
    """The largest relative L2 error over the entries of the first `lead` axes."""
    g = got.detach().cpu().double().reshape(-1, *got.shape[lead:]).flatten(1)
    r = ref.double().reshape(-1, *ref.shape[lead:]).flatten(1)
    assert torch.isfinite(g).all()
    num, den = (g - r).norm(dim=1), r.norm(dim=1)
    return torch.where(den > 0, num / den.clamp_min(1e-300), num).max().item()
