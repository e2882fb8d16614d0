"""Linear attention with a decay for each head, and layer norm: what is measured.

Operators (phi applied by the caller, g_h = exp(log_decay_h), fp32 state):

    S_t = g_h S_{t-1} + k_t v_t^T,   o_t = scale * S_t^T q_t            (prefill, step)
    y   = (o - mean(o)) / sqrt(var(o) + eps) * weight + bias            (layer norm)

`run` with ``own`` false computes them in plain torch operations in fp32, with
``own`` true through the library's entry points.
"""
import math

import torch

own = False

EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

# Fixed decays of a stack's heads: "slow" spreads 1 - g over 1/32 .. 1/512, "steep" spreads
# -log g over 2^(-8/H) .. 2^-8 (the first heads forget within a few tokens).


def listed():
    return [
        # prompts of the bench's prefill shape
        dict(name="prefill_bf16_b8h16t4096", op="prefill", dtype="bf16", B=8, H=16, T=4096, d=128,
             decay="slow", s0=False, ragged=False, norm=False),
        # one long document: few chains, many tokens
        dict(name="prefill_bf16_b1h32t32768", op="prefill", dtype="bf16", B=1, H=32, T=32768,
             d=128, decay="slow", s0=False, ragged=False, norm=False),
        # a short chat turn that continues a state: latency counts
        dict(name="prefill_bf16_b1h16t37", op="prefill", dtype="bf16", B=1, H=16, T=37, d=64,
             decay="steep", s0=True, ragged=False, norm=True),
        # a padded batch of prompts of different lengths (one of them empty), output norm fused
        dict(name="prefill_bf16_ragged_norm", op="prefill", dtype="bf16", B=12, H=16, T=1777,
             d=128, decay="steep", s0=True, ragged=True, norm=True),
        # an fp32 evaluation batch, padded
        dict(name="prefill_f32_ragged", op="prefill", dtype="f32", B=4, H=8, T=1000, d=64,
             decay="slow", s0=True, ragged=True, norm=False),
        # a training step's mixer: forward and backward pass
        dict(name="train_bf16_b8h16t2048", op="train", dtype="bf16", B=8, H=16, T=2048, d=128,
             decay="slow", s0=False, ragged=False),
        # an fp32 training step on an odd length with a carried state and its gradient
        dict(name="train_f32_b2h8t1023", op="train", dtype="f32", B=2, H=8, T=1023, d=64,
             decay="steep", s0=True, ragged=False),
        # one decode step of a full serving batch (the bench's decode shape)
        dict(name="step_bf16_b256h32", op="step", dtype="bf16", B=256, H=32, d=128, decay="slow",
             norm=False),
        # one decode step of a single user, output norm fused
        dict(name="step_bf16_b1h16", op="step", dtype="bf16", B=1, H=16, d=128, decay="slow",
             norm=True),
        # the norm of a decode batch's rows
        dict(name="norm_bf16_64x2048", op="norm", dtype="bf16", rows=64, width=2048),
        # a training step's norm over the model width, forward and backward
        dict(name="norm_train_bf16_32768x2048", op="norm_train", dtype="bf16", rows=32768,
             width=2048),
        # the same over an odd width in fp32
        dict(name="norm_train_f32_5000x1023", op="norm_train", dtype="f32", rows=5000, width=1023),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "train", "step", "norm", "norm_train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "norm_train"):
        width = _log_uniform(rng, 32, 8192)
        if rng.random() < 0.5:
            width = (width + 7) // 8 * 8
        most = (1 << 26) // (width * (2 if dtype == "f32" else 1))
        return dict(op=op, dtype=dtype, rows=min(_log_uniform(rng, 1, 1 << 19), most), width=width)
    d = rng.choice([64, 128, 128])
    decay = rng.choice(["slow", "steep"])
    if op == "step":
        return dict(op=op, dtype=dtype, B=_log_uniform(rng, 1, 256), H=rng.randint(1, 32), d=d,
                    decay=decay, norm=rng.random() < 0.5)
    B, H = rng.randint(1, 12), rng.randint(1, 32)
    most = (1 << (23 if dtype == "f32" else 25 if op == "train" else 26)) // (B * H * d)
    T = min(_log_uniform(rng, 1, 32768), most)
    case = dict(op=op, dtype=dtype, B=B, H=H, T=T, d=d, decay=decay, s0=rng.random() < 0.5,
                ragged=rng.random() < 0.4)
    if op == "prefill":
        case["norm"] = rng.random() < 0.5
    return case


def _lens(case):
    """Lengths of a padded batch: spread over 0 .. T, the second row empty, the first full."""
    B, T = case["B"], case["T"]
    out = [int(T * ((0.6180339887 * b) % 1.0)) for b in range(B)]
    out[0] = T
    if B > 1:
        out[1] = 0
    return out


def _log_decay(case, device):
    H = case["H"]
    h = torch.arange(H, dtype=torch.float64)
    if case["decay"] == "slow":
        x = torch.log1p(-torch.exp(torch.linspace(math.log(1 / 32), math.log(1 / 512), H,
                                                  dtype=torch.float64)))
    else:
        x = -torch.exp2(-8.0 * (h + 1) / H)
    return x.to(device=device, dtype=torch.float32)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def normal(*shape, dtype=dt, std=1.0):
        return (torch.randn(shape, generator=g, device=dev, dtype=torch.float32) * std).to(dtype)

    st = {"case": case}
    op = case["op"]
    if op in ("norm", "norm_train"):
        n, w = case["rows"], case["width"]
        # residual-stream rows: a mean and a spread of their own
        mu = torch.randn((n, 1), generator=g, device=dev)
        st["x"] = (torch.randn((n, w), generator=g, device=dev) * (1 + mu * mu) + mu).to(dt)
        st["weight"] = 1 + normal(w, dtype=torch.float32, std=0.2)
        st["bias"] = normal(w, dtype=torch.float32, std=0.2)
        if op == "norm_train":
            st["dy"] = normal(n, w)
        return st
    B, H, d = case["B"], case["H"], case["d"]
    st["scale"] = d ** -0.5
    st["log_decay"] = _log_decay(case, dev)
    lead = (B, H) if op == "step" else (B, H, case["T"])
    for name in ("q", "k", "v"):
        st[name] = normal(*lead, d)
    if case.get("norm"):
        st["weight"] = 1 + normal(d, dtype=torch.float32, std=0.2)
        st["bias"] = normal(d, dtype=torch.float32, std=0.2)
    if op == "step":
        # what a few hundred tokens leave behind
        st["S"] = normal(B, H, d, d, dtype=torch.float32, std=8.0)
        return st
    st["S0"] = normal(B, H, d, d, dtype=torch.float32, std=8.0) if case["s0"] else None
    st["lens"] = (torch.tensor(_lens(case), device=dev, dtype=torch.int32) if case["ragged"]
                  else None)
    if op == "train":
        st["do"] = normal(*lead, d)
        st["dS_T"] = normal(B, H, d, d, dtype=torch.float32) if case["s0"] else None
    return st


# ---- plain forms ---------------------------------------------------------------

CHUNK = 64


def _plain_norm(x, weight, bias):
    mean = x.mean(-1, keepdim=True)
    xc = x - mean
    rstd = torch.rsqrt((xc * xc).mean(-1, keepdim=True) + EPS)
    return xc * rstd * weight + bias, mean, rstd


def _plain_scan(a, b, c, log_decay, X, lens, reverse):
    """out_i = sum_j g^|i-j| (a_i.b_j) c_j over j <= i (reverse: j >= i) plus the carried state's
    read, in fp32 chunk by chunk.  Forward: X' = g^n X + sum_j g^(n-1-j) b_j c_j^T, read with
    g^(i+1).  Reverse: X' = g^n X + sum_j g^(j+1) b_j c_j^T, read with g^(n-1-i).  n counts the
    chunk's rows before the sequence's end.  Returns (out, X)."""
    B, H, T, d = a.shape
    dev = a.device
    X = torch.zeros((B, H, d, d), device=dev) if X is None else X.float()
    ends = torch.full((B,), T, device=dev) if lens is None else lens.long()
    ld = log_decay.double().view(1, H, 1)
    out = torch.zeros((B, H, T, d), device=dev)
    starts = range(0, T, CHUNK)
    for c0 in (reversed(starts) if reverse else starts):
        c1 = min(c0 + CHUNK, T)
        i = torch.arange(c1 - c0, device=dev)
        n = (ends - c0).clamp(0, c1 - c0).view(B, 1, 1)
        valid = (i.view(1, 1, -1) < n).float()
        A, Bk, C = (t[:, :, c0:c1].float() for t in (a, b, c))
        lag = i.view(-1, 1) - i.view(1, -1)
        if reverse:
            lag = -lag
            read, write = n - 1 - i.view(1, 1, -1), (i + 1).view(1, 1, -1)
        else:
            read, write = (i + 1).view(1, 1, -1), n - 1 - i.view(1, 1, -1)
        decay = torch.exp(ld.view(1, H, 1, 1) * lag.clamp(min=0)).float() * (lag >= 0)
        wr = torch.exp(ld * write.clamp(min=0)).float() * valid
        rd = torch.exp(ld * read.clamp(min=0)).float()
        Bk = Bk * valid[..., None]
        P = torch.matmul(A, Bk.transpose(-1, -2)) * decay
        o = torch.matmul(P, C) + rd[..., None] * torch.matmul(A, X)
        out[:, :, c0:c1] = o * valid[..., None]
        X = torch.exp(ld * n).float()[..., None] * X + torch.matmul(
            (Bk * wr[..., None]).transpose(-1, -2), C)
    return out, X


def _plain(st):
    case = st["case"]
    op, dt = case["op"], DTYPES[case["dtype"]]
    if op == "norm":
        return [_plain_norm(st["x"].float(), st["weight"], st["bias"])[0].to(dt)]
    if op == "norm_train":
        x, dy = st["x"].float(), st["dy"].float()
        y, mean, rstd = _plain_norm(x, st["weight"], st["bias"])
        xh = (x - mean) * rstd
        wdy = dy * st["weight"]
        dx = rstd * (wdy - wdy.mean(-1, keepdim=True) - xh * (wdy * xh).mean(-1, keepdim=True))
        return [y.to(dt), dx.to(dt), (dy * xh).sum(0), dy.sum(0)]
    scale = st["scale"]
    if op == "step":
        q, k, v = (st[x].float() for x in "qkv")
        gamma = torch.exp(st["log_decay"]).view(1, -1, 1, 1)
        S = gamma * st["S"] + k[..., :, None] * v[..., None, :]
        o = scale * torch.matmul(q[..., None, :], S)[..., 0, :]
        if case["norm"]:
            o = _plain_norm(o, st["weight"], st["bias"])[0]
        st["S"].copy_(S)
        return [o.to(dt), st["S"]]
    q, k, v, ld, lens = st["q"], st["k"], st["v"], st["log_decay"], st["lens"]
    o, S_T = _plain_scan(q, k, v, ld, st["S0"], lens, False)
    o = o * scale
    if op == "prefill":
        if case["norm"]:
            o = _plain_norm(o, st["weight"], st["bias"])[0]
            if lens is not None:
                t = torch.arange(case["T"], device=o.device)
                o = torch.where((t.view(1, 1, -1, 1) < lens.view(-1, 1, 1, 1)), o, 0.0)
        return [o.to(dt), S_T]
    do, dS = st["do"], st["dS_T"]
    S0t = None if st["S0"] is None else st["S0"].transpose(-1, -2)
    dSt = None if dS is None else dS.transpose(-1, -2)
    dos = do.float() * scale
    dq, _ = _plain_scan(dos, v, k, ld, S0t, lens, False)
    dv, dS0 = _plain_scan(k, q, dos, ld, dS, lens, True)
    dk, _ = _plain_scan(v, dos, q, ld, dSt, lens, True)
    out = [o.to(dt), S_T, dq.to(dt), dk.to(dt), dv.to(dt)]
    return out + [dS0] if case["s0"] else out


# ---- the library's calls -------------------------------------------------------


def _own(st):
    from linear_token_mixer_gb300 import fw
    case = st["case"]
    op = case["op"]
    if op == "norm":
        return [fw.layer_norm(st["x"], st["weight"], st["bias"], eps=EPS)[0]]
    if op == "norm_train":
        y, mean, rstd = fw.layer_norm(st["x"], st["weight"], st["bias"], eps=EPS)
        dx, dw, db = fw.layer_norm_backward(st["dy"], st["x"], st["weight"], mean, rstd)
        return [y, dx, dw, db]
    norm = (st["weight"], st["bias"]) if case.get("norm") else None
    q, k, v, ld, scale = st["q"], st["k"], st["v"], st["log_decay"], st["scale"]
    if op == "step":
        return [fw.decay_step(q, k, v, ld, st["S"], scale=scale, norm=norm, norm_eps=EPS), st["S"]]
    o, S_T = fw.decay_prefill(q, k, v, ld, st["S0"], scale=scale, lens=st["lens"], norm=norm,
                              norm_eps=EPS)
    if op == "prefill":
        return [o, S_T]
    dq, dk, dv, dS0 = fw.decay_backward(q, k, v, ld, st["do"], st["S0"], st["dS_T"], scale=scale,
                                        lens=st["lens"])
    out = [o, S_T, dq, dk, dv]
    return out + [dS0] if case["s0"] else out


def run(state):
    return _own(state) if own else _plain(state)


# ---- the definition in 64 bits, token by token ---------------------------------


def _exact_norm(o, st):
    m = o.sum(-1, keepdim=True) / o.shape[-1]
    var = ((o - m) ** 2).sum(-1, keepdim=True) / o.shape[-1]
    return (o - m) / torch.sqrt(var + EPS) * st["weight"].double() + st["bias"].double()


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        return [_exact_norm(st["x"].double(), st)]
    if op == "norm_train":
        x, dy, w = st["x"].double(), st["dy"].double(), st["weight"].double()
        y = _exact_norm(x, st)
        m = x.sum(-1, keepdim=True) / case["width"]
        s = torch.sqrt(((x - m) ** 2).sum(-1, keepdim=True) / case["width"] + EPS)
        xh = (x - m) / s
        c1 = (dy * w).sum(-1, keepdim=True) / case["width"]
        c2 = (dy * w * xh).sum(-1, keepdim=True) / case["width"]
        return [y, (dy * w - c1 - xh * c2) / s, torch.einsum("nw,nw->w", dy, xh), dy.sum(0)]
    B, H, d = case["B"], case["H"], case["d"]
    n, scale = B * H, st["scale"]
    gam = torch.exp(st["log_decay"].double()).repeat(B).view(n, 1, 1)
    if op == "step":
        q, k, v = (st[x].double().view(n, d) for x in "qkv")
        S = gam * st["S"].double().view(n, d, d) + torch.einsum("ni,nj->nij", k, v)
        o = scale * torch.einsum("ni,nij->nj", q, S)
        if case["norm"]:
            o = _exact_norm(o, st)
        return [o.view(B, H, d), S.view(B, H, d, d)]
    T = case["T"]
    names = ("q", "k", "v", "do") if op == "train" else ("q", "k", "v")
    # token-major copies, so that one token of every chain is one contiguous block
    tok = {x: st[x].view(n, T, d).transpose(0, 1).contiguous() for x in names}
    lens = torch.full((B,), T) if st["lens"] is None else st["lens"].cpu().long()
    live = (torch.arange(T).view(T, 1) < lens.repeat_interleave(H).view(1, n)).to(gam.device)

    def state(name):
        return (torch.zeros((n, d, d), dtype=torch.float64, device=gam.device)
                if st.get(name) is None else st[name].double().view(n, d, d).clone())

    S = state("S0")
    o = torch.zeros((T, n, d), dtype=torch.float64, device=gam.device)
    dq, dk, dv = (torch.zeros_like(o) if op == "train" else None for _ in range(3))
    for t in range(T):
        on = live[t].view(n, 1, 1)
        k = tok["k"][t].double().view(n, d, 1) * on
        S.mul_(torch.where(on, gam, 1.0)).baddbmm_(k, tok["v"][t].double().view(n, 1, d))
        o[t] = torch.bmm(tok["q"][t].double().view(n, 1, d), S)[:, 0] * scale
        if op == "train":
            dq[t] = torch.bmm(S, tok["do"][t].double().view(n, d, 1))[..., 0] * scale
    if op == "prefill" and case["norm"]:
        o = _exact_norm(o, st)
    if op == "train":
        D = state("dS_T")
        for t in reversed(range(T)):
            on = live[t].view(n, 1, 1)
            q = tok["q"][t].double().view(n, d, 1) * on * scale
            D.baddbmm_(q, tok["do"][t].double().view(n, 1, d))
            dk[t] = torch.bmm(D, tok["v"][t].double().view(n, d, 1))[..., 0]
            dv[t] = torch.bmm(tok["k"][t].double().view(n, 1, d), D)[:, 0]
            D.mul_(torch.where(on, gam, 1.0))

    def rows(x):
        return (x * live[..., None]).transpose(0, 1).reshape(B, H, T, d)

    out = [rows(o), S.view(B, H, d, d)]
    if op == "train":
        out += [rows(dq), rows(dk), rows(dv)]
        if case["s0"]:
            out.append(D.view(B, H, d, d))
    return out


def work(case):
    """Bytes: every input read once, every output written once (rows before each sequence's end).
    Operations: the recurrence's multiply-adds (a write and a read of the state per token; in the
    backward pass the state again, its gradient, and three reads)."""
    op = case["op"]
    e = 2 if case["dtype"] == "bf16" else 4
    if op in ("norm", "norm_train"):
        n, w = case["rows"], case["width"]
        if op == "norm":
            return {"bytes": 2 * n * w * e + 8 * w, "flops": 8 * n * w}
        return {"bytes": 4 * n * w * e + 16 * w, "flops": 20 * n * w}
    B, H, d = case["B"], case["H"], case["d"]
    state = B * H * d * d * 4
    if op == "step":
        return {"bytes": 2 * state + 4 * B * H * d * e, "flops": 5 * B * H * d * d}
    tok = H * (sum(_lens(case)) if case["ragged"] else B * case["T"])
    s0 = 1 if case["s0"] else 0
    if op == "prefill":
        return {"bytes": 4 * tok * d * e + (1 + s0) * state, "flops": 4 * tok * d * d}
    return {"bytes": 8 * tok * d * e + (1 + 3 * s0) * state, "flops": 14 * tok * d * d}
