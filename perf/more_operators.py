"""Short causal convolution, selective scan and gated norm: what is measured.

    y_t = act(bias + sum_w weight[w] x_{t-W+1+w})                          (conv; act: silu or none)
    dt_t = softplus(dt_raw_t + dt_bias_h),  g_t = exp(log_decay_h dt_t),
    S_t = g_t S_{t-1} + dt_t k_t v_t^T,  o_t = scale S_t^T q_t + skip_h v_t   (select, S in fp32)
    u = x + scale * residual,  s = u silu(gate),  y = norm(s) weight + bias   (gated norm, gate before)
    u = x + scale * residual,  y = (norm(u) weight + bias) silu(gate)         (gated norm, gate after)

`run` with ``own`` false computes them in plain torch operations in fp32, with
``own`` true through the library's entry points.
"""
import math

import torch

own = False

EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one decode step's convolution of a full serving batch (the bench's decode shape)
        dict(name="conv_step_bf16_b256h32", op="conv_step", dtype="bf16", B=256, H=32, d=128, W=4, silu=True),
        # a training step's convolution of one of q, k, v: forward and backward pass
        dict(name="conv_train_bf16_b8h16t2048", op="conv_train", dtype="bf16", B=8, H=16, T=2048, d=128, W=4,
             silu=True, state=False, ragged=False),
        # an fp32 training step on a padded batch of odd lengths that continues carried rows
        dict(name="conv_train_f32_b4h8t1023", op="conv_train", dtype="f32", B=4, H=8, T=1023, d=65, W=3,
             silu=False, state=True, ragged=True),
        # prompts of the bench's prefill shape, keys and queries for each head
        dict(name="select_bf16_b8h16t4096", op="select", dtype="bf16", B=8, H=16, G=16, T=4096, d=128, s0=False,
             ragged=False, softplus=True, skip=True),
        # one long document, keys and queries shared by eight heads: few chains, many tokens
        dict(name="select_bf16_b1h32t32768", op="select", dtype="bf16", B=1, H=32, G=4, T=32768, d=128, s0=False,
             ragged=False, softplus=True, skip=True),
        # a padded batch of prompts of different lengths (one of them empty) that continue states
        dict(name="select_bf16_ragged", op="select", dtype="bf16", B=12, H=16, G=2, T=1777, d=128, s0=True,
             ragged=True, softplus=True, skip=True),
        # a short chat turn that continues a state: latency counts
        dict(name="select_bf16_b1h16t37", op="select", dtype="bf16", B=1, H=16, G=1, T=37, d=64, s0=True,
             ragged=False, softplus=True, skip=True),
        # an fp32 evaluation batch, padded, steps formed by the caller
        dict(name="select_f32_ragged", op="select", dtype="f32", B=4, H=8, G=8, T=1000, d=64, s0=True, ragged=True,
             softplus=False, skip=False),
        # one decode step of a full serving batch
        dict(name="select_step_bf16_b256h32", op="select_step", dtype="bf16", B=256, H=32, G=4, d=128,
             softplus=True, skip=True),
        # the norm of a decode batch's rows, with the residual sum before it
        dict(name="norm_bf16_64x2048", op="norm", dtype="bf16", H=1, rows=64, width=2048, rms=True, gate="none",
             residual=True, bias=False),
        # behind a training step's mixer: each head's rows gated, normed with its own weights, and back
        dict(name="norm_train_bf16_262144x128", op="norm_train", dtype="bf16", H=16, rows=262144, width=128,
             rms=True, gate="before", residual=False, bias=False),
        # a training step's norm over an odd width in fp32, scaled residual sum before it, gate behind it
        dict(name="norm_train_f32_5000x1023", op="norm_train", dtype="f32", H=1, rows=5000, width=1023, rms=False,
             gate="after", residual=True, bias=True),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "conv_train", "conv_step", "select", "select", "select", "select_step", "norm",
                     "norm_train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    half = 1 if dtype == "bf16" else 2
    if op in ("norm", "norm_train"):
        width = _log_uniform(rng, 32, 8192)
        if rng.random() < 0.5:
            width = (width + 7) // 8 * 8
        H = rng.choice([1, 1, rng.randint(2, 24)])
        rows = min(_log_uniform(rng, 1, 1 << 18), (1 << 24) // (width * half))
        gate = rng.choice(["none", "before", "after"])
        return dict(op=op, dtype=dtype, H=H, rows=max(rows // H, 1) * H, width=width, rms=rng.random() < 0.5,
                    gate=gate, residual=gate == "none" or rng.random() < 0.5, bias=rng.random() < 0.5)
    if op.startswith("conv"):
        W = rng.choice([2, 3, 4, 4, 4, 5, 8])
        d = _log_uniform(rng, 16, 4096)
        if rng.random() < 0.6:
            d = (d + 7) // 8 * 8
        B, H, silu = rng.randint(1, 16), rng.randint(1, 8), rng.random() < 0.7
        if op == "conv_step":
            return dict(op=op, dtype=dtype, B=_log_uniform(rng, 1, 64), H=H, d=d, W=W, silu=silu)
        most = max((1 << 25) // (B * H * d * half), 1)
        return dict(op=op, dtype=dtype, B=B, H=H, T=min(_log_uniform(rng, 1, 32768), most), d=d, W=W, silu=silu,
                    state=rng.random() < 0.5, ragged=rng.random() < 0.4)
    d = rng.choice([64, 128, 128])
    G = rng.randint(1, 8)
    H = G * rng.choice([1, 2, 3, 4]) if rng.random() < 0.6 else G
    case = dict(op=op, dtype=dtype, H=H, G=G, d=d, softplus=rng.random() < 0.7, skip=rng.random() < 0.6)
    if op == "select_step":
        return dict(case, B=_log_uniform(rng, 1, 256))
    B = rng.randint(1, 12)
    most = max((1 << (23 if dtype == "f32" else 26)) // (B * H * d), 1)
    return dict(case, B=B, T=min(_log_uniform(rng, 1, 32768), most), s0=rng.random() < 0.5,
                ragged=rng.random() < 0.4)


def _lens(case):
    """Lengths of a padded batch: spread over 0 .. T, the second row empty, the first full."""
    B, T = case["B"], case["T"]
    out = [int(T * ((0.6180339887 * b) % 1.0)) for b in range(B)]
    out[0] = T
    if B > 1:
        out[1] = 0
    return out


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    dt, f32 = DTYPES[case["dtype"]], torch.float32

    def normal(*shape, dtype=dt, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=g, device=dev, dtype=f32) * std + mean).to(dtype)

    def uniform(lo, hi, *shape):
        return lo + (hi - lo) * torch.rand(shape, generator=g, device=dev, dtype=f32)

    st = {"case": case}
    op = case["op"]
    if op in ("norm", "norm_train"):
        H, n, w = case["H"], case["rows"], case["width"]
        shape = (H, n // H, w) if H > 1 else (n, w)
        par = (H, w) if H > 1 else (w,)
        st["x"] = normal(*shape) * 2 + normal(*shape[:-1], 1)
        st["weight"] = normal(*par, dtype=f32, std=0.2, mean=1.0)
        st["bias"] = normal(*par, dtype=f32, std=0.2) if case["bias"] else None
        st["gate"] = normal(*shape) if case["gate"] != "none" else None
        st["residual"] = normal(*shape, std=4.0) if case["residual"] else None
        st["scale"] = normal(*par, dtype=f32, std=0.2, mean=0.5) if case["residual"] else None
        if op == "norm_train":
            st["dy"] = normal(*shape)
            st["dtotal"] = normal(*shape) if case["residual"] else None
        return st
    B, H, d = case["B"], case["H"], case["d"]
    if op.startswith("conv"):
        W = case["W"]
        st["weight"] = normal(H, d, W, dtype=f32, std=W ** -0.5)
        st["bias"] = normal(H, d, dtype=f32, std=0.2)
        if op == "conv_step":
            st["x"], st["state"] = normal(B, H, d), normal(B, H, W - 1, d)
            return st
        st["x"] = normal(B, H, case["T"], d)
        st["state"] = normal(B, H, W - 1, d) if case["state"] else None
        st["lens"] = torch.tensor(_lens(case), device=dev, dtype=torch.int32) if case["ragged"] else None
        if op == "conv_train":
            st["dy"] = normal(B, H, case["T"], d)
            st["dstate"] = normal(B, H, W - 1, d) if case["state"] else None
        return st
    G = case["G"]
    tok = () if op == "select_step" else (case["T"],)
    st["scale"] = d ** -0.5
    st["q"], st["k"], st["v"] = normal(B, G, *tok, d), normal(B, G, *tok, d), normal(B, H, *tok, d)
    # rates of 1 .. 16 and steps of about 0.001 .. 0.1: from heads that keep thousands of tokens to
    # heads that forget within a few
    st["log_decay"] = -uniform(1.0, 16.0, H)
    step = torch.exp(uniform(math.log(0.001), math.log(0.1), H))
    raw = normal(B, H, *tok, dtype=f32)
    if case["softplus"]:
        st["dt_bias"] = step + torch.log(-torch.expm1(-step))
        st["dt"] = raw.to(dt)
    else:
        st["dt_bias"] = None
        st["dt"] = (torch.exp(0.5 * raw) * step.view(1, H, *(1 for _ in tok))).to(dt)
    st["skip"] = normal(H, dtype=f32, std=0.2, mean=1.0) if case["skip"] else None
    if op == "select_step":
        st["S"] = normal(B, H, d, d, dtype=f32, std=0.2)
        return st
    st["S0"] = normal(B, H, d, d, dtype=f32, std=0.2) if case["s0"] else None
    st["lens"] = torch.tensor(_lens(case), device=dev, dtype=torch.int32) if case["ragged"] else None
    return st


# ---- plain forms ---------------------------------------------------------------


def _valid(case, st, dev):
    """[B, 1, T, 1]: the tokens before each row's end."""
    t = torch.arange(case["T"], device=dev).view(1, 1, -1, 1)
    ends = (torch.full((case["B"],), case["T"], device=dev) if st["lens"] is None else st["lens"].long())
    return t < ends.view(-1, 1, 1, 1), ends


def _plain_conv(case, st):
    dt, W, T = DTYPES[case["dtype"]], case["W"], case["T"]
    B, H, d = case["B"], case["H"], case["d"]
    x, wt, bias = st["x"].float(), st["weight"], st["bias"]
    on, ends = _valid(case, st, x.device)
    x = torch.where(on, x, 0.0)
    past = x.new_zeros((B, H, W - 1, d)) if st["state"] is None else st["state"].float()
    rows = torch.cat([past, x], 2)                                   # [B, H, W - 1 + T, d]
    pre = (rows.unfold(2, W, 1) * wt.view(1, H, 1, d, W)).sum(-1) + bias.view(1, H, 1, d)
    sig = torch.sigmoid(pre)
    y = torch.where(on, pre * sig if case["silu"] else pre, 0.0)
    at = (ends.view(B, 1, 1, 1) + torch.arange(W - 1, device=x.device).view(1, 1, -1, 1)).expand(B, H, W - 1, d)
    out = [y.to(dt), rows.gather(2, at).to(dt)]
    if case["op"] == "conv":
        return out
    dpre = st["dy"].float() * (sig * (1.0 + pre * (1.0 - sig)) if case["silu"] else 1.0)
    dpre = torch.where(on, dpre, 0.0)
    wide = torch.nn.functional.pad(dpre, (0, 0, W - 1, W - 1)).unfold(2, W, 1)
    drows = (wide * wt.flip(-1).view(1, H, 1, d, W)).sum(-1)         # [B, H, W - 1 + T, d]
    if st["dstate"] is not None:
        drows = drows.scatter_add(2, at, st["dstate"].float())
    dw = (rows.unfold(2, W, 1) * dpre.unsqueeze(-1)).sum((0, 2))
    out += [torch.where(on, drows[:, :, W - 1:], 0.0).to(dt), dw, dpre.sum((0, 2))]
    return out + [drows[:, :, :W - 1].to(dt)] if case["state"] else out


def _plain_conv_step(case, st):
    dt, W = DTYPES[case["dtype"]], case["W"]
    rows = torch.cat([st["state"], st["x"].unsqueeze(2)], 2)          # [B, H, W, d]
    pre = torch.einsum("bhwd,hdw->bhd", rows.float(), st["weight"]) + st["bias"]
    st["state"].copy_(rows[:, :, 1:])
    return [(pre * torch.sigmoid(pre) if case["silu"] else pre).to(dt), st["state"]]


def _steps(case, st):
    """dt and its log decays [B, H, ..] in 64 bits: sums of them follow."""
    H = case["H"]
    shape = (1, H, 1)[:st["dt"].dim()]
    x = st["dt"].double()
    if case["softplus"]:
        x = x + st["dt_bias"].double().view(shape)
        x = torch.clamp(x, min=0.0) + torch.log1p(torch.exp(-x.abs()))
    return x, x * st["log_decay"].double().view(shape)


CHUNK = 128


def _plain_select(case, st):
    B, H, G, T, d = (case[x] for x in "BHGTd")
    dt_, C = DTYPES[case["dtype"]], CHUNK
    dev = st["q"].device
    on, ends = _valid(case, st, dev)
    n = (T + C - 1) // C
    steps, logs = _steps(case, st)
    steps, logs = (torch.where(on[..., 0], x, 0.0) for x in (steps, logs))

    def chunks(x):   # [B, H, T, ..] -> [B, H, n, C, ..], zeros behind the end
        pad = x.new_zeros(x.shape[:2] + (n * C - T,) + x.shape[3:])
        return torch.cat([x, pad], 2).view(x.shape[:2] + (n, C) + x.shape[3:])

    def heads(x):
        return x.repeat_interleave(H // G, 1)

    q = heads(chunks(st["q"].float()))
    k = heads(chunks(torch.where(on, st["k"].float(), 0.0)))
    v = chunks(torch.where(on, st["v"].float(), 0.0))
    w = chunks(steps)
    c = torch.cumsum(chunks(logs), 3)                                 # [B, H, n, C], within a chunk
    tri = torch.ones((C, C), dtype=torch.bool, device=dev).tril()
    lag = torch.where(tri, c.unsqueeze(-1) - c.unsqueeze(-2), 0.0).float()
    P = torch.matmul(q, k.transpose(-1, -2)) * (torch.exp(lag) * tri * w.float().unsqueeze(-2))
    last = c[..., -1:]
    M = torch.matmul((k * (w * torch.exp(last - c)).float().unsqueeze(-1)).transpose(-1, -2), v)
    # the states on entry to the chunks and behind the last: sums of the chunks' own with the decays between
    e = torch.cumsum(torch.cat([last.new_zeros(B, H, 1), last[..., 0]], 2), 2)   # [B, H, n + 1]
    below = torch.ones((n + 1, n), dtype=torch.bool, device=dev).tril(-1)
    D = torch.where(below, torch.exp(torch.where(below, e.unsqueeze(-1) - e[..., 1:].unsqueeze(-2), 0.0)), 0.0)
    X = torch.matmul(D.float(), M.view(B, H, n, d * d))
    if st["S0"] is not None:
        X = X + torch.exp(e).float().unsqueeze(-1) * st["S0"].view(B, H, 1, d * d)
    X = X.view(B, H, n + 1, d, d)
    o = torch.matmul(P, v) + torch.exp(c).float().unsqueeze(-1) * torch.matmul(q, X[:, :, :n])
    o = o.view(B, H, n * C, d)[:, :, :T] * st["scale"]
    if st["skip"] is not None:
        o = o + st["skip"].view(1, H, 1, 1) * st["v"].float()
    return [torch.where(on, o, 0.0).to(dt_), X[:, :, n].contiguous()]


def _plain_select_step(case, st):
    H, G = case["H"], case["G"]
    steps, logs = _steps(case, st)
    q, k = (st[x].float().repeat_interleave(H // G, 1) for x in "qk")
    v = st["v"].float()
    S = torch.exp(logs).float()[..., None, None] * st["S"] + (
        (steps.float().unsqueeze(-1) * k)[..., :, None] * v[..., None, :])
    o = st["scale"] * torch.matmul(q[..., None, :], S)[..., 0, :]
    if st["skip"] is not None:
        o = o + st["skip"].view(1, H, 1) * v
    st["S"].copy_(S)
    return [o.to(DTYPES[case["dtype"]]), st["S"]]


def _plain_norm(case, st):
    dt, gate = DTYPES[case["dtype"]], case["gate"]

    def par(x, default):   # [width] or [H, width] against [.., H, rows, width]
        return default if x is None else x.unsqueeze(1) if x.dim() == 2 else x

    lead = (0,) if case["H"] == 1 else (1,)
    w, b, sc = par(st["weight"], 1.0), par(st["bias"], 0.0), par(st["scale"], 1.0)
    x = st["x"].float()
    r = None if st["residual"] is None else st["residual"].float()
    z = None if st["gate"] is None else st["gate"].float()
    u = x if r is None else x + sc * r
    sig = None if z is None else torch.sigmoid(z)
    s = u * (z * sig) if gate == "before" else u
    mean = s.new_zeros(s.shape[:-1] + (1,)) if case["rms"] else s.mean(-1, keepdim=True)
    sh = s - mean
    rstd = torch.rsqrt((sh * sh).mean(-1, keepdim=True) + EPS)
    sh = sh * rstd
    n = sh * w + b
    y = n * (z * sig) if gate == "after" else n
    out = [y.to(dt)] + ([] if r is None else [u.to(dt)])
    if case["op"] == "norm":
        return out
    dy = st["dy"].float()
    dsilu = None if z is None else sig * (1.0 + z * (1.0 - sig))
    dn = dy * (z * sig) if gate == "after" else dy
    wd = dn * w
    ds = wd - sh * (wd * sh).mean(-1, keepdim=True)
    if not case["rms"]:
        ds = ds - wd.mean(-1, keepdim=True)
    ds = ds * rstd
    du = ds * (z * sig) if gate == "before" else ds
    if r is not None:
        du = du + st["dtotal"].float()
    out += [du.to(dt), (dn * sh).sum(lead)]
    if st["bias"] is not None:
        out.append(dn.sum(lead))
    if z is not None:
        out.append((ds * u * dsilu if gate == "before" else dy * n * dsilu).to(dt))
    if r is not None:
        out += [(sc * du).to(dt), (du * r).sum(lead)]
    return out


PLAIN = {"conv": _plain_conv, "conv_train": _plain_conv, "conv_step": _plain_conv_step, "select": _plain_select,
         "select_step": _plain_select_step, "norm": _plain_norm, "norm_train": _plain_norm}


# ---- the library's calls -------------------------------------------------------


def _own(case, st):
    from linear_token_mixer_gb300 import fw
    op = case["op"]
    if op in ("norm", "norm_train"):
        kind = dict(gate=st["gate"], residual=st["residual"], scale=st["scale"], rms=case["rms"],
                    gate_after=case["gate"] == "after")
        train = op == "norm_train"
        y, total, mean, rstd = fw.gated_norm(st["x"], st["weight"], st["bias"], eps=EPS, stats=train, **kind)
        out = [y] + ([] if total is None else [total])
        if not train:
            return out
        grads = fw.gated_norm_backward(st["dy"], st["x"], st["weight"], st["bias"], mean, rstd,
                                       dtotal=st["dtotal"], **kind)
        dx, dweight, dbias, dgate, dresidual, dscale = grads
        return out + [t for t in (dx, dweight, dbias if case["bias"] else None, dgate, dresidual, dscale)
                      if t is not None]
    if op == "conv_step":
        return [fw.conv_step(st["x"], st["weight"], st["bias"], st["state"], silu=case["silu"]), st["state"]]
    if op.startswith("conv"):
        kind = dict(silu=case["silu"], lens=st["lens"])
        y, state = fw.conv_prefill(st["x"], st["weight"], st["bias"], st["state"], **kind)
        if op == "conv":
            return [y, state]
        dx, dw, db, dstate = fw.conv_backward(st["dy"], st["x"], st["weight"], st["bias"], st["state"], st["dstate"],
                                              **kind)
        return [y, state, dx, dw, db] + ([dstate] if case["state"] else [])
    kind = dict(dt_bias=st["dt_bias"], softplus=case["softplus"], skip=st["skip"], scale=st["scale"])
    if op == "select_step":
        return [fw.select_step(st["q"], st["k"], st["v"], st["dt"], st["log_decay"], st["S"], **kind), st["S"]]
    return list(fw.select_prefill(st["q"], st["k"], st["v"], st["dt"], st["log_decay"], st["S0"], lens=st["lens"],
                                  **kind))


def run(state):
    case = state["case"]
    return _own(case, state) if own else PLAIN[case["op"]](case, state)


# ---- the definitions in 64 bits, from the formulas -----------------------------


def _exact_norm(case, st):
    """Rows as leaves of a graph: the gradients come from differentiating the definition."""
    names = ["x", "weight", "bias", "gate", "residual", "scale"]
    leaf = {n: st[n].double().requires_grad_() for n in names if st[n] is not None}

    def wide(n):
        t = leaf[n]
        return t[:, None, :] if t.dim() == 2 else t

    u = leaf["x"] + wide("scale") * leaf["residual"] if case["residual"] else leaf["x"] * 1.0
    act = leaf["gate"] / (1.0 + torch.exp(-leaf["gate"])) if case["gate"] != "none" else 1.0
    s = u * act if case["gate"] == "before" else u
    m = 0.0 if case["rms"] else s.sum(-1, keepdim=True) / case["width"]
    y = (s - m) / torch.sqrt(((s - m) ** 2).sum(-1, keepdim=True) / case["width"] + EPS) * wide("weight")
    if case["bias"]:
        y = y + wide("bias")
    if case["gate"] == "after":
        y = y * act
    out = [y.detach()] + ([u.detach()] if case["residual"] else [])
    if case["op"] == "norm":
        return out
    loss = (y * st["dy"].double()).sum()
    if case["residual"]:
        loss = loss + (u * st["dtotal"].double()).sum()
    order = ["x", "weight", "bias", "gate", "residual", "scale"]
    return out + list(torch.autograd.grad(loss, [leaf[n] for n in order if n in leaf]))


def _exact_conv(case, st):
    """Tap by tap over whole sequences, gradients by differentiating it."""
    B, H, T, d, W = (case[x] for x in "BHTdW")
    state = torch.zeros((B, H, W - 1, d), device=st["x"].device) if st["state"] is None else st["state"]
    leaf = [t.double().requires_grad_() for t in (st["x"], st["weight"], st["bias"], state)]
    x, w, b, s = leaf
    lens = [T] * B if st["lens"] is None else [int(n) for n in st["lens"].tolist()]
    ys, ends = [], []
    for row in range(B):
        n = lens[row]
        r = torch.cat([s[row], x[row, :, :n]], 1)                     # [H, W - 1 + n, d]
        a = b[:, None, :].expand(H, n, d)
        for tap in range(W):
            a = a + w[:, None, :, tap] * r[:, tap:tap + n]
        y = a / (1.0 + torch.exp(-a)) if case["silu"] else a
        ys.append(torch.cat([y, torch.zeros((H, T - n, d), dtype=y.dtype, device=y.device)], 1))
        ends.append(r[:, n:n + W - 1])
    y, end = torch.stack(ys), torch.stack(ends)
    out = [y.detach(), end.detach()]
    if case["op"] == "conv":
        return out
    on, _ = _valid(case, st, y.device)
    loss = (y * torch.where(on, st["dy"].double(), 0.0)).sum()
    if st["dstate"] is not None:
        loss = loss + (end * st["dstate"].double()).sum()
    grads = torch.autograd.grad(loss, leaf, allow_unused=True)
    return out + list(grads if case["state"] else grads[:3])


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "norm_train"):
        return _exact_norm(case, st)
    if op == "conv_step":
        r = torch.cat([st["state"].double(), st["x"].double()[:, :, None]], 2)
        a = st["bias"].double() + sum(r[:, :, t] * st["weight"].double()[:, :, t] for t in range(case["W"]))
        return [a / (1.0 + torch.exp(-a)) if case["silu"] else a, r[:, :, 1:]]
    if op.startswith("conv"):
        return _exact_conv(case, st)
    B, H, G, d = (case[x] for x in "BHGd")
    N, T = B * H, case.get("T", 1)
    head = torch.arange(N, device=st["q"].device)
    group = head // H * G + head % H // (H // G)                      # of each chain, among B * G
    q, k = (st[x].view(B * G, T, d).transpose(0, 1).contiguous() for x in "qk")
    v = st["v"].view(N, T, d).transpose(0, 1).contiguous()
    raw = st["dt"].double().view(N, T).t().contiguous()
    if case["softplus"]:
        z = raw + st["dt_bias"].double().repeat(B)
        raw = torch.where(z > 30.0, z, torch.log(1.0 + torch.exp(torch.clamp(z, max=30.0))))
    rate = st["log_decay"].double().repeat(B)
    skip = torch.zeros(H) if st["skip"] is None else st["skip"]
    skip = skip.to(rate).repeat(B).view(N, 1)
    start = st.get("S") if op == "select_step" else st["S0"]
    S = (torch.zeros((N, d, d), dtype=torch.float64, device=rate.device) if start is None
         else start.double().view(N, d, d).clone())
    lens = st.get("lens")
    live = torch.ones((T, N), dtype=torch.bool) if lens is None else (
        torch.arange(T).view(T, 1) < lens.cpu().long().repeat_interleave(H).view(1, N))
    live = live.to(rate.device)
    o = torch.zeros((T, N, d), dtype=torch.float64, device=rate.device)
    for t in range(T):
        on = live[t].view(N, 1, 1)
        vt = v[t].double()
        S.mul_(torch.where(on, torch.exp(rate * raw[t]).view(N, 1, 1), 1.0))
        S.baddbmm_((k[t].double()[group] * raw[t].view(N, 1)).view(N, d, 1) * on, vt.view(N, 1, d))
        o[t] = torch.bmm(q[t].double()[group].view(N, 1, d), S)[:, 0] * st["scale"] + skip * vt
    if op == "select_step":
        return [o[0].view(B, H, d), S.view(B, H, d, d)]
    o = (o * live[..., None]).transpose(0, 1).reshape(B, H, T, d)
    return [o, S.view(B, H, d, d)]


def work(case):
    """Bytes: every input read once, every output written once (rows before each sequence's end).
    Operations: the recurrence's multiply-adds (a write and a read of the state a token), a
    convolution's taps, and about ten an element of a norm."""
    op = case["op"]
    e = 2 if case["dtype"] == "bf16" else 4
    if op in ("norm", "norm_train"):
        n, par = case["rows"] * case["width"], case["H"] * case["width"] * 4
        res, gate = int(case["residual"]), int(case["gate"] != "none")
        b = (2 + 2 * res + gate) * n * e + (1 + int(case["bias"]) + res) * par
        f = (6 + 2 * res + 5 * gate) * n
        if op == "norm_train":   # what the forward pass has read, and its outputs, are not read again
            b += (2 + 2 * res + gate) * n * e + (1 + int(case["bias"]) + res) * par
            f *= 3
        return {"bytes": b, "flops": f}
    B, H, d = case["B"], case["H"], case["d"]
    if op.startswith("conv"):
        W = case["W"]
        rows, par = B * H * (W - 1) * d * e, H * d * (W + 1) * 4
        if op == "conv_step":
            return {"bytes": 2 * B * H * d * e + 2 * rows + par, "flops": (2 * W + 5) * B * H * d}
        n = H * d * (sum(_lens(case)) if case["ragged"] else B * case["T"])
        s = int(case["state"])
        if op == "conv":
            return {"bytes": 2 * n * e + (1 + s) * rows + par, "flops": (2 * W + 5) * n}
        return {"bytes": 4 * n * e + (1 + 3 * s) * rows + 2 * par, "flops": (6 * W + 15) * n}
    G, state = case["G"], B * H * d * d * 4
    if op == "select_step":
        return {"bytes": 2 * state + B * (2 * H + 2 * G) * d * e + B * H * e, "flops": 5 * B * H * d * d}
    tok = sum(_lens(case)) if case["ragged"] else B * case["T"]
    return {"bytes": tok * (2 * (H + G) * d + H) * e + (1 + int(case["s0"])) * state, "flops": 4 * tok * H * d * d}
