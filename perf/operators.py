"""Measured cases of the gated delta rule and of layer norm.

The gated delta rule is the dense-key form of this package's write/read: every row of a Dk x Dv state
decays by one factor a token, the token's key retrieves, its value is delta-written, its query reads:

    d = exp(g) S;   r = v - d^T k;   S = d + beta k r^T;   o = scale S^T q

Layer norm stands before such a layer (rows of the model's width) and on its readings (rows of one
head's width). `run` makes one pass in the package's kernels where `own` is true, and in elementary
32-bit torch operations where it is false. `exact` is the definition, token by token, in 64 bits.
"""
import math

import torch

own = False

CHUNK = 64
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one user's next token in a layer of 16 heads: latency only
        dict(name="delta step, 1 sequence", op="delta", B=1, T=1, Hk=16, H=16, Dk=128, Dv=128, dtype="bf16", ragged=False),
        # a serving batch's next token, two value heads for each key head: the states' bandwidth
        dict(name="delta step, 256 sequences", op="delta", B=256, T=1, Hk=16, H=32, Dk=128, Dv=128, dtype="bf16", ragged=False),
        # a few short, unequal prompts of a small float32 model
        dict(name="delta short prompts, float32", op="delta", B=3, T=75, Hk=2, H=6, Dk=64, Dv=96, dtype="f32", ragged=True),
        # one long prompt: few heads, a long chain of chunks
        dict(name="delta long prompt", op="delta", B=1, T=16384, Hk=16, H=32, Dk=128, Dv=128, dtype="bf16", ragged=False),
        # a batch of unequal prompts: throughput
        dict(name="delta prompt batch", op="delta", B=8, T=4096, Hk=16, H=32, Dk=128, Dv=128, dtype="bf16", ragged=True),
        # a training step's forward and backward through the layer
        dict(name="delta train", op="delta_train", B=2, T=4096, Hk=16, H=32, Dk=128, Dv=128, dtype="bf16", ragged=False),
        # a small float32 model's training step on unequal sequences of odd length
        dict(name="delta train, float32", op="delta_train", B=2, T=1003, Hk=2, H=4, Dk=64, Dv=64, dtype="f32", ragged=True),
        # the layer's input norm for a decode batch: latency only
        dict(name="norm, 32 tokens", op="norm", rows=32, N=2048, dtype="bf16", bias=True),
        # the norm of every head's readings of a prompt batch: many short rows
        dict(name="norm, heads", op="norm", rows=1048576, N=128, dtype="bf16", bias=False),
        # the input norm of a training step, forward and backward
        dict(name="norm train, wide", op="norm_train", rows=32768, N=4096, dtype="bf16", bias=True),
        # the readings' norm of a training step, forward and backward
        dict(name="norm train, heads", op="norm_train", rows=262144, N=128, dtype="bf16", bias=False),
        # a width that no vector load divides
        dict(name="norm train, odd, float32", op="norm_train", rows=5003, N=1007, dtype="f32", bias=True),
    ]


def draw(rng):
    def span(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    dtype = rng.choice(["bf16", "bf16", "f32"])
    kind = rng.choice(["step", "delta", "delta", "train", "norm", "norm_train"])
    if kind in ("norm", "norm_train"):
        n = span(64, 8192)
        if rng.random() < 0.6:
            n = max(64, n // 8 * 8)
        return dict(op=kind, rows=span(1, max(2, (64 << 20) // n)), N=n, dtype=dtype, bias=rng.random() < 0.5)
    group = rng.choice([1, 1, 2, 4])
    hk = span(1, 32 // group)
    dk, dv = rng.choice([32, 64, 96, 128, 128]), rng.choice([32, 64, 128, 128, 192])
    h = hk * group
    if kind == "step":
        return dict(op="delta", B=span(1, max(1, 6144 // h)), T=rng.choice([1, 1, 1, 2, 4]), Hk=hk, H=h, Dk=dk, Dv=dv, dtype=dtype, ragged=False)
    if kind == "delta":
        t = span(5, 16384)
        most = 524288 if dtype == "bf16" else 131072
        return dict(op="delta", B=span(1, max(1, min(16, most // (h * t)))), T=t, Hk=hk, H=h, Dk=dk, Dv=dv, dtype=dtype, ragged=rng.random() < 0.5)
    t = span(5, 4096)
    most = 131072 if dtype == "bf16" else 32768
    return dict(op="delta_train", B=span(1, max(1, min(8, most // (h * t)))), T=t, Hk=hk, H=h, Dk=dk, Dv=dv, dtype=dtype, ragged=rng.random() < 0.5)


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    if case["op"] in ("norm", "norm_train"):
        rows, n = case["rows"], case["N"]
        # activations with a mean and a few wide columns, as a residual stream has
        wide = 1 + 4 * (torch.rand(n, device="cuda", generator=gen) < 0.01)
        s = dict(case=case, x=(normal(rows, n) * wide + 0.3 * normal(n)).to(dt), weight=1 + 0.1 * normal(n),
                 bias=0.1 * normal(n) if case["bias"] else None)
        if case["op"] == "norm_train":
            s["grad"] = normal(rows, n).to(dt)
        return s
    B, T, Hk, H, Dk, Dv = (case[x] for x in ("B", "T", "Hk", "H", "Dk", "Dv"))
    # queries and keys as such a layer makes them: an activation, then unit length
    q, k = (torch.nn.functional.normalize(torch.nn.functional.silu(normal(B, T, Hk, Dk)), dim=-1).to(dt) for _ in range(2))
    s = dict(case=case, q=q, k=k, v=normal(B, T, H, Dv).to(dt), g=-0.1 * torch.nn.functional.softplus(normal(B, T, H)),
             beta=torch.sigmoid(normal(B, T, H)), state=0.1 * normal(B, H, Dk, Dv), scale=Dk ** -0.5, valid=None)
    if case["ragged"]:
        s["valid"] = torch.randint(T // 2, T + 1, (B,), device="cuda", generator=gen, dtype=torch.int32)
    if case["op"] == "delta_train":
        s["grad"] = normal(B, T, H, Dv).to(dt)
        s["grad_state"] = 0.1 * normal(B, H, Dk, Dv)
    return s


def run(s):
    op = s["case"]["op"]
    if op == "norm":
        if own:
            import sparse_addressed_delta_gb300 as sdm
            return sdm.layer_norm(s["x"], s["weight"], s["bias"])
        return _norm(s["x"].float(), s["weight"], s["bias"])[0].to(s["x"].dtype)
    if op == "norm_train":
        if own:
            import sparse_addressed_delta_gb300 as sdm
            y, stats = sdm.layer_norm_save(s["x"], s["weight"], s["bias"])
            return {"y": y, **sdm.layer_norm_backward(s["grad"], s["x"], s["weight"], stats, bias=s["bias"] is not None)}
        return _norm_train(s)
    if op == "delta":
        args = (s["q"], s["k"], s["v"], s["g"], s["beta"])
        if own:
            import sparse_addressed_delta_gb300 as sdm
            o = sdm.gated_delta(s["state"], *args, s["valid"], scale=s["scale"])
        elif s["case"]["T"] == 1 and s["valid"] is None:
            o = _step(s["state"], *args, s["scale"])
        else:
            o = _chunks(s["state"], *args, s["valid"], s["scale"])[0]
        return {"readings": o, "state": s["state"]}
    if own:
        import sparse_addressed_delta_gb300 as sdm
        state = s["state"].clone()
        args = (s["q"], s["k"], s["v"], s["g"], s["beta"], s["valid"])
        o, saved = sdm.gated_delta_save(state, *args, scale=s["scale"])
        return {"readings": o, "state": state,
                **sdm.gated_delta_backward(*args, saved, s["grad"], grad_state=s["grad_state"], scale=s["scale"])}
    return _delta_train(s)


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("norm", "norm_train"):
        cells, n = case["rows"] * case["N"], case["N"]
        if case["op"] == "norm":  # x read, y written
            return {"bytes": 2 * es * cells + 8 * n, "flops": 7 * cells}
        # x read, y written; the gradient read, x's gradient written (x is read again: one pass cannot keep it)
        return {"bytes": 5 * es * cells + 16 * n, "flops": 20 * cells}
    B, T, Hk, H, Dk, Dv = (case[x] for x in ("B", "T", "Hk", "H", "Dk", "Dv"))
    tok, st = B * T, B * H * Dk * Dv
    qk, v, gates = 2 * tok * Hk * Dk * es, tok * H * Dv * es, 2 * tok * H * 4
    if case["op"] == "delta":  # retrieve, write and read: a product of Dk x Dv each
        return {"bytes": qk + 2 * v + gates + 8 * st, "flops": 6 * tok * H * Dk * Dv}
    # forward, then: inputs and the readings' gradient read, every gradient written
    return {"bytes": (qk + 2 * v + gates + 8 * st) + (2 * qk + 3 * v + 2 * gates + 8 * st), "flops": 18 * tok * H * Dk * Dv}


# ---- the plain forms: 32 bits, rounded once at the end ----------------------------------------

def _norm(x, weight, bias, eps=1e-5):
    mean = x.mean(-1, keepdim=True)
    xc = x - mean
    rstd = (xc.square().mean(-1, keepdim=True) + eps).rsqrt()
    xhat = xc * rstd
    y = xhat * weight
    return y if bias is None else y + bias, xhat, rstd


def _norm_train(s):
    y, xhat, rstd = _norm(s["x"].float(), s["weight"], s["bias"])
    dy = s["grad"].float()
    w = dy * s["weight"]
    dx = rstd * (w - w.mean(-1, keepdim=True) - xhat * (w * xhat).mean(-1, keepdim=True))
    out = {"y": y.to(s["x"].dtype), "grad_x": dx.to(s["x"].dtype), "grad_weight": (dy * xhat).sum(0)}
    if s["bias"] is not None:
        out["grad_bias"] = dy.sum(0)
    return out


def _step(state, q, k, v, g, beta, scale):
    rep = state.shape[1] // q.shape[2]
    q, k = (x[:, 0].float().repeat_interleave(rep, 1) for x in (q, k))
    d = state * g[:, 0, :, None, None].exp()
    u = beta[:, 0, :, None] * (v[:, 0].float() - (k[..., None] * d).sum(-2))
    state.copy_(d + k[..., None] * u[..., None, :])
    return (scale * (q[..., None] * state).sum(-2)).to(v.dtype)[:, None]


def _split(x, rep, live, pad):
    """[B, T, h, ...] -> [B, H, chunks, CHUNK, ...] in 32 bits, zero where no token is."""
    x = x.float().transpose(1, 2)
    x = torch.where(live.view(live.shape[0], 1, -1, *[1] * (x.dim() - 3)), x, 0.0)
    x = torch.nn.functional.pad(x, [0, 0] * (x.dim() - 3) + [0, pad]).repeat_interleave(rep, 1)
    return x.reshape(*x.shape[:2], -1, CHUNK, *x.shape[3:])


def _join(x, T, dtype):
    return x.flatten(2, 3)[:, :, :T].transpose(1, 2).to(dtype)


def _local(q, k, v, g, beta, valid, scale):
    """What each chunk has before any state: its rows, decays, products and inverse."""
    B, T, H = g.shape
    pad, rep = -T % CHUNK, H // q.shape[2]
    live = torch.arange(T, device=q.device)[None] < (valid[:, None] if valid is not None else T)
    live = live.expand(B, T)
    c = {"q": _split(q, rep, live, pad) * scale, "k": _split(k, rep, live, pad), "v": _split(v, 1, live, pad),
         "beta": _split(beta, 1, live, pad)[..., None], "live": live}
    run = _split(g, 1, live, pad).cumsum(-1)
    lower = torch.ones(CHUNK, CHUNK, device=q.device).tril() > 0
    c["pair"] = torch.where(lower, run[..., :, None] - run[..., None, :], -torch.inf).exp()
    c["from"], c["to"] = run.exp()[..., None], (run[..., -1:] - run).exp()[..., None]
    c["whole"] = run[..., -1].exp()[..., None, None]
    c["kk"] = (c["k"] @ c["k"].mT) * c["pair"].tril(-1)
    c["qk"] = (c["q"] @ c["k"].mT) * c["pair"]
    m = c["beta"] * c["kk"]
    x = torch.eye(CHUNK, device=q.device).expand_as(m).clone()
    for t in range(1, CHUNK):  # rows of the inverse of I + m, from the rows above
        x[..., t, :t] = -(m[..., t, None, :t] @ x[..., :t, :t])[..., 0, :]
    c["x"] = x
    return c


def _chunks(state, q, k, v, g, beta, valid, scale, keep=False):
    c = _local(q, k, v, g, beta, valid, scale)
    S, starts, outs, us = state, [], [], []
    for n in range(c["k"].shape[2]):
        starts.append(S)
        w = c["v"][:, :, n] - c["from"][:, :, n] * (c["k"][:, :, n] @ S)
        u = c["x"][:, :, n] @ (c["beta"][:, :, n] * w)
        outs.append(c["from"][:, :, n] * (c["q"][:, :, n] @ S) + c["qk"][:, :, n] @ u)
        S = c["whole"][:, :, n] * S + (c["to"][:, :, n] * c["k"][:, :, n]).mT @ u
        us.append(u)
    o = _join(torch.stack(outs, 2), q.shape[1], v.dtype)
    if keep:
        return o, S, c, torch.stack(starts, 2), torch.stack(us, 2)
    state.copy_(S)
    return o, S


def _delta_train(s):
    q, k, v, g, beta, valid, scale = (s[x] for x in ("q", "k", "v", "g", "beta", "valid", "scale"))
    o, state, c, starts, u = _chunks(s["state"], q, k, v, g, beta, valid, scale, keep=True)
    B, T, H = g.shape
    rep = H // q.shape[2]
    do = _split(s["grad"], 1, c["live"], -T % CHUNK)
    dS, ends, dws = s["grad_state"], [], []
    qk_do = c["qk"].mT @ do
    for n in reversed(range(c["k"].shape[2])):
        ends.append(dS)
        du = qk_do[:, :, n] + c["to"][:, :, n] * (c["k"][:, :, n] @ dS)
        dw = c["x"][:, :, n].mT @ du
        dws.append(dw)
        dS = c["whole"][:, :, n] * dS + (c["from"][:, :, n] * c["q"][:, :, n]).mT @ do[:, :, n] \
            - c["k"][:, :, n].mT @ (c["beta"][:, :, n] * c["from"][:, :, n] * dw)
    ends, dw = torch.stack(ends[::-1], 2), torch.stack(dws[::-1], 2)
    lost = c["from"] * (c["k"] @ starts)  # what the keys retrieve from the chunk's start
    dm = dw @ u.mT
    dkk = -(c["beta"] * dm).tril(-1)
    dqk = (do @ u.mT).tril()
    a, p = dkk * c["pair"], dqk * c["pair"]
    dq_start = c["from"] * (do @ starts.mT)
    dk_start = -c["beta"] * c["from"] * (dw @ starts.mT)
    dk_end = c["to"] * (u @ ends.mT)
    dq = scale * (p @ c["k"] + dq_start)
    dk = p.mT @ c["q"] + (a + a.mT) @ c["k"] + dk_start + dk_end
    z = dkk * c["kk"] + dqk * c["qk"]
    end = (c["k"] * dk_end).sum(-1)
    drun = z.sum(-1) - z.sum(-2) + (c["q"] * dq_start).sum(-1) + (c["k"] * dk_start).sum(-1) - end
    drun[..., -1] += end.sum(-1) + (c["whole"] * starts * ends).sum((-1, -2))
    dg = drun.flip(-1).cumsum(-1).flip(-1)
    dbeta = (dw * (c["v"] - lost)).sum(-1) - (dm * c["kk"]).sum(-1)
    live = c["live"][..., None]

    def shared(x, like):  # heads that share a key head add up
        x = x.unflatten(1, (-1, rep)).sum(2)
        return torch.where(live[..., None], _join(x, T, like.dtype), 0)

    return {"readings": o, "state": state, "grad_q": shared(dq, q), "grad_k": shared(dk, k),
            "grad_v": torch.where(live[..., None], _join(c["beta"] * dw, T, v.dtype), 0),
            "grad_log_decay": torch.where(live, _join(dg, T, torch.float32), 0),
            "grad_beta": torch.where(live, _join(dbeta, T, torch.float32), 0), "grad_state": dS}


# ---- the definitions in 64 bits, token by token -------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm", "norm_train"):
        return _exact_norm(s)
    if case["B"] * case["T"] * case["H"] * case["Dk"] * case["Dv"] > 1.8e10:
        return None
    return _exact_delta(s)


def _exact_norm(s):
    x, w = s["x"].double(), s["weight"].double()
    n = x.shape[1]
    mu = x.sum(1) / n
    sd = (((x - mu[:, None]) ** 2).sum(1) / n + 1e-5).sqrt()
    z = (x - mu[:, None]) / sd[:, None]
    y = z * w + (s["bias"].double() if s["bias"] is not None else 0.0)
    if s["case"]["op"] == "norm":
        return y
    dy = s["grad"].double()
    out = {"y": y, "grad_weight": torch.einsum("rn,rn->n", dy, z)}
    if s["bias"] is not None:
        out["grad_bias"] = dy.sum(0)
    dz = dy * w
    out["grad_x"] = (dz - (dz.sum(1) / n)[:, None] - z * (torch.einsum("rn,rn->r", dz, z) / n)[:, None]) / sd[:, None]
    return out


def _exact_delta(s):
    case = s["case"]
    B, T, H, Hk = case["B"], case["T"], case["H"], case["Hk"]
    owner = torch.arange(H, device="cuda") // (H // Hk)
    q, k, v, beta = s["q"].double()[:, :, owner], s["k"].double()[:, :, owner], s["v"].double(), s["beta"].double()
    fade = s["g"].double().exp()
    valid = s["valid"] if s["valid"] is not None else torch.full((B,), T, device="cuda", dtype=torch.int32)
    on = (torch.arange(T, device="cuda")[None] < valid[:, None]).double()

    def token(S, t):
        """One token: (state after it, decayed state, what the value lacks)."""
        d = fade[:, t, :, None, None] * S
        r = v[:, t] - (k[:, t, :, None] @ d)[:, :, 0]
        after = d + (beta[:, t, :, None] * k[:, t])[..., None] * r[:, :, None]
        m = on[:, t, None, None, None]
        return m * after + (1 - m) * S, d, r

    S, marks = s["state"].double(), []
    o = torch.zeros_like(v)
    for t in range(T):
        if t % 64 == 0:
            marks.append(S)
        S = token(S, t)[0]
        o[:, t] = on[:, t, None, None] * s["scale"] * (q[:, t, :, None] @ S)[:, :, 0]
    out = {"readings": o, "state": S}
    if case["op"] == "delta":
        return out
    dS, do = s["grad_state"].double(), s["grad"].double()
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, dbeta = torch.zeros_like(beta), torch.zeros_like(beta)
    for first in reversed(range(0, T, 64)):
        S, kept = marks.pop(), []
        for t in range(first, min(T, first + 64)):
            after, d, r = token(S, t)
            kept.append((after, d, r))
            S = after
        for t in reversed(range(first, min(T, first + 64))):
            after, d, r = kept.pop()
            m1, m2, m3 = on[:, t, None], on[:, t, None, None], on[:, t, None, None, None]
            got = do[:, t] * s["scale"]
            dq[:, t] = m2 * (after @ got[..., None])[..., 0]
            dA = dS + q[:, t, :, :, None] * got[:, :, None]
            b = beta[:, t, :, None]
            kd = (k[:, t, :, None] @ dA)[:, :, 0]
            dbeta[:, t] = m1 * (kd * r).sum(-1)
            dr = b * kd
            dv[:, t] = m2 * dr
            dk[:, t] = m2 * (b * (dA @ r[..., None])[..., 0] - (d @ dr[..., None])[..., 0])
            dD = dA - k[:, t, :, :, None] * dr[:, :, None]
            dg[:, t] = m1 * (dD * d).sum((-1, -2))
            dS = m3 * fade[:, t, :, None, None] * dD + (1 - m3) * dS
    add = torch.zeros(Hk, H, device="cuda", dtype=torch.float64)
    add[owner, torch.arange(H, device="cuda")] = 1
    out |= {"grad_q": torch.einsum("gh,bthd->btgd", add, dq), "grad_k": torch.einsum("gh,bthd->btgd", add, dk), "grad_v": dv,
            "grad_log_decay": dg, "grad_beta": dbeta, "grad_state": dS}
    return out
