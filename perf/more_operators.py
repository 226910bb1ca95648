"""Measured cases of linear attention with a decay for each head and of group norm with an activation.

Linear attention is the write/read without the delta: a head's Dk x Dv state decays by the head's own factor
at every token, the token's key writes its value, its query reads:

    S = exp(g) S + k v^T;   o = scale S^T q            (g: one number a head)

Group norm stands on such readings (a token's heads as groups of channels) and on maps whose positions share
their statistics; channels are the last dimension, and an activation may follow:

    z = (x - mean) rstd weight + bias;   y = z, or z / (1 + exp(-z))

`run` makes one pass in the package's kernels where `own` is true, and in elementary 32-bit torch operations
where it is false. `exact` is the definition in 64 bits, linear attention token by token.
"""
import math

import torch

own = False

CHUNK = 64
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one user's next token in a layer of 16 heads: latency only
        dict(name="linear step 1 sequence", op="linear", B=1, T=1, Hk=16, H=16, Dk=128, Dv=128, dtype="bf16", ragged=False),
        # a serving batch's next token, two value heads for each key head: the states' bandwidth
        dict(name="linear step 256 sequences", op="linear", B=256, T=1, Hk=16, H=32, Dk=128, Dv=128, dtype="bf16", ragged=False),
        # a few short, unequal prompts of a small float32 model
        dict(name="linear short prompts float32", op="linear", B=3, T=75, Hk=2, H=6, Dk=64, Dv=96, dtype="f32", ragged=True),
        # one long prompt: few heads, many chunks
        dict(name="linear long prompt", op="linear", B=1, T=16384, Hk=16, H=32, Dk=128, Dv=128, dtype="bf16", ragged=False),
        # a batch of unequal prompts with values twice as wide as the keys: throughput
        dict(name="linear prompt batch", op="linear", B=8, T=4096, Hk=16, H=16, Dk=128, Dv=256, dtype="bf16", ragged=True),
        # a training step's forward and backward, the decays learned too
        dict(name="linear train", op="linear_train", B=2, T=4096, Hk=16, H=32, Dk=128, Dv=128, dtype="bf16", ragged=False, decay=True),
        # a small float32 model's training step on unequal sequences of odd length, the decays fixed
        dict(name="linear train float32", op="linear_train", B=2, T=1003, Hk=2, H=4, Dk=64, Dv=64, dtype="f32", ragged=True, decay=False),
        # the readings' norm for a decode batch: latency only
        dict(name="group norm 32 tokens", op="group", N=32, L=1, C=2048, G=16, dtype="bf16", act="silu"),
        # the readings' norm of a prompt batch, every head a group: many rows
        dict(name="group norm heads", op="group", N=32768, L=1, C=4096, G=32, dtype="bf16", act="silu"),
        # maps whose positions share their statistics
        dict(name="group norm maps", op="group", N=8, L=4096, C=512, G=32, dtype="bf16", act="silu"),
        # the readings' norm of a training step, forward and backward
        dict(name="group norm train heads", op="group_train", N=16384, L=1, C=4096, G=32, dtype="bf16", act="silu"),
        # a small float32 model's maps, groups of nine channels, no activation
        dict(name="group norm train odd maps float32", op="group_train", N=3, L=1551, C=180, G=20, dtype="f32", act=None),
    ]


def draw(rng):
    def span(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    dtype = rng.choice(["bf16", "bf16", "f32"])
    kind = rng.choice(["step", "linear", "linear", "train", "group", "group", "group_train"])
    if kind in ("group", "group_train"):
        groups = rng.choice([1, 4, 8, 16, 20, 32, 32])
        channels = groups * span(2, max(3, 4096 // groups))
        if rng.random() < 0.6:
            channels = max(8 * groups, channels // (8 * groups) * 8 * groups)
        cells = (64 << 20) if kind == "group" else (32 << 20)
        length = 1 if rng.random() < 0.4 else span(2, 16384)
        length = max(1, min(length, cells // channels))
        return dict(op=kind, N=span(1, max(2, cells // (channels * length))), L=length, C=channels, G=groups, dtype=dtype,
                    act=rng.choice(["silu", "silu", None]))
    group = rng.choice([1, 1, 2, 4])
    hk = span(1, 32 // group)
    dk, dv = rng.choice([32, 64, 96, 128, 128]), rng.choice([32, 64, 128, 128, 192, 256])
    h = hk * group
    if kind == "step":
        return dict(op="linear", B=span(1, max(1, 4096 // h)), T=rng.choice([1, 1, 1, 2, 4]), Hk=hk, H=h, Dk=dk, Dv=dv, dtype=dtype, ragged=False)
    if kind == "linear":
        t = span(5, 16384)
        most = 524288 if dtype == "bf16" else 131072
        return dict(op="linear", B=span(1, max(1, min(16, most // (h * t)))), T=t, Hk=hk, H=h, Dk=dk, Dv=dv, dtype=dtype, ragged=rng.random() < 0.5)
    t = span(5, 4096)
    most = 131072 if dtype == "bf16" else 32768
    return dict(op="linear_train", B=span(1, max(1, min(8, most // (h * t)))), T=t, Hk=hk, H=h, Dk=dk, Dv=dv, dtype=dtype,
                ragged=rng.random() < 0.5, decay=rng.random() < 0.5)


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    if case["op"] in ("group", "group_train"):
        N, L, C = case["N"], case["L"], case["C"]
        # activations with a mean and a few wide channels, as a residual stream has
        wide = 1 + 4 * (torch.rand(C, device="cuda", generator=gen) < 0.01)
        s = dict(case=case, x=(normal(N, L, C) * wide + 0.3 * normal(C)).to(dt), weight=1 + 0.1 * normal(C), bias=0.1 * normal(C))
        if case["op"] == "group_train":
            s["grad"] = normal(N, L, C).to(dt)
        return s
    B, T, Hk, H, Dk, Dv = (case[x] for x in ("B", "T", "Hk", "H", "Dk", "Dv"))
    # queries and keys as such a layer makes them: an activation, then unit length
    q, k = (torch.nn.functional.normalize(torch.nn.functional.silu(normal(B, T, Hk, Dk)), dim=-1).to(dt) for _ in range(2))
    # a head forgets a quarter to a five-hundredth of its state at a token, from the first head to the last
    forget = torch.exp(torch.linspace(math.log(1 / 4), math.log(1 / 512), H, device="cuda") + 0.05 * normal(H))
    s = dict(case=case, q=q, k=k, v=normal(B, T, H, Dv).to(dt), g=torch.log1p(-forget), state=0.1 * normal(B, H, Dk, Dv),
             scale=Dk ** -0.5, valid=None)
    if case["ragged"]:
        s["valid"] = torch.randint(T // 2, T + 1, (B,), device="cuda", generator=gen, dtype=torch.int32)
    if case["op"] == "linear_train":
        s["grad"] = normal(B, T, H, Dv).to(dt)
        s["grad_state"] = 0.1 * normal(B, H, Dk, Dv)
    return s


def run(s):
    case = s["case"]
    op = case["op"]
    if op == "group":
        if own:
            import sparse_addressed_delta_gb300 as sdm
            return sdm.group_norm(s["x"], case["G"], s["weight"], s["bias"], activation=case["act"])
        return _group(s)[0]
    if op == "group_train":
        if own:
            import sparse_addressed_delta_gb300 as sdm
            y, stats = sdm.group_norm_save(s["x"], case["G"], s["weight"], s["bias"], activation=case["act"])
            return {"y": y, **sdm.group_norm_backward(s["grad"], s["x"], case["G"], s["weight"], s["bias"], stats, activation=case["act"])}
        return _group_train(s)
    args = (s["q"], s["k"], s["v"], s["g"])
    if op == "linear":
        if own:
            import sparse_addressed_delta_gb300 as sdm
            o = sdm.linear_attention(s["state"], *args, s["valid"], scale=s["scale"])
        elif case["T"] == 1 and s["valid"] is None:
            o = _step(s["state"], *args, s["scale"])
        else:
            o, state = _chunks(s["state"], *args, s["valid"], s["scale"])
            s["state"].copy_(state)
        return {"readings": o, "state": s["state"]}
    if own:
        import sparse_addressed_delta_gb300 as sdm
        state = s["state"].clone()
        o, saved = sdm.linear_attention_save(state, *args, s["valid"], scale=s["scale"])
        return {"readings": o, "state": state,
                **sdm.linear_attention_backward(*args, s["valid"], saved, s["grad"], grad_state=s["grad_state"], scale=s["scale"],
                                                decay=case["decay"])}
    return _linear_train(s)


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("group", "group_train"):
        cells, c = case["N"] * case["L"] * case["C"], case["C"]
        if case["op"] == "group":  # x read, y written
            return {"bytes": 2 * es * cells + 8 * c, "flops": 10 * cells}
        # x read, y written; x and the gradient read, x's gradient written (a forward cannot keep x on the chip)
        return {"bytes": 5 * es * cells + 16 * c, "flops": 30 * cells}
    B, T, Hk, H, Dk, Dv = (case[x] for x in ("B", "T", "Hk", "H", "Dk", "Dv"))
    tok, st = B * T, B * H * Dk * Dv
    qk, v = 2 * tok * Hk * Dk * es, tok * H * Dv * es
    if case["op"] == "linear":  # write and read: a product of Dk x Dv each
        return {"bytes": qk + 2 * v + 8 * st, "flops": 4 * tok * H * Dk * Dv}
    # forward, then: inputs and the readings' gradient read, every gradient written
    return {"bytes": (qk + 2 * v + 8 * st) + (2 * qk + 3 * v + 8 * st), "flops": 12 * tok * H * Dk * Dv}


# ---- the plain forms: 32 bits, rounded once at the end ----------------------------------------

def _norm(s):
    """(xhat, rstd) as [N, L, G, C / G] and [N, 1, G, 1]."""
    x = s["x"].float().unflatten(-1, (s["case"]["G"], -1))
    xc = x - x.mean((1, 3), keepdim=True)
    rstd = (xc.square().mean((1, 3), keepdim=True) + 1e-5).rsqrt()
    return xc * rstd, rstd


def _group(s):
    xhat, rstd = _norm(s)
    z = xhat.flatten(2) * s["weight"] + s["bias"]
    y = z / (1 + torch.exp(-z)) if s["case"]["act"] else z
    return y.to(s["x"].dtype), xhat, rstd, z


def _group_train(s):
    y, xhat, rstd, z = _group(s)
    dz = s["grad"].float()
    if s["case"]["act"]:
        p = 1 / (1 + torch.exp(-z))
        dz = dz * p * (1 + z * (1 - p))
    w = (dz * s["weight"]).unflatten(-1, (s["case"]["G"], -1))
    dx = rstd * (w - w.mean((1, 3), keepdim=True) - xhat * (w * xhat).mean((1, 3), keepdim=True))
    return {"y": y, "grad_x": dx.flatten(2).to(y.dtype), "grad_weight": (dz * xhat.flatten(2)).sum((0, 1)), "grad_bias": dz.sum((0, 1))}


def _step(state, q, k, v, g, scale):
    rep = state.shape[1] // q.shape[2]
    q, k = (x[:, 0].float().repeat_interleave(rep, 1) for x in (q, k))
    state.copy_(state * g[None, :, None, None].exp() + k[..., None] * v[:, 0].float()[..., None, :])
    return (scale * (q[..., None] * state).sum(-2)).to(v.dtype)[:, None]


def _split(x, rep, live, pad):
    """[B, T, h, D] -> [B, H, chunks, CHUNK, D] in 32 bits, zero where no token is."""
    x = torch.where(live[:, None, :, None], x.float().transpose(1, 2), 0.0)
    x = torch.nn.functional.pad(x, [0, 0, 0, pad]).repeat_interleave(rep, 1)
    return x.reshape(*x.shape[:2], -1, CHUNK, x.shape[3])


def _join(x, T):
    return x.flatten(2, 3)[:, :, :T].transpose(1, 2)


def _chunks(state, q, k, v, g, valid, scale, keep=False):
    (B, T, H), rep, pad = v.shape[:3], v.shape[2] // q.shape[2], -v.shape[1] % CHUNK
    live = (torch.arange(T, device=q.device)[None] < (valid[:, None] if valid is not None else T)).expand(B, T)
    q, k, v32 = _split(q, rep, live, pad) * scale, _split(k, rep, live, pad), _split(v, 1, live, pad)
    n = k.shape[2]
    # tokens of each chunk, and the decays from its start, to its end, across it and between its tokens
    tokens = live.sum(1)[:, None] - CHUNK * torch.arange(n, device=q.device)
    tokens = tokens.clamp(0, CHUNK)[:, None, :, None].double()
    at, rate = torch.arange(CHUNK, device=q.device, dtype=torch.float64), g.double()[:, None, None]
    c = {"q": q, "k": k, "v": v32, "live": live, "at": at, "tokens": tokens, "from": ((at + 1) * rate).exp().float()[..., None],
         "to": ((tokens - 1 - at).clamp(min=0) * rate).exp().float()[..., None], "whole": (tokens * rate).exp().float()[..., None]}
    apart = at[:, None] - at
    c["pair"] = torch.where(apart >= 0, (apart * rate).exp(), 0.0).float()[None, :, None]
    p, S, starts, outs = (q @ k.mT) * c["pair"], state, [], []
    writes = (c["to"] * k).mT @ v32
    for i in range(n):
        starts.append(S)
        outs.append(c["from"][:, 0] * (q[:, :, i] @ S) + p[:, :, i] @ v32[:, :, i])
        S = c["whole"][:, :, i] * S + writes[:, :, i]
    o = torch.where(live[..., None, None], _join(torch.stack(outs, 2), T), 0).to(v.dtype)
    return (o, S, c, torch.stack(starts, 2), p) if keep else (o, S)


def _linear_train(s):
    o, state, c, starts, p = _chunks(s["state"], s["q"], s["k"], s["v"], s["g"], s["valid"], s["scale"], keep=True)
    T, rep = s["v"].shape[1], s["v"].shape[2] // s["q"].shape[2]
    do = _split(s["grad"], 1, c["live"], -T % CHUNK)
    reads, dS, ends = (c["from"] * c["q"]).mT @ do, s["grad_state"], []
    for i in reversed(range(do.shape[2])):
        ends.append(dS)
        dS = c["whole"][:, :, i] * dS + reads[:, :, i]
    ends = torch.stack(ends[::-1], 2)
    dp = (do @ c["v"].mT) * c["pair"]
    dq_start, dk_end = c["from"] * (do @ starts.mT), c["to"] * (c["v"] @ ends.mT)
    dq, dk = s["scale"] * (dp @ c["k"] + dq_start), dp.mT @ c["q"] + dk_end
    dv = p.mT @ do + c["to"] * (c["k"] @ ends)

    def out(x, like, heads):  # heads that share a key head add up
        x = torch.where(c["live"][..., None, None], _join(x, T), 0)
        return x.unflatten(2, (-1, heads)).sum(3).to(like.dtype)

    grads = {"readings": o, "state": state, "grad_q": out(dq, s["q"], rep), "grad_k": out(dk, s["k"], rep), "grad_v": out(dv, s["v"], 1),
             "grad_state": dS}
    if s["case"]["decay"]:
        at, tokens = c["at"].float()[:, None], c["tokens"].float()[..., None]
        apart = (at - at.mT).clamp(min=0)
        dg = (apart * ((c["q"] @ c["k"].mT) * dp)).sum((2, 3, 4)) + ((at + 1) * c["q"] * dq_start).sum((2, 3, 4)) \
            + ((tokens - 1 - at).clamp(min=0) * c["k"] * dk_end).sum((2, 3, 4)) \
            + (tokens * c["whole"][..., None].reshape(tokens.shape[0], -1, tokens.shape[2], 1, 1) * starts * ends).sum((2, 3, 4))
        grads["grad_log_decay"] = dg.sum(0)
    return grads


# ---- the definitions in 64 bits -----------------------------------------------------------------

def exact(case, seed):
    if case["op"] in ("group", "group_train"):
        return _exact_group(prepare(case, seed))
    if case["B"] * case["T"] * case["H"] * case["Dk"] * case["Dv"] > 1.8e10:
        return None
    return _exact_linear(prepare(case, seed))


def _exact_group(s):
    case = s["case"]
    x = s["x"].double()
    groups, width = case["G"], case["C"] // case["G"]
    owner = torch.arange(case["C"], device="cuda") // width
    pick = torch.nn.functional.one_hot(owner, groups).double()
    count = case["L"] * width
    mu = (x.sum(1) @ pick) / count                             # [N, G]
    off = x - mu[:, owner][:, None]
    sd = torch.sqrt((off ** 2).sum(1) @ pick / count + 1e-5)[:, owner][:, None]
    h = off / sd
    z = h * s["weight"].double() + s["bias"].double()
    sig = torch.sigmoid(z)
    y = z * sig if case["act"] else z
    if case["op"] == "group":
        return y
    dz = s["grad"].double()
    if case["act"]:
        dz = dz * (sig + y - y * sig)
    out = {"y": y, "grad_weight": torch.einsum("nlc,nlc->c", dz, h), "grad_bias": torch.einsum("nlc->c", dz)}
    dh = dz * s["weight"].double()
    m0, m1 = (dh.sum(1) @ pick / count)[:, owner][:, None], ((dh * h).sum(1) @ pick / count)[:, owner][:, None]
    out["grad_x"] = (dh - m0 - h * m1) / sd
    return out


def _exact_linear(s):
    case = s["case"]
    B, T, H, Hk = case["B"], case["T"], case["H"], case["Hk"]
    owner = torch.arange(H, device="cuda") // (H // Hk)
    q, k, v = s["q"].double()[:, :, owner], s["k"].double()[:, :, owner], s["v"].double()
    fade = s["g"].double().exp()[None, :, None, None]
    valid = s["valid"] if s["valid"] is not None else torch.full((B,), T, device="cuda", dtype=torch.int32)
    on = (torch.arange(T, device="cuda")[None] < valid[:, None]).double()

    def after(S, t):
        m = on[:, t, None, None, None]
        return m * (fade * S + k[:, t, :, :, None] * v[:, t, :, None]) + (1 - m) * S

    S, marks, o = s["state"].double(), [], torch.zeros_like(v)
    for t in range(T):
        if t % 64 == 0:
            marks.append(S)
        S = after(S, t)
        o[:, t] = on[:, t, None, None] * s["scale"] * (q[:, t, :, None] @ S)[:, :, 0]
    out = {"readings": o, "state": S}
    if case["op"] == "linear":
        return out
    dS, do = s["grad_state"].double(), s["grad"].double()
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg = torch.zeros(H, device="cuda", dtype=torch.float64)
    for first in reversed(range(0, T, 64)):
        states = [marks.pop()]
        for t in range(first, min(T, first + 64)):
            states.append(after(states[-1], t))
        for t in reversed(range(first, min(T, first + 64))):
            now, before = states.pop(), states[-1]
            m2, m3 = on[:, t, None, None], on[:, t, None, None, None]
            got = s["scale"] * do[:, t]
            dq[:, t] = m2 * (now @ got[..., None])[..., 0]
            dA = dS + q[:, t, :, :, None] * got[:, :, None]
            dk[:, t] = m2 * (dA @ v[:, t, :, :, None])[..., 0]
            dv[:, t] = m2 * (k[:, t, :, None] @ dA)[:, :, 0]
            dg += (m3 * fade * dA * before).sum((0, 2, 3))
            dS = m3 * fade * dA + (1 - m3) * dS
    add = torch.zeros(Hk, H, device="cuda", dtype=torch.float64)
    add[owner, torch.arange(H, device="cuda")] = 1
    out |= {"grad_q": torch.einsum("gh,bthd->btgd", add, dq), "grad_k": torch.einsum("gh,bthd->btgd", add, dk), "grad_v": dv, "grad_state": dS}
    if case["decay"]:
        out["grad_log_decay"] = dg
    return out
