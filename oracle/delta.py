"""The gated delta rule and layer norm in float64 (numpy), straight from their definitions.

Per token and head, with S the [Dk, Dv] state:
    d = exp(g) S;  r = v - d^T k;  S = d + beta k r^T;  o = scale S^T q
Tokens at or past valid change nothing, and none of their inputs is read.
"""

from __future__ import annotations

import numpy as np


def _heads(x, H):
    """[B, T, Hk, D] -> [B, T, H, D]: value head h uses key head h // (H // Hk)."""
    return np.repeat(x, H // x.shape[2], axis=2)


def gated_delta(state, q, k, v, g, beta, valid=None, scale=1.0, log=None):
    """(readings [B, T, H, Dv], final state). ``log``: a list that takes each token's
    (live rows, state before, decayed state, r, state after)."""
    B, T, H, _ = v.shape
    S = np.array(state, dtype=np.float64)
    o = np.zeros(v.shape)
    n = np.full(B, T) if valid is None else np.clip(valid, 0, T)
    for t in range(T):
        b = np.nonzero(t < n)[0]
        if len(b):
            qt, kt = (_heads(x[b, t:t + 1], H)[:, 0] for x in (q, k))
            d = np.exp(g[b, t])[..., None, None] * S[b]
            r = v[b, t] - np.einsum("bhk,bhkv->bhv", kt, d)
            after = d + beta[b, t][..., None, None] * kt[..., None] * r[..., None, :]
            o[b, t] = scale * np.einsum("bhk,bhkv->bhv", qt, after)
        else:
            d = r = after = None
        if log is not None:
            log.append((b, S[b].copy(), d, r, after))
        if len(b):
            S[b] = after
    return o, S


def gated_delta_backward(state, q, k, v, g, beta, do, dS=None, valid=None, scale=1.0):
    """Reverse mode, token by token: a dict of the gradients, those of shared key heads summed."""
    log = []
    gated_delta(state, q, k, v, g, beta, valid, scale, log)
    B, T, H, Dv = v.shape
    Hk, Dk = q.shape[2:]
    dS = np.zeros((B, H, Dk, Dv)) if dS is None else np.array(dS, dtype=np.float64)
    dq, dk = np.zeros((B, T, H, Dk)), np.zeros((B, T, H, Dk))
    dv, dg, db = np.zeros(v.shape), np.zeros(g.shape), np.zeros(g.shape)
    for t in reversed(range(T)):
        b, before, d, r, after = log[t]
        if not len(b):
            continue
        qt, kt = (_heads(x[b, t:t + 1], H)[:, 0] for x in (q, k))
        got, be = scale * do[b, t], beta[b, t][..., None]
        dq[b, t] = np.einsum("bhkv,bhv->bhk", after, got)
        dA = dS[b] + qt[..., None] * got[..., None, :]              # of the state after
        kd = np.einsum("bhk,bhkv->bhv", kt, dA)
        db[b, t] = (kd * r).sum(-1)
        dr = be * kd
        dv[b, t] = dr
        dk[b, t] = np.einsum("bhkv,bhv->bhk", dA, be * r) - np.einsum("bhkv,bhv->bhk", d, dr)
        dd = dA - kt[..., None] * dr[..., None, :]                  # of the decayed state
        dg[b, t] = (dd * d).sum((-1, -2))
        dS[b] = np.exp(g[b, t])[..., None, None] * dd
    add = lambda x: x.reshape(B, T, Hk, H // Hk, Dk).sum(3)  # noqa: E731
    return {"grad_q": add(dq), "grad_k": add(dk), "grad_v": dv, "grad_log_decay": dg,
            "grad_beta": db, "grad_state": dS}


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """(y, mean, rstd) over the last dimension."""
    mean = x.mean(-1, keepdims=True)
    rstd = 1 / np.sqrt(((x - mean) ** 2).mean(-1, keepdims=True) + eps)
    y = (x - mean) * rstd
    if weight is not None:
        y = y * weight
    return (y if bias is None else y + bias), mean, rstd


def layer_norm_backward(dy, x, weight=None, eps=1e-5):
    """{grad_x, grad_weight, grad_bias}, the last two summed over all leading dimensions."""
    xhat, _, rstd = layer_norm(x, eps=eps)
    w = dy if weight is None else dy * weight
    dx = rstd * (w - w.mean(-1, keepdims=True) - xhat * (w * xhat).mean(-1, keepdims=True))
    lead = tuple(range(x.ndim - 1))
    return {"grad_x": dx, "grad_weight": (dy * xhat).sum(lead), "grad_bias": dy.sum(lead)}
