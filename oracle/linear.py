"""Linear attention with a decay for each head and group norm with an activation in float64 (numpy),
straight from their definitions.

Per token and head, with S the [Dk, Dv] state:  S = exp(g) S + k v^T;  o = scale S^T q
Tokens at or past valid change nothing, and none of their inputs is read.
"""

from __future__ import annotations

import numpy as np


def _heads(x, H):
    """[B, T, Hk, D] -> [B, T, H, D]: value head h uses key head h // (H // Hk)."""
    return np.repeat(x, H // x.shape[2], axis=2)


def linear_attention(state, q, k, v, g, valid=None, scale=1.0, log=None):
    """(readings [B, T, H, Dv], final state). ``log``: a list that takes each token's (live rows, state before)."""
    B, T, H, _ = v.shape
    S = np.array(state, dtype=np.float64)
    o = np.zeros(v.shape)
    n = np.full(B, T) if valid is None else np.clip(valid, 0, T)
    fade = np.exp(g)[:, None, None]
    for t in range(T):
        b = np.nonzero(t < n)[0]
        if log is not None:
            log.append((b, S[b].copy()))
        if len(b):
            qt, kt = (_heads(x[b, t:t + 1], H)[:, 0] for x in (q, k))
            S[b] = fade * S[b] + kt[..., None] * v[b, t][..., None, :]
            o[b, t] = scale * np.einsum("bhk,bhkv->bhv", qt, S[b])
    return o, S


def linear_attention_backward(state, q, k, v, g, do, dS=None, valid=None, scale=1.0):
    """Reverse mode, token by token: a dict of the gradients, those of shared key heads summed."""
    log = []
    linear_attention(state, q, k, v, g, valid, scale, log)
    B, T, H, Dv = v.shape
    Hk, Dk = q.shape[2:]
    dS = np.zeros((B, H, Dk, Dv)) if dS is None else np.array(dS, dtype=np.float64)
    dq, dk, dv, dg = np.zeros((B, T, H, Dk)), np.zeros((B, T, H, Dk)), np.zeros(v.shape), np.zeros(H)
    fade = np.exp(g)[:, None, None]
    for t in reversed(range(T)):
        b, before = log[t]
        if not len(b):
            continue
        qt, kt = (_heads(x[b, t:t + 1], H)[:, 0] for x in (q, k))
        after = fade * before + kt[..., None] * v[b, t][..., None, :]
        got = scale * do[b, t]
        dq[b, t] = np.einsum("bhkv,bhv->bhk", after, got)
        dA = dS[b] + qt[..., None] * got[..., None, :]              # of the state after
        dk[b, t] = np.einsum("bhkv,bhv->bhk", dA, v[b, t])
        dv[b, t] = np.einsum("bhkv,bhk->bhv", dA, kt)
        dg += (fade * dA * before).sum((0, 2, 3))
        dS[b] = fade * dA
    shared = lambda x: x.reshape(B, T, Hk, H // Hk, Dk).sum(3)  # noqa: E731
    return {"grad_q": shared(dq), "grad_k": shared(dk), "grad_v": dv, "grad_log_decay": dg, "grad_state": dS}


def _silu(z):
    return 1 / (1 + np.exp(-z))


def group_norm(x, groups, weight=None, bias=None, activation=None, eps=1e-5):
    """x [N, ..., C], statistics over the positions and C / groups channels: (y, stats [N, groups, 2])."""
    h = x.reshape(x.shape[0], -1, groups, x.shape[-1] // groups)
    mean = h.mean((1, 3), keepdims=True)
    rstd = 1 / np.sqrt(((h - mean) ** 2).mean((1, 3), keepdims=True) + eps)
    z = ((h - mean) * rstd).reshape(x.shape)
    z = z * (1 if weight is None else weight) + (0 if bias is None else bias)
    y = z * _silu(z) if activation == "silu" else z
    return y, np.stack([mean[:, 0, :, 0], rstd[:, 0, :, 0]], -1)


def group_norm_backward(dy, x, groups, weight=None, bias=None, activation=None, eps=1e-5):
    """(grad_x, grad_weight, grad_bias)."""
    C = x.shape[-1]
    w = np.ones(C) if weight is None else weight
    h = x.reshape(x.shape[0], -1, groups, C // groups)
    mean = h.mean((1, 3), keepdims=True)
    rstd = 1 / np.sqrt(((h - mean) ** 2).mean((1, 3), keepdims=True) + eps)
    xhat = ((h - mean) * rstd).reshape(x.shape)
    z = xhat * w + (0 if bias is None else bias)
    dz = dy * (_silu(z) * (1 + z * (1 - _silu(z))) if activation == "silu" else 1)
    lead = tuple(range(x.ndim - 1))
    dh = (dz * w).reshape(h.shape)
    xh = xhat.reshape(h.shape)
    dx = rstd * (dh - dh.mean((1, 3), keepdims=True) - xh * (dh * xh).mean((1, 3), keepdims=True))
    return dx.reshape(x.shape), (dz * xhat).sum(lead), dz.sum(lead)
