"""The float64 definitions of linear attention and group norm: hand-worked values, and their gradients against
central differences."""

import numpy as np
import pytest

from oracle import linear as ol

rng = np.random.default_rng(5)


def test_two_tokens_by_hand():
    q, k, v = np.array([[[[1.0]], [[2.0]]]]), np.array([[[[3.0]], [[5.0]]]]), np.array([[[[7.0]], [[11.0]]]])
    o, S = ol.linear_attention(np.array([[[[4.0]]]]), q, k, v, np.array([np.log(0.5)]), scale=10.0)
    assert np.allclose(o.ravel(), [10 * (2 + 21), 10 * 2 * (11.5 + 55)]) and np.allclose(S, 66.5)
    o, S = ol.linear_attention(np.array([[[[4.0]]]]), q, k, v, np.array([-np.inf]), valid=[1])
    assert np.allclose(o.ravel(), [21, 0]) and np.allclose(S, 21)


def test_linear_gradients():
    B, T, Hk, H, Dk, Dv = 2, 5, 1, 2, 3, 4
    x = [rng.normal(size=s) for s in ((B, H, Dk, Dv), (B, T, Hk, Dk), (B, T, Hk, Dk), (B, T, H, Dv))] + [-rng.uniform(0.1, 1, H)]
    do, dS, valid = rng.normal(size=(B, T, H, Dv)), rng.normal(size=(B, H, Dk, Dv)), [5, 3]
    grads = ol.linear_attention_backward(*x, do, dS, valid, 0.7)

    def loss():
        o, S = ol.linear_attention(*x, valid=valid, scale=0.7)
        return (o * do).sum() + (S * dS).sum()

    for t, name in zip(x, ("grad_state", "grad_q", "grad_k", "grad_v", "grad_log_decay"), strict=True):
        for i in rng.choice(t.size, min(t.size, 12), replace=False):
            at, h = np.unravel_index(i, t.shape), 1e-6
            t[at] += h
            up = loss()
            t[at] -= 2 * h
            down = loss()
            t[at] += h
            assert abs((up - down) / (2 * h) - grads[name][at]) < 1e-7 * max(1, np.abs(grads[name]).max())


@pytest.mark.parametrize("act", [None, "silu"])
def test_group_norm_gradients(act):
    x, w, b = rng.normal(size=(2, 3, 2, 6)), rng.normal(size=6), rng.normal(size=6)
    dy = rng.normal(size=x.shape)
    y, stats = ol.group_norm(x, 3, w, b, act)
    part = x[1, :, :, 2:4]
    assert np.allclose(stats[1, 1], [part.mean(), 1 / np.sqrt(part.var() + 1e-5)])
    z = (x[0, 1, 1, 5] - stats[0, 2, 0]) * stats[0, 2, 1] * w[5] + b[5]
    assert np.isclose(y[0, 1, 1, 5], z / (1 + np.exp(-z)) if act else z)
    for t, g in zip((x, w, b), ol.group_norm_backward(dy, x, 3, w, b, act), strict=True):
        for i in rng.choice(t.size, 6, replace=False):
            at, h = np.unravel_index(i, t.shape), 1e-6
            t[at] += h
            up = (ol.group_norm(x, 3, w, b, act)[0] * dy).sum()
            t[at] -= 2 * h
            down = (ol.group_norm(x, 3, w, b, act)[0] * dy).sum()
            t[at] += h
            assert abs((up - down) / (2 * h) - g[at]) < 1e-7 * max(1, np.abs(g).max())
