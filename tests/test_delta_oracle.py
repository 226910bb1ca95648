"""The float64 definitions of the gated delta rule and of layer norm: against an explicit matrix
form, against each other's special cases, and their gradients against finite differences."""

import numpy as np
import pytest

from oracle import delta as od


def draw(seed, B=2, T=7, Hk=2, H=4, Dk=5, Dv=3):
    r = np.random.default_rng(seed)
    k = r.standard_normal((B, T, Hk, Dk))
    return dict(state=r.standard_normal((B, H, Dk, Dv)), q=r.standard_normal((B, T, Hk, Dk)),
                k=k / np.linalg.norm(k, axis=-1, keepdims=True), v=r.standard_normal((B, T, H, Dv)),
                g=-0.3 * r.random((B, T, H)), beta=r.random((B, T, H)))


def test_matrix_form():
    x = draw(1)
    o, S = od.gated_delta(**x, scale=0.5)
    for b in range(2):
        for h in range(4):
            M = x["state"][b, h]
            for t in range(7):
                k, q = x["k"][b, t, h // 2], x["q"][b, t, h // 2]
                be = x["beta"][b, t, h]
                M = np.exp(x["g"][b, t, h]) * (np.eye(5) - be * np.outer(k, k)) @ M \
                    + be * np.outer(k, x["v"][b, t, h])
                assert np.allclose(o[b, t, h], 0.5 * M.T @ q, rtol=1e-12, atol=1e-12)
            assert np.allclose(S[b, h], M, rtol=1e-12, atol=1e-12)


def test_valid_tokens_stop_the_sequence():
    x = draw(2)
    o, S = od.gated_delta(**x, valid=np.array([3, 0]))
    cut = {n: (a if n == "state" else a[:1, :3]) for n, a in x.items()}
    cut["state"] = x["state"][:1]
    o1, S1 = od.gated_delta(**cut)
    assert np.array_equal(o[0, :3], o1[0]) and np.array_equal(S[0], S1[0])
    assert not o[0, 3:].any() and not o[1].any() and np.array_equal(S[1], x["state"][1])


def test_a_reset_forgets_everything():
    x = draw(3)
    x["g"][:, 4] = -np.inf
    a = od.gated_delta(**x)[1]
    x["state"] = 5 * x["state"]
    assert np.array_equal(a, od.gated_delta(**x)[1])


def difference(f, x, d, h=1e-5):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


@pytest.mark.parametrize("name", ["state", "q", "k", "v", "g", "beta"])
def test_delta_gradient_against_differences(name):
    x, r = draw(4), np.random.default_rng(5)
    do, dS, valid = r.standard_normal(x["v"].shape), r.standard_normal(x["state"].shape), np.array([7, 4])

    def loss(a):
        o, S = od.gated_delta(**{**x, name: a}, valid=valid, scale=0.7)
        return (o * do).sum() + (S * dS).sum()

    grads = od.gated_delta_backward(**x, do=do, dS=dS, valid=valid, scale=0.7)
    key = {"g": "grad_log_decay"}.get(name, "grad_" + name)
    for _ in range(3):
        d = r.standard_normal(x[name].shape)
        assert difference(loss, x[name], d) == pytest.approx((grads[key] * d).sum(), rel=1e-6, abs=1e-7)


@pytest.mark.parametrize("name", ["x", "weight", "bias"])
def test_norm_gradient_against_differences(name):
    r = np.random.default_rng(6)
    x = dict(x=r.standard_normal((4, 9)), weight=r.standard_normal(9), bias=r.standard_normal(9))
    dy = r.standard_normal((4, 9))
    grads = od.layer_norm_backward(dy, x["x"], x["weight"])
    d = r.standard_normal(x[name].shape)
    got = difference(lambda a: (od.layer_norm(**{**x, name: a})[0] * dy).sum(), x[name], d)
    assert got == pytest.approx((grads["grad_" + name] * d).sum(), rel=1e-6, abs=1e-8)
