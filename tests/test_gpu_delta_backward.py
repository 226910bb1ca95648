"""The gated delta rule's saving forward and backward against the float64 reverse mode on the stored
inputs.

Tolerances, as max|error| / max|reference|: float32 gradients, and the gates' and the state's for any
input, are chains of products that keep float32's accuracy, through the forward's recurrence and the
backward's: twice the forward's 2e-5. The gradient of a log-decay is a running sum over the chunk of
terms that partly cancel: 1e-4 of its largest. bfloat16 gradients add two units of 2^-9."""

import numpy as np
import pytest
import torch

import sparse_addressed_delta_gb300 as sdm
from oracle import delta as od
from test_gpu_delta import DT, F32_TOL, TOL, call, draw, err, host, ref

pytestmark = pytest.mark.gpu

GRAD_F32 = 4e-5
GRAD = {"f32": GRAD_F32, "bf16": 2.0 ** -8 + GRAD_F32}
GATE = 1e-4


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    sdm.library()


def grads(shape, dtype, seed=100):
    B, T, Hk, H, Dk, Dv = shape
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(B, T, H, Dv, generator=gen).to(DT[dtype]).cuda(),
            0.3 * torch.randn(B, H, Dk, Dv, generator=gen).cuda())


def train(x, do, dS=None, valid=None, **kw):
    vt = None if valid is None else torch.tensor(valid, dtype=torch.int32, device="cuda")
    state = x["state"].clone()
    args = (x["q"], x["k"], x["v"], x["g"], x["beta"], vt)
    o, saved = sdm.gated_delta_save(state, *args, **kw)
    return o, state, sdm.gated_delta_backward(*args, saved, do, grad_state=dS, **kw)


def check(x, do, dS, dtype, valid=None, scale=None):
    kw = {} if scale is None else {"scale": scale}
    o, state, g = train(x, do, dS, valid, **kw)
    ro, rs = ref(x, valid, scale)
    assert err(o, ro) <= TOL[dtype] and err(state, rs) <= F32_TOL
    want = od.gated_delta_backward(**{n: host(t) for n, t in x.items()}, do=host(do), dS=None if dS is None else host(dS),
                                   valid=valid, scale=x["q"].shape[-1] ** -0.5 if scale is None else scale)
    assert set(g) == set(want)
    for name, a in g.items():
        tol = GATE if name == "grad_log_decay" else GRAD[dtype] if name in ("grad_q", "grad_k", "grad_v") else GRAD_F32
        assert a.dtype == (DT[dtype] if name in ("grad_q", "grad_k", "grad_v") else torch.float32)
        assert err(a, want[name]) <= tol, name
    return o, state, g


SHAPES = [  # B, T, Hk, H, Dk, Dv
    (2, 1, 2, 4, 128, 128), (1, 1, 1, 1, 16, 16), (3, 2, 1, 3, 48, 80), (1, 31, 2, 2, 64, 64), (1, 32, 1, 1, 32, 48),
    (1, 33, 1, 2, 112, 16), (2, 63, 1, 1, 128, 128), (2, 64, 1, 1, 128, 128), (1, 65, 2, 4, 128, 128),
    (1, 128, 1, 1, 80, 96), (2, 200, 1, 3, 64, 144), (1, 150, 2, 2, 128, 256), (3, 129, 2, 2, 16, 32), (1, 70, 1, 160, 64, 80),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_sizes(dtype, shape):
    do, dS = grads(shape, dtype)
    check(draw(*shape, dtype, seed=sum(shape)), do, dS, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_gradient_of_the_final_state_and_a_scale(dtype):
    shape = (2, 100, 2, 4, 64, 48)
    check(draw(*shape, dtype, seed=1), grads(shape, dtype)[0], None, dtype, scale=0.7)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [5, 150])
def test_valid_tokens(dtype, T):
    shape = (6, T, 2, 4, 64, 48)
    x, (do, dS) = draw(*shape, dtype, seed=T), grads(shape, dtype)
    valid = [T, 0, 1, T // 2, T + 9, -3]
    o, s, g = check(x, do, dS, dtype, valid)
    for b, n in enumerate(np.clip(valid, 0, T)):
        for t in (x["q"], x["k"], x["v"], x["g"], x["beta"], do):
            t[b, n:] = float("nan")
    o2, s2, g2 = train(x, do, dS, valid)
    assert torch.equal(o, o2) and torch.equal(s, s2) and all(torch.equal(g[n], g2[n]) for n in g)
    for b, n in enumerate(np.clip(valid, 0, T)):
        assert not any(g[m][b, n:].any() for m in g if m != "grad_state")
    assert torch.equal(g["grad_state"][1], dS[1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_resets_decays_and_betas(dtype):
    shape = (2, 100, 1, 2, 32, 32)
    x, (do, dS) = draw(*shape, dtype, seed=7, decay=2.0), grads(shape, dtype)
    x["g"][0, 50] = -torch.inf
    x["g"][1, 1:3] = -torch.inf
    x["g"][1, 3:, 0] = 0.0
    x["beta"][0, :30] = 0.0
    x["beta"][0, 30:60] = 1.0
    check(x, do, dS, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strides(dtype):
    shape = B, T, Hk, H, Dk, Dv = 2, 80, 2, 4, 32, 48
    x, (do, dS) = draw(*shape, dtype, seed=10), grads(shape, dtype)
    want = train(x, do, dS)
    fused = torch.cat([x[n].flatten(2) for n in ("q", "k", "v")], -1)
    q, k, v = fused.split([Hk * Dk, Hk * Dk, H * Dv], -1)
    gates = torch.stack([x["g"], x["beta"]], -1)
    y = dict(x, q=q.unflatten(-1, (Hk, Dk)), k=k.unflatten(-1, (Hk, Dk)), v=v.unflatten(-1, (H, Dv)), g=gates[..., 0], beta=gates[..., 1])
    turned = do.transpose(1, 2).contiguous().transpose(1, 2)
    got = train(y, turned, dS)
    assert torch.equal(got[0], want[0]) and all(torch.equal(got[2][n], want[2][n]) for n in got[2])
    flat = do[:1, :1].expand(B, T, H, Dv)
    a, b = train(x, flat, dS)[2], train(x, flat.contiguous(), dS)[2]
    assert all(torch.equal(a[n], b[n]) for n in a)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_same_bits_again_on_another_stream_and_the_plain_forward(dtype):
    shape = (3, 100, 2, 4, 64, 64)
    x, (do, dS) = draw(*shape, dtype, seed=12), grads(shape, dtype)
    o, s, g = train(x, do, dS)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    state = x["state"].clone()
    st.wait_stream(torch.cuda.current_stream())
    args = (x["q"], x["k"], x["v"], x["g"], x["beta"], None)
    o2, saved = sdm.gated_delta_save(state, *args, stream=st)
    g2 = sdm.gated_delta_backward(*args, saved, do, grad_state=dS, stream=st)
    st.synchronize()
    assert torch.equal(o, o2) and torch.equal(s, state) and all(torch.equal(g[n], g2[n]) for n in g)
    plain = call(x)
    assert torch.equal(plain[0], o) and torch.equal(plain[1], s)


def test_no_tokens():
    shape = (2, 0, 1, 2, 32, 32)
    x, (do, dS) = draw(*shape, "f32"), grads(shape, "f32")
    o, s, g = train(x, do, dS)
    assert torch.equal(s, x["state"]) and torch.equal(g["grad_state"], dS) and g["grad_q"].shape == (2, 0, 1, 32)
    assert not train(x, do, None)[2]["grad_state"].any()


@pytest.mark.parametrize("name", ["state", "q", "k", "v", "g", "beta"])
def test_gradient_against_differences(name):
    """The kernels' own forward, moved along a direction; float32 readings."""
    shape = (1, 70, 1, 2, 32, 32)
    x, (do, dS) = draw(*shape, "f32", seed=13), grads(shape, "f32")
    g = train(x, do, dS)[2]["grad_" + {"g": "log_decay"}.get(name, name)]
    d = torch.randn(x[name].shape, generator=torch.Generator().manual_seed(14)).cuda()
    h = 1e-2 / float(d.norm())

    def loss(step):
        o, s = call({**x, name: x[name] + step * d})
        return float((o.double() * do.double()).sum() + (s.double() * dS.double()).sum())

    want = float((g.double() * d.double()).sum())
    # second order of the difference, h^2, and the forward's rounding over h
    size = float(g.double().norm() * d.double().norm())
    assert (loss(h) - loss(-h)) / (2 * h) == pytest.approx(want, abs=2e-3 * size)


def test_refusals():
    shape = (2, 20, 2, 4, 32, 32)
    x, (do, dS) = draw(*shape, "bf16"), grads(shape, "bf16")
    args = (x["q"], x["k"], x["v"], x["g"], x["beta"], None)
    saved = sdm.gated_delta_save(x["state"].clone(), *args)[1]
    for bad, kind in ((do.float(), TypeError), (do[:, :3], ValueError), (do.cpu(), ValueError),
                      (torch.zeros((2, 20, 4, 33), dtype=torch.bfloat16, device="cuda")[..., 1:], ValueError)):
        with pytest.raises(kind):
            sdm.gated_delta_backward(*args, saved, bad)
    with pytest.raises(ValueError):
        sdm.gated_delta_backward(*args, saved, do, grad_state=dS[:1])
    with pytest.raises(sdm.SdmError, match="saved buffer"):
        sdm.gated_delta_backward(*args, saved[:256], do)
    with pytest.raises(sdm.SdmError, match="workspace"):
        sdm.gated_delta_backward(*args, saved, do, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(sdm.SdmError, match="saved buffer"):
        sdm.gated_delta_save(x["state"].clone(), *args, saved=torch.empty(256, dtype=torch.uint8, device="cuda"))
