"""The gated delta rule's kernels against the float64 token loop on the stored inputs.

Tolerances, as max|error| / max|reference|. State and float32 results: every product keeps float32's
accuracy (sums of 2^-24 roundings, a few dozen deep in a chunk, carried along by a recurrence that
does not amplify them for unit keys and beta in [0, 1]): 2e-5. bfloat16 readings add half a unit in
the last place, 2^-9 of the value; twice that is allowed."""

import numpy as np
import pytest
import torch

import sparse_addressed_delta_gb300 as sdm
from oracle import delta as od

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
F32_TOL = 2e-5
TOL = {"f32": F32_TOL, "bf16": 2.0 ** -8 + F32_TOL}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    sdm.library()


def host(t):
    return t.double().cpu().numpy()


def err(a, ref):
    assert tuple(a.shape) == tuple(ref.shape)
    return np.abs(host(a) - ref).max() / max(np.abs(ref).max(), 1e-30) if a.numel() else 0.0


def draw(B, T, Hk, H, Dk, Dv, dtype, seed=0, decay=0.1):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    unit = lambda x: torch.nn.functional.normalize(torch.nn.functional.silu(x), dim=-1)  # noqa: E731
    x = dict(state=0.3 * n(B, H, Dk, Dv), q=unit(n(B, T, Hk, Dk)).to(DT[dtype]), k=unit(n(B, T, Hk, Dk)).to(DT[dtype]),
             v=n(B, T, H, Dv).to(DT[dtype]), g=-decay * torch.nn.functional.softplus(n(B, T, H)), beta=torch.sigmoid(n(B, T, H)))
    return {k: v.cuda() for k, v in x.items()}


def ref(x, valid=None, scale=None):
    scale = x["q"].shape[-1] ** -0.5 if scale is None else scale
    return od.gated_delta(**{n: host(t) for n, t in x.items()}, valid=valid, scale=scale)


def call(x, valid=None, **kw):
    state = x["state"].clone()
    vt = None if valid is None else torch.tensor(valid, dtype=torch.int32, device="cuda")
    o = sdm.gated_delta(state, x["q"], x["k"], x["v"], x["g"], x["beta"], vt, **kw)
    return o, state


def check(x, dtype, valid=None, scale=None):
    o, state = call(x, valid, **({} if scale is None else {"scale": scale}))
    ro, rs = ref(x, valid, scale)
    assert o.dtype == DT[dtype] and o.is_contiguous()
    assert err(o, ro) <= TOL[dtype]
    assert err(state, rs) <= F32_TOL
    return o, state


SHAPES = [  # B, T, Hk, H, Dk, Dv
    (2, 1, 2, 4, 128, 128), (1, 1, 1, 1, 16, 16), (3, 2, 1, 3, 48, 80), (40, 1, 2, 16, 128, 128), (5, 1, 4, 8, 96, 192),
    (1, 5, 2, 2, 64, 512), (2, 16, 1, 2, 128, 64), (2, 17, 1, 2, 128, 64), (1, 31, 2, 2, 64, 64), (1, 32, 1, 1, 32, 48),
    (1, 33, 1, 2, 112, 16), (2, 63, 1, 1, 128, 128), (2, 64, 1, 1, 128, 128), (1, 65, 2, 4, 128, 128),
    (1, 128, 1, 1, 80, 96), (2, 200, 1, 3, 64, 144), (1, 333, 2, 2, 128, 256), (3, 129, 2, 2, 16, 32), (1, 70, 20, 20, 64, 64),
    (1, 70, 1, 160, 64, 32),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_sizes(dtype, shape):
    check(draw(*shape, dtype, seed=sum(shape)), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [3, 40, 150])
def test_valid_tokens(dtype, T):
    """Unequal, empty and out-of-range lengths; whatever stands behind them is not used."""
    x = draw(6, T, 2, 4, 64, 48, dtype, seed=T)
    valid = [T, 0, 1, T // 2, T + 9, -3]
    clamped = np.clip(valid, 0, T)
    want = check(x, dtype, valid)
    for b, n in enumerate(clamped):
        for name in ("q", "k", "v", "g", "beta"):
            x[name][b, n:] = float("nan")
    got = call(x, valid)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for b, n in enumerate(clamped):
        assert not got[0][b, n:].any()
    assert torch.equal(got[1][1], x["state"][1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [4, 90])
def test_resets_and_strong_decays(dtype, T):
    """-inf forgets the state whole; strong and absent decays; a written token survives its own reset."""
    x = draw(2, T, 1, 2, 32, 32, dtype, seed=7, decay=3.0)
    x["g"][0, T // 2] = -torch.inf
    x["g"][1, 1:3] = -torch.inf
    x["g"][1, 3:, 0] = 0.0
    x["g"][0, T // 2 + 1:, 1] = -200.0
    check(x, dtype)
    x["state"][1] = 1e30                      # forgotten, not multiplied by something small
    x["g"][1, 0] = -torch.inf
    assert torch.isfinite(call(x)[0]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_beta_zero_one_two_and_scale(dtype):
    x = draw(2, 100, 2, 2, 64, 64, dtype, seed=8)
    x["beta"][0, :30] = 0.0
    x["beta"][0, 30:60] = 1.0
    x["beta"][1, :20] = 1.9                   # a reflection: still no growth
    check(x, dtype, scale=1.5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_equal_keys(dtype):
    """One key for every token, beta 1, no decay: the chunk's system is as far from diagonal as it gets."""
    x = draw(1, 130, 1, 1, 64, 32, dtype, seed=9)
    x["k"][:] = x["k"][:, :1]
    x["k"][:] = torch.nn.functional.one_hot(torch.tensor(5), 64).to(x["k"])
    x["g"].zero_()
    x["beta"].fill_(1.0)
    check(x, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [6, 80])
def test_strides(dtype, T):
    """Views into a fused projection, head-major tensors and broadcast inputs."""
    B, Hk, H, Dk, Dv = 2, 2, 4, 32, 48
    x = draw(B, T, Hk, H, Dk, Dv, dtype, seed=10)
    want = call(x)
    fused = torch.cat([x[n].flatten(2) for n in ("q", "k", "v")], -1)
    q, k, v = fused.split([Hk * Dk, Hk * Dk, H * Dv], -1)
    y = dict(x, q=q.unflatten(-1, (Hk, Dk)), k=k.unflatten(-1, (Hk, Dk)), v=v.unflatten(-1, (H, Dv)))
    assert not y["q"].is_contiguous()
    gates = torch.stack([x["g"], x["beta"]], -1)
    y |= {"g": gates[..., 0], "beta": gates[..., 1]}
    got = call(y)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    z = {n: (x[n] if n == "state" else x[n].transpose(1, 2).contiguous().transpose(1, 2)) for n in x}
    got = call(z)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    e = dict(x, k=x["k"][:, :, :1].expand(B, T, Hk, Dk), beta=x["beta"][:, :1].expand(B, T, H))
    f = {n: t.contiguous() for n, t in e.items()}
    assert all(torch.equal(a, b) for a, b in zip(call(e), call(f)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cut", [1, 7, 64, 100])
def test_pieces_of_a_sequence(dtype, cut):
    """A sequence in two calls is the sequence in one, within rounding."""
    x = draw(2, 161, 1, 2, 64, 64, dtype, seed=11)
    o, S = call(x)
    a = {n: (t if n == "state" else t[:, :cut]) for n, t in x.items()}
    o1, s1 = call(a)
    o2, s2 = call({n: (s1 if n == "state" else t[:, cut:]) for n, t in x.items()})
    assert err(torch.cat([o1, o2], 1), host(o)) <= 2 * TOL[dtype]
    assert err(s2, host(S)) <= 2 * F32_TOL


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 100])
def test_the_same_bits_again_and_on_another_stream(dtype, T):
    x = draw(3, T, 2, 4, 64, 64, dtype, seed=12)
    want = call(x)
    got = call(x)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    state = x["state"].clone()
    s.wait_stream(torch.cuda.current_stream())
    o = sdm.gated_delta(state, x["q"], x["k"], x["v"], x["g"], x["beta"], stream=s)
    s.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(state, want[1])


def test_no_tokens_and_no_sequences():
    x = draw(2, 0, 1, 2, 32, 32, "f32")
    o, s = call(x)
    assert o.shape == (2, 0, 2, 32) and torch.equal(s, x["state"])
    x = draw(0, 5, 1, 2, 32, 32, "f32")
    assert call(x)[0].shape == (0, 5, 2, 32)


def test_a_given_buffer_and_guard_bytes():
    """Nothing is written outside the readings and the state."""
    x = draw(1, 75, 1, 2, 64, 48, "bf16", seed=13)
    n = 75 * 2 * 48
    buf = torch.full((n + 256,), 7.0, dtype=torch.bfloat16, device="cuda")
    st = torch.full((2 * 64 * 48 + 128,), 7.0, device="cuda")
    state = st[64:-64].view(1, 2, 64, 48)
    state.copy_(x["state"])
    out = buf[128:-128].view(1, 75, 2, 48)
    o = sdm.gated_delta(state, x["q"], x["k"], x["v"], x["g"], x["beta"], readings=out)
    assert o is out and torch.equal(out, call(x)[0])
    assert (buf[:128] == 7).all() and (buf[-128:] == 7).all() and (st[:64] == 7).all() and (st[-64:] == 7).all()


def test_refusals():
    x = draw(2, 4, 2, 4, 32, 32, "bf16")

    def go(**kw):
        y = {**x, **kw}
        return sdm.gated_delta(y["state"], y["q"], y["k"], y["v"], y["g"], y["beta"], y.get("valid"),
                               **{n: y[n] for n in ("readings", "workspace", "scale") if n in y})

    for kw, kind in ((dict(q=x["q"].float()), TypeError), (dict(q=x["q"].half()), TypeError), (dict(k=x["k"][:, :3]), ValueError),
                     (dict(g=x["g"].bfloat16()), TypeError), (dict(beta=x["beta"][..., None]), ValueError),
                     (dict(state=x["state"].bfloat16()), TypeError), (dict(state=x["state"][:1]), ValueError),
                     (dict(state=x["state"].transpose(2, 3)), ValueError), (dict(v=x["v"].cpu()), ValueError),
                     (dict(valid=torch.ones(2, device="cuda")), TypeError), (dict(q=x["q"][0]), ValueError),
                     (dict(v=x["v"].transpose(2, 3).contiguous().transpose(2, 3)), ValueError),
                     (dict(v=torch.zeros((2, 4, 4, 33), dtype=torch.bfloat16, device="cuda")[..., 1:]), ValueError),
                     (dict(readings=x["v"][:, :3]), ValueError), (dict(scale=float("nan")), sdm.SdmError)):
        with pytest.raises(kind):
            go(**kw)
    for Hk, H, Dk, Dv in ((2, 3, 32, 32), (1, 1, 24, 32), (1, 1, 144, 32), (1, 1, 32, 8), (1, 1, 32, 528)):
        with pytest.raises(sdm.SdmError):
            call(draw(1, 2, Hk, H, Dk, Dv, "f32") if H % Hk == 0 else
                 dict(draw(1, 2, 1, H, Dk, Dv, "f32"), q=x["q"][:1, :2].float(), k=x["k"][:1, :2].float()))
