"""Linear attention with a decay for each head against the float64 token loop on the stored inputs.

Tolerances, as max|error| / max|reference|. State and float32 results: products keep float32's accuracy (a value is a
sum of a few hundred products that are 2^-24 off each, within a chunk and carried along by decays of at most 1, which
do not amplify it): 2e-5 covers 2^-24 times the 300 terms' sum of magnitudes. bfloat16 results are such values rounded
once, by at most half a step: 2^-8 of the value on top."""

import numpy as np
import pytest
import torch

import sparse_addressed_delta_gb300 as sdm
from oracle import linear as ol

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


def draw(B, T, Hk, H, Dk, Dv, dtype, seed=0, forget=(0.3, 0.003)):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    unit = lambda x: torch.nn.functional.normalize(torch.nn.functional.silu(x), dim=-1)  # noqa: E731
    x = dict(state=0.3 * n(B, H, Dk, Dv), q=unit(n(B, T, Hk, Dk)).to(DT[dtype]), k=unit(n(B, T, Hk, Dk)).to(DT[dtype]),
             v=n(B, T, H, Dv).to(DT[dtype]), g=torch.log1p(-torch.exp(torch.linspace(np.log(forget[0]), np.log(forget[1]), H))))
    return {k: v.cuda() for k, v in x.items()}


def ref(x, valid=None, scale=None):
    scale = x["q"].shape[-1] ** -0.5 if scale is None else scale
    return ol.linear_attention(**{n: host(t) for n, t in x.items()}, valid=valid, scale=scale)


def lengths(valid):
    return None if valid is None else torch.tensor(valid, dtype=torch.int32, device="cuda")


def call(x, valid=None, **kw):
    state = x["state"].clone()
    return sdm.linear_attention(state, x["q"], x["k"], x["v"], x["g"], lengths(valid), **kw), state


def check(x, dtype, valid=None, scale=None):
    o, state = call(x, valid, **({} if scale is None else {"scale": scale}))
    ro, rs = ref(x, valid, scale)
    assert o.dtype == DT[dtype] and o.is_contiguous()
    assert err(o, ro) <= TOL[dtype]
    assert err(state, rs) <= F32_TOL
    return o, state


SHAPES = [  # B, T, Hk, H, Dk, Dv
    (2, 1, 2, 4, 128, 128), (1, 1, 1, 1, 16, 16), (3, 2, 1, 3, 48, 80), (40, 1, 2, 16, 128, 128), (5, 1, 4, 8, 96, 192),
    (1, 5, 2, 2, 64, 512), (2, 12, 1, 2, 32, 64), (2, 13, 1, 2, 128, 64), (2, 17, 1, 2, 128, 64), (1, 31, 2, 2, 64, 64),
    (1, 33, 1, 2, 112, 16), (2, 63, 1, 1, 128, 128), (2, 64, 1, 1, 128, 128), (1, 65, 2, 4, 128, 128),
    (1, 128, 1, 1, 80, 96), (2, 200, 1, 3, 64, 144), (1, 333, 2, 2, 128, 256), (3, 129, 2, 2, 16, 32), (1, 70, 20, 20, 64, 64),
    (1, 70, 1, 160, 64, 32), (1, 1500, 1, 2, 64, 64), (1, 900, 2, 2, 48, 272),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_sizes(dtype, shape):
    check(draw(*shape, dtype, seed=sum(shape)), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [3, 40, 150, 1100])
def test_valid_tokens(dtype, T):
    """Unequal, empty and out-of-range lengths; whatever stands behind them is not used."""
    x = draw(6, T, 2, 4, 64, 48, dtype, seed=T)
    valid = [T, 0, 1, T // 2, T + 9, -3]
    clamped = np.clip(valid, 0, T)
    want = check(x, dtype, valid)
    for b, n in enumerate(clamped):
        for name in ("q", "k", "v"):
            x[name][b, n:] = float("nan")
    got = call(x, valid)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for b, n in enumerate(clamped):
        assert not got[0][b, n:].any()
    assert torch.equal(got[1][1], x["state"][1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [4, 90, 1000])
def test_decays(dtype, T):
    """No decay, strong ones, and resets at every token."""
    x = draw(2, T, 1, 5, 32, 32, dtype, seed=7)
    x["g"].copy_(torch.tensor([0.0, -3.0, -20.0, -torch.inf, -200.0]))
    o, state = check(x, dtype)
    reset = x["k"][:, -1, :, :, None].float() * x["v"][:, -1, 3:, None].float()
    assert torch.allclose(state[:, 3:], reset, rtol=1e-6, atol=0)
    x["state"][:, 3:] = 1e30                  # forgotten, not multiplied by something small
    assert torch.isfinite(call(x)[0]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scale_and_zeros(dtype):
    x = draw(2, 100, 2, 2, 64, 64, dtype, seed=8)
    check(x, dtype, scale=-3.0)
    x["k"].zero_()
    x["state"].zero_()
    o, state = call(x)
    assert not o.any() and not state.any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [6, 200])
def test_layouts(dtype, T):
    """Heads cut out of wider rows, heads first, and inputs broadcast along each dimension."""
    x = draw(2, T, 2, 4, 32, 48, dtype, seed=9)
    want = call(x)
    wide = torch.randn(2, T, 4 * 48 + 2 * 2 * 32 + 16, device="cuda").to(DT[dtype])
    y = dict(x, q=wide[..., :64].unflatten(-1, (2, 32)), k=wide[..., 64:128].unflatten(-1, (2, 32)), v=wide[..., 144:336].unflatten(-1, (4, 48)))
    for name in ("q", "k", "v"):
        y[name].copy_(x[name])
    got = call(y)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    y = dict(x, **{n: x[n].transpose(1, 2).contiguous().transpose(1, 2) for n in ("q", "k", "v")})
    got = call(y)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for dim in range(3):
        y = dict(x, **{n: x[n].narrow(dim, 0, 1).expand_as(x[n]) for n in ("q", "k", "v")})
        got, whole = call(y), call({n: t.contiguous() for n, t in y.items()})
        assert torch.equal(got[0], whole[0]) and torch.equal(got[1], whole[1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_in_pieces(dtype):
    """A prompt in unequal pieces, then single tokens, is the whole sequence."""
    x = draw(2, 300, 1, 2, 64, 64, dtype, seed=10)
    ro, rs = ref(x)
    state, at, parts = x["state"].clone(), 0, []
    for n in (130, 1, 7, 64, 90, 1, 1, 6):
        cut = [x[name][:, at:at + n] for name in ("q", "k", "v")]
        parts.append(sdm.linear_attention(state, *cut, x["g"]))
        at += n
    assert at == 300
    assert err(torch.cat(parts, 1), ro) <= TOL[dtype] and err(state, rs) <= F32_TOL


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_empty(dtype):
    x = draw(2, 0, 2, 2, 32, 32, dtype)
    o, state = call(x)
    assert o.shape == (2, 0, 2, 32) and torch.equal(state, x["state"])
    x = draw(0, 5, 2, 2, 32, 32, dtype)
    assert call(x)[0].shape == (0, 5, 2, 32)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [5, 100, 1200])
def test_nan_and_infinity(dtype, T):
    """A NaN or infinity of a token reaches that token's and later tokens' readings, those of a value in its
    column alone."""
    x = draw(2, T, 1, 2, 32, 48, dtype, seed=11)
    want = call(x)[0]
    at = T - 3
    for name, where, bad in (("v", (0, at, 1, 5), float("nan")), ("v", (0, at, 1, 5), float("inf")), ("k", (0, at, 0, 7), float("nan")),
                             ("q", (0, at, 0, 7), float("nan"))):
        y = dict(x, **{name: x[name].clone()})
        y[name][where] = bad
        o, state = call(y)
        touched = torch.zeros_like(o, dtype=torch.bool)
        if name == "v":
            touched[0, at:, 1, 5] = True
        else:
            touched[0, at:at + 1 if name == "q" else T] = True
        # (the column is taken again token by token, in another order of sums)
        assert err(o[~touched], host(want[~touched])) <= TOL[dtype]
        assert not torch.isfinite(o[touched]).any()
        if name == "q":
            assert torch.isfinite(state).all()


def test_streams_and_graphs():
    x = draw(2, 150, 2, 4, 64, 64, "bf16", seed=12)
    want = call(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    state = x["state"].clone()
    side.wait_stream(torch.cuda.current_stream())
    o = sdm.linear_attention(state, x["q"], x["k"], x["v"], x["g"], stream=side)
    side.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(state, want[1])
    for T in (1, 150):
        cut = {n: x[n][:, :T].contiguous() for n in ("q", "k", "v")}
        state = x["state"].clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o = sdm.linear_attention(state, cut["q"], cut["k"], cut["v"], x["g"])
        for _ in range(2):
            state.copy_(x["state"])
            graph.replay()
            want = call(dict(x, **cut))
            assert torch.equal(o, want[0]) and torch.equal(state, want[1])
            cut["v"].copy_(-cut["v"])


def test_refusals():
    x = draw(2, 20, 2, 4, 32, 32, "bf16", seed=13)
    ok = dict(state=x["state"], q=x["q"], k=x["k"], v=x["v"], log_decay=x["g"])
    for change, kind in ((dict(q=x["q"].float()), TypeError), (dict(k=x["k"][:, :5]), ValueError), (dict(v=x["v"].cpu()), ValueError),
                         (dict(log_decay=x["g"][:2]), ValueError), (dict(log_decay=x["g"].double()), TypeError),
                         (dict(state=x["state"].bfloat16()), TypeError), (dict(state=x["state"].mT), ValueError),
                         (dict(valid_tokens=torch.ones(2, device="cuda")), TypeError), (dict(scale=float("nan")), sdm.SdmError),
                         (dict(q=x["q"][..., 1:17], k=x["k"][..., 1:17]), ValueError),
                         (dict(v=x["v"][:, :, :3]), sdm.SdmError), (dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda")), sdm.SdmError)):
        with pytest.raises(kind):
            args = dict(ok, **change)
            if "v" in change and change["v"].shape[2] == 3:
                args.update(state=x["state"][:, :3].contiguous(), log_decay=x["g"][:3].contiguous())
            sdm.linear_attention(**args)
    y = draw(1, 20, 1, 1, 24, 32, "bf16")
    with pytest.raises(sdm.SdmError):
        call(y)
