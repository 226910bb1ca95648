"""The backward of linear attention against the float64 reverse mode and against differences.

Tolerances, as max|error| / max|reference|: float32 gradients 4e-5 (twice the forward's: the state and its gradient are
both such sums), a decay's gradient 4e-5 of the sum of its terms' magnitudes over all tokens; bfloat16 gradients are
rounded once, half a step (2^-8 of the value) on top."""

import numpy as np
import pytest
import torch

import sparse_addressed_delta_gb300 as sdm
from oracle import linear as ol
from test_gpu_linear import DT, call, draw, err, host, lengths

pytestmark = pytest.mark.gpu
F32_TOL = 4e-5
TOL = {"f32": F32_TOL, "bf16": 2.0 ** -8 + F32_TOL}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    sdm.library()


def grads_of(x, dtype, seed, with_state=True):
    gen = torch.Generator().manual_seed(seed + 1000)
    do = torch.randn(x["v"].shape, generator=gen).to(DT[dtype]).cuda()
    return do, 0.2 * torch.randn(x["state"].shape, generator=gen).cuda() if with_state else None


def train(x, do, dS, valid=None, scale=None, **kw):
    state = x["state"].clone()
    args = (x["q"], x["k"], x["v"], x["g"], lengths(valid))
    o, saved = sdm.linear_attention_save(state, *args, scale=scale)
    return o, state, sdm.linear_attention_backward(*args, saved, do, grad_state=dS, scale=scale, **kw)


def decay_terms(x, do, dS, valid, scale):
    """A bound of the magnitudes that a decay's gradient sums: its token terms by the absolute values' recurrence."""
    pos = {n: np.abs(host(t)) if n != "g" else host(t) for n, t in x.items()}
    return ol.linear_attention_backward(**pos, do=np.abs(host(do)), dS=None if dS is None else np.abs(host(dS)), valid=valid,
                                        scale=abs(scale))["grad_log_decay"]


def check(x, dtype, seed=0, valid=None, scale=None, with_state=True):
    do, dS = grads_of(x, dtype, seed, with_state)
    kept = None if dS is None else dS.clone()
    o, state, got = train(x, do, dS, valid, scale)
    plain = call(x, valid, **({} if scale is None else {"scale": scale}))
    if x["v"].shape[1] > sdm.LINEAR_STEP_TOKENS:
        assert torch.equal(o, plain[0]) and torch.equal(state, plain[1])
    assert dS is None or torch.equal(dS, kept)
    scale = x["q"].shape[-1] ** -0.5 if scale is None else scale
    want = ol.linear_attention_backward(**{n: host(t) for n, t in x.items()}, do=host(do), dS=None if dS is None else host(dS), valid=valid,
                                        scale=scale)
    assert set(got) == set(want)
    for name in ("grad_q", "grad_k", "grad_v"):
        assert got[name].dtype == DT[dtype] and err(got[name], want[name]) <= TOL[dtype], name
    assert err(got["grad_state"], want["grad_state"]) <= F32_TOL
    off = np.abs(host(got["grad_log_decay"]) - want["grad_log_decay"])
    assert (off <= F32_TOL * decay_terms(x, do, dS, valid, scale) + 1e-30).all()
    return got


SHAPES = [  # B, T, Hk, H, Dk, Dv
    (2, 1, 2, 4, 128, 128), (1, 1, 1, 1, 16, 16), (3, 2, 1, 3, 48, 80), (2, 9, 1, 2, 128, 64), (1, 33, 1, 2, 112, 16),
    (2, 63, 1, 1, 128, 128), (2, 64, 2, 2, 128, 128), (1, 65, 2, 4, 128, 128), (2, 200, 1, 3, 64, 144), (1, 333, 2, 2, 128, 256),
    (3, 129, 2, 2, 16, 32), (1, 70, 20, 20, 64, 64), (1, 1500, 1, 2, 64, 64), (1, 600, 1, 2, 48, 272), (2, 700, 2, 2, 128, 128),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_sizes(dtype, shape):
    check(draw(*shape, dtype, seed=sum(shape)), dtype, seed=sum(shape))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [3, 40, 150, 1100])
def test_valid_tokens(dtype, T):
    x = draw(6, T, 2, 4, 64, 48, dtype, seed=T)
    valid = [T, 0, 1, T // 2, T + 9, -3]
    want = check(x, dtype, T, valid)
    do, dS = grads_of(x, dtype, T)
    for b, n in enumerate(np.clip(valid, 0, T)):
        for t in (x["q"], x["k"], x["v"], do):
            t[b, n:] = float("nan")
    got = train(x, do, dS, valid)[2]
    for name, t in got.items():
        assert torch.equal(t, want[name]), name
    for b, n in enumerate(np.clip(valid, 0, T)):
        assert not any(got[name][b, n:].any() for name in ("grad_q", "grad_k", "grad_v"))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [30, 600])
def test_decays(dtype, T):
    x = draw(2, T, 1, 5, 32, 32, dtype, seed=21)
    x["g"].copy_(torch.tensor([0.0, -0.5, -3.0, -10.0, -110.0]))
    got = check(x, dtype, 3)
    want = host(got["grad_log_decay"])
    x["g"][4] = -torch.inf
    do, dS = grads_of(x, dtype, 3)
    reset = train(x, do, dS)[2]["grad_log_decay"]
    assert reset[4] == 0 and np.array_equal(host(reset)[:4], want[:4])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_options(dtype):
    """No gradient of the final state, another scale, fixed decays, strided and broadcast gradients."""
    x = draw(2, 90, 1, 2, 64, 64, dtype, seed=22)
    check(x, dtype, 4, with_state=False, scale=-2.0)
    do, dS = grads_of(x, dtype, 5)
    want = train(x, do, dS)[2]
    got = train(x, do, dS, decay=False)[2]
    assert set(want) - set(got) == {"grad_log_decay"} and all(torch.equal(got[n], want[n]) for n in got)
    first = do.transpose(1, 2).contiguous().transpose(1, 2)
    got = train(x, first, dS)[2]
    assert all(torch.equal(got[n], want[n]) for n in want)
    for dim in range(3):
        one = do.narrow(dim, 0, 1).expand_as(do)
        a, b = train(x, one, dS)[2], train(x, one.contiguous(), dS)[2]
        assert all(torch.equal(a[n], b[n]) for n in a)


def test_differences():
    """Against central differences of the kernels' own forward, summed in float64, along one direction for each input:
    the difference of two float32 results 1e-2 apart leaves 1e-3 of the derivative. The loss is linear in every input but
    the decays; of its terms, e^(n g) times a constant with n up to T, a difference over h w of g is off by (h w n)^2 / 6."""
    x = draw(2, 100, 1, 2, 32, 32, "f32", seed=23)
    do, dS = grads_of(x, "f32", 6)
    got = train(x, do, dS)[2]
    gen = torch.Generator().manual_seed(9)
    for name, grad in (("state", "grad_state"), ("q", "grad_q"), ("k", "grad_k"), ("v", "grad_v"), ("g", "grad_log_decay")):
        way = torch.randn(x[name].shape, generator=gen).cuda()
        way = way if name != "g" else way.abs()
        h = 1e-2 if name != "g" else 1e-3

        def loss(by):
            o, s = call(dict(x, **{name: x[name] + by * way}))
            return (o.double() * do.double()).sum() + (s.double() * dS.double()).sum()

        slope = (loss(h) - loss(-h)) / (2 * h)
        want = (got[grad].double() * way.double()).sum()
        scale = (got[grad].double() * way.double()).abs().sum()
        curved = (h * way.max().item() * 100) ** 2 / 6 if name == "g" else 0
        assert abs(slope - want) <= (1e-3 + curved) * scale


def test_empty_and_alias():
    x = draw(2, 0, 2, 2, 32, 32, "bf16")
    do, dS = grads_of(x, "bf16", 7)
    got = train(x, do, dS)[2]
    assert torch.equal(got["grad_state"], dS) and not got["grad_log_decay"].any()
    got = train(x, do, None)[2]
    assert not got["grad_state"].any()
    x = draw(0, 5, 2, 2, 32, 32, "bf16")
    do, dS = grads_of(x, "bf16", 7)
    assert not train(x, do, dS)[2]["grad_log_decay"].any()


def test_graph():
    """A training step captured and replayed."""
    x = draw(2, 150, 2, 4, 64, 64, "bf16", seed=24)
    do, dS = grads_of(x, "bf16", 8)
    state = x["state"].clone()
    args = (x["q"], x["k"], x["v"], x["g"], None)

    def step():
        o, saved = sdm.linear_attention_save(state, *args)
        return o, sdm.linear_attention_backward(*args, saved, do, grad_state=dS)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, got = step()
    for _ in range(2):
        state.copy_(x["state"])
        graph.replay()
        wo, _, want = train(x, do, dS)
        assert torch.equal(o, wo) and all(torch.equal(got[n], want[n]) for n in want)
        x["v"].copy_(-x["v"])


def test_refusals():
    x = draw(2, 20, 2, 4, 32, 32, "bf16", seed=25)
    do, dS = grads_of(x, "bf16", 9)
    args = (x["q"], x["k"], x["v"], x["g"], None)
    saved = sdm.linear_attention_save(x["state"].clone(), *args)[1]
    with pytest.raises(TypeError):
        sdm.linear_attention_backward(*args, None, do)
    with pytest.raises(TypeError):
        sdm.linear_attention_backward(*args, saved, do.float())
    with pytest.raises(ValueError):
        sdm.linear_attention_backward(*args, saved, do[:, :10])
    with pytest.raises(TypeError):
        sdm.linear_attention_backward(*args, saved, do, grad_state=dS.double())
    with pytest.raises(sdm.SdmError):
        sdm.linear_attention_backward(*args, saved[:256], do)
