"""Group norm with an activation, forward and backward, against float64 on the stored inputs.

Tolerances. float32 results: 4e-6 of the magnitudes that they are sums of (sums of up to 2^17 values kept in parts of a few
dozen, each a few 2^-24 of its magnitudes off, and a dozen roundings after them). xhat is a difference of x and the mean,
times rstd: 4e-6 of max |x| rstd, which is more than xhat where a group of two channels has two nearly equal values; the
activation's slope is at most 1.1, and changes by at most 1/2 as z does by 1. grad_x is rstd times the difference of three
terms. bfloat16 results are rounded once more, by at most half a step, 2^-8 of the value. Weight and bias gradients are
float32 sums over all samples and positions."""

import numpy as np
import pytest
import torch

import sparse_addressed_delta_gb300 as sdm
from oracle import linear as ol

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
F32_TOL = 4e-6
TOL = {"f32": F32_TOL, "bf16": 2.0 ** -8 + F32_TOL}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    sdm.library()


def host(t):
    return None if t is None else t.double().cpu().numpy()


def off(a, ref):
    assert tuple(a.shape) == tuple(ref.shape)
    return np.abs(host(a) - ref).max() / max(np.abs(ref).max(), 1e-30)


def draw(shape, dtype, seed=0, mean=0.5, wdtype=torch.float32):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    C = shape[-1]
    x = (n(*shape) * (1 + 2 * torch.rand(C, generator=gen)) + mean * n(C)).to(DT[dtype])
    return x.cuda(), (1 + 0.2 * n(C)).to(wdtype).cuda(), (0.2 * n(C)).to(wdtype).cuda(), n(*shape).to(DT[dtype]).cuda()


def check(x, groups, w, b, dy, act, dtype):
    y, stats = sdm.group_norm_save(x, groups, w, b, activation=act)
    hx, hw, hb, hd = host(x), host(w), host(b), host(dy)
    ry, rs = ol.group_norm(hx, groups, hw, hb, act)
    half = 2.0 ** -8 if dtype == "bf16" else 0.0
    each = x.shape[-1] // groups
    wide = lambda t: np.repeat(t, each, -1).reshape(x.shape[:1] + (1,) * (x.ndim - 2) + x.shape[-1:])  # noqa: E731
    rstd, top = wide(rs[..., 1]), wide(np.abs(hx.reshape(x.shape[0], -1, groups, each)).max((1, 3)))
    aw = np.ones(x.shape[-1]) if w is None else np.abs(hw)
    doubt = F32_TOL * top * rstd                            # of xhat
    assert y.dtype == DT[dtype] and y.is_contiguous()
    assert (np.abs(host(y) - ry) <= half * np.abs(ry) + 1.1 * (doubt * aw + F32_TOL * (np.abs(ry) + 1))).all()
    assert (np.abs(host(stats)[..., 0] - rs[..., 0]) <= F32_TOL * top.reshape(x.shape[0], groups, each)[..., 0]).all()
    assert (np.abs(host(stats)[..., 1] / rs[..., 1] - 1) <= F32_TOL + 2 * doubt.reshape(x.shape[0], groups, each)[..., 0]).all()
    assert torch.equal(sdm.group_norm(x, groups, w, b, activation=act), y)
    got = sdm.group_norm_backward(dy, x, groups, w, b, stats, activation=act)
    rx, rw, rb = ol.group_norm_backward(hd, hx, groups, hw, hb, act)
    assert set(got) == {"grad_x"} | ({"grad_weight"} if w is not None else set()) | ({"grad_bias"} if b is not None else set())
    xhat = np.abs(ol.group_norm(hx, groups)[0])
    terms = 1.1 * np.abs(hd) * aw
    mean = lambda t: wide(t.reshape(x.shape[0], -1, groups, each).mean((1, 3)))  # noqa: E731
    # the terms' own errors, and those that xhat's doubt brings into each of them (by the slope's change too)
    sizes = terms + mean(terms) + xhat * mean(terms * xhat)
    moved = (terms * aw + mean(terms * aw) + xhat * mean(terms * aw * xhat) + mean(terms * xhat) + xhat * mean(terms)) * doubt + 3 * doubt * sizes
    assert got["grad_x"].dtype == DT[dtype]
    assert (np.abs(host(got["grad_x"]) - rx) <= half * np.abs(rx) + rstd * (F32_TOL * sizes + moved)).all()
    lead = tuple(range(x.ndim - 1))
    slope = 1.1 * np.abs(hd)
    if w is not None:
        assert (np.abs(host(got["grad_weight"]) - rw) <= (slope * (F32_TOL * xhat + doubt * (1 + aw * xhat))).sum(lead)).all()
    if b is not None:
        assert (np.abs(host(got["grad_bias"]) - rb) <= (slope * (F32_TOL + doubt * aw)).sum(lead)).all()
    return y, got


SHAPES = [  # samples.., channels; groups
    ((1, 1), 1), ((3, 8), 1), ((5, 16), 8), ((33, 2048), 16), ((7, 4096), 32), ((300, 96), 6), ((130, 60), 20), ((9, 35), 5), ((3, 4098), 2),
    ((2, 8192), 1), ((2, 16384), 1), ((5, 16384), 8192), ((1000, 18), 2), ((40, 100), 100), ((3, 7, 64), 8), ((2, 1, 64), 4),
    ((3, 33, 47, 20), 4), ((2, 100, 512), 32), ((4, 1000, 8), 1), ((1, 5000, 24), 3), ((2, 300, 1030), 103), ((2, 90, 4096), 32),
    ((3, 1551, 180), 20), ((70, 9, 40), 5), ((2, 3, 16384), 2), ((1, 2, 2), 1), ((6, 40, 3), 3),
]


@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape,groups", SHAPES, ids=str)
def test_sizes(shape, groups, dtype, act):
    x, w, b, dy = draw(shape, dtype, seed=sum(shape))
    check(x, groups, w, b, dy, act, dtype)


@pytest.mark.parametrize("shape,groups", [((40, 256), 8), ((3, 70, 96), 6)], ids=str)
def test_parameters(shape, groups):
    """Each parameter left out, and parameters of the channels' own type."""
    for act in (None, "silu"):
        x, w, b, dy = draw(shape, "bf16", seed=3)
        check(x, groups, None, None, dy, act, "bf16")
        check(x, groups, w, None, dy, act, "bf16")
        check(x, groups, None, b, dy, act, "bf16")
        x, w, b, dy = draw(shape, "bf16", seed=4, wdtype=torch.bfloat16)
        check(x, groups, w, b, dy, act, "bf16")


@pytest.mark.parametrize("shape,groups", [((40, 256), 8), ((3, 70, 96), 6), ((20, 90), 6)], ids=str)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_layouts(shape, groups, dtype):
    """Positions cut out of wider ones, at 16-byte and at odd offsets, and in place."""
    x, w, b, dy = draw(shape, dtype, seed=5)
    want = sdm.group_norm_save(x, groups, w, b, activation="silu")
    grads = sdm.group_norm_backward(dy, x, groups, w, b, want[1], activation="silu")
    C = shape[-1]
    for first, width in ((16, C + 32), (3, C + 5)):
        both = [torch.randn(*shape[:-1], width, device="cuda").to(DT[dtype]) for _ in range(2)]
        cut = [t[..., first:first + C] for t in both]
        cut[0].copy_(x)
        cut[1].copy_(dy)
        y, stats = sdm.group_norm_save(cut[0], groups, w, b, activation="silu")
        # another vector width adds a sum's values in another order
        assert off(y, host(want[0])) <= 2 * TOL[dtype] and off(stats, host(want[1])) <= 2 * F32_TOL
        got = sdm.group_norm_backward(cut[1], cut[0], groups, w, b, stats, activation="silu")
        assert off(got["grad_x"], host(grads["grad_x"])) <= 2 * TOL[dtype]
        if first == 16:
            assert torch.equal(y, want[0]) and all(torch.equal(got[n], grads[n]) for n in grads)
    z = x.clone()
    assert sdm.group_norm(z, groups, w, b, activation="silu", out=z) is z and torch.equal(z, want[0])


def test_far_means():
    """A mean of 3000 deviations: the squares are taken around means, so what is lost are the mean's own roundings, 2^-24
    of it each: at most one for each of the 16 (split positions: 64) values that a thread adds, and seven joining them."""
    gen = torch.Generator().manual_seed(6)
    for shape, groups in (((50, 256), 4), ((2, 900, 64), 4)):
        x = (3000 + torch.randn(*shape, generator=gen)).cuda()
        y, stats = sdm.group_norm_save(x, groups)
        ry, rs = ol.group_norm(host(x), groups)
        assert np.abs(host(y) - ry).max() <= (16 + 7 if len(shape) == 2 else 64 + 7) * 3000 * 2.0 ** -24
        assert np.abs(host(stats)[..., 1] / rs[..., 1] - 1).max() <= 1e-5


def test_constant_and_nonfinite():
    """A constant group has variance 0; NaN and infinity stay in their sample's group."""
    for shape in ((6, 64), (6, 50, 64)):
        x, w, b, dy = draw(shape, "f32", seed=7)
        want = sdm.group_norm(x, 4, w, b)
        x[1, ..., :16] = 2.0
        x[3, ..., 20] = float("nan")
        x[4, ..., 40] = float("inf")
        y = sdm.group_norm(x, 4, w, b)
        assert torch.allclose(y[1, ..., :16], b[:16].expand_as(y[1, ..., :16]))
        assert y[3, ..., 16:32].isnan().all() and y[4, ..., 32:48].isnan().all()
        keep = torch.ones_like(x, dtype=torch.bool)
        keep[1, ..., :16] = keep[3, ..., 16:32] = keep[4, ..., 32:48] = False
        assert torch.equal(y[keep], want[keep])
        assert torch.isfinite(sdm.group_norm(torch.full_like(x, -1e4), 4, w, b - 200, activation="silu")).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_differences(dtype):
    """The gradients against central differences of the float64 definition, along one direction for each input: bfloat16
    gradients' roundings (2^-9 each) average out over a thousand terms, float32's are far below the differences' 1e-6."""
    for shape, groups in (((20, 64), 4), ((3, 20, 24), 3)):
        x, w, b, dy = draw(shape, dtype, seed=8)
        stats = sdm.group_norm_save(x, groups, w, b, activation="silu")[1]
        got = sdm.group_norm_backward(dy, x, groups, w, b, stats, activation="silu")
        rng = np.random.default_rng(9)
        args = [host(x), host(w), host(b)]
        for i, name in enumerate(("grad_x", "grad_weight", "grad_bias")):
            way, h = rng.normal(size=args[i].shape), 1e-4
            loss = lambda by: (ol.group_norm(*[a + (by * way if j == i else 0) for j, a in enumerate(args)][:1], groups,  # noqa: E731
                                             *[a + (by * way if j == i else 0) for j, a in enumerate(args)][1:], "silu")[0] * host(dy)).sum()
            slope = (loss(h) - loss(-h)) / (2 * h)
            terms = host(got[name]) * way
            assert abs(slope - terms.sum()) <= (2.0 ** -8 if dtype == "bf16" and i == 0 else 1e-5) * np.abs(terms).sum()


def test_empty():
    for shape in ((0, 64), (3, 0, 64), (0, 5, 64)):
        x, w, b, dy = draw(shape, "bf16")
        y, stats = sdm.group_norm_save(x, 4, w, b)
        assert y.shape == shape and stats.shape == (shape[0], 4, 2)
        got = sdm.group_norm_backward(dy, x, 4, w, b, stats)
        assert not got["grad_weight"].any() and not got["grad_bias"].any()


def test_streams_and_graphs():
    for shape in ((40, 256), (3, 200, 64)):
        x, w, b, dy = draw(shape, "bf16", seed=10)

        def step(**kw):
            y, stats = sdm.group_norm_save(x, 8, w, b, activation="silu", **kw)
            return [y, *sdm.group_norm_backward(dy, x, 8, w, b, stats, activation="silu", **kw).values()]

        want = step()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = step(stream=side)
        side.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(got, want, strict=True))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step()
        x.mul_(1.5)
        graph.replay()
        assert all(torch.equal(a, c) for a, c in zip(got, step(), strict=True))


def test_refusals():
    x, w, b, dy = draw((4, 10, 64), "bf16")
    stats = sdm.group_norm_save(x, 4, w, b)[1]
    for args, kw, kind in (((x, 5, w, b), {}, ValueError), ((x, 0), {}, ValueError), ((x, 4, w[:32], b), {}, ValueError),
                           ((x, 4, w.double(), None), {}, TypeError), ((x, 4, w, b.bfloat16()), {}, TypeError),
                           ((x, 4, w, b), dict(activation="relu"), ValueError), ((x, 4, w, b), dict(eps=-1.0), sdm.SdmError),
                           ((x[0, 0], 4), {}, ValueError), ((x.half(), 4), {}, (TypeError, ValueError)), ((x.cpu(), 4), {}, ValueError),
                           ((x.transpose(1, 2), 2), {}, ValueError), ((x, 4, w, b), dict(out=x.float()), TypeError),
                           ((x, 4, w, b), dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda")), sdm.SdmError)):
        with pytest.raises(kind):
            sdm.group_norm(*args, **kw)
    with pytest.raises(sdm.SdmError):
        sdm.group_norm(torch.zeros(2, 16400, device="cuda"), 4)
    for bad in ((dy[:2], x), (dy.float(), x)):
        with pytest.raises(ValueError):
            sdm.group_norm_backward(*bad, 4, w, b, stats)
    with pytest.raises(ValueError):
        sdm.group_norm_backward(dy, x, 8, w, b, stats)
