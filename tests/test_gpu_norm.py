"""Layer norm's kernels against the float64 definition on the stored inputs.

Tolerances, as max|error| / max|reference|: a float32 sum of n terms is at most about
(16 + 10 + 16) roundings deep (a thread's 16 elements, the warp, the block's warps), each 2^-24 of
the terms' size, and a row's result is a handful of such sums over values of its own size: 1e-5
covers it. The gradient of x is a difference of such terms, rstd w dy and its means, and is held to
their size: with few columns the difference itself is next to nothing (none is left of it at n = 1).
bfloat16 results add half a unit in the last place, 2^-9 of the value; twice that is allowed. Column sums add the rows of a block in one chain, at most 2^11 deep here: 1e-4 of the
largest sum's terms, in practice far less."""

import numpy as np
import pytest
import torch

import sparse_addressed_delta_gb300 as sdm
from oracle import delta as od

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
TOL = {"f32": 1e-5, "bf16": 2.0 ** -8 + 1e-5}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    sdm.library()


def host(t):
    return t.double().cpu().numpy()


def err(a, ref):
    assert a.shape == ref.shape
    return np.abs(host(a) - ref).max() / max(np.abs(ref).max(), 1e-30) if a.numel() else 0.0


def draw(shape, dtype, seed, shift=0.5):
    r = np.random.default_rng(seed)
    return torch.from_numpy(r.standard_normal(shape) + shift).to(DT[dtype]).cuda()


def check(x, dy, weight, bias, dtype, eps=1e-5):
    y, stats = sdm.layer_norm_save(x, weight, bias, eps=eps)
    w64 = None if weight is None else host(weight)
    ry, mean, rstd = od.layer_norm(host(x), w64, None if bias is None else host(bias), eps)
    assert y.is_contiguous() and y.dtype == x.dtype
    assert err(y, ry) <= TOL[dtype]
    assert torch.equal(sdm.layer_norm(x, weight, bias, eps=eps), y)
    assert err(stats[..., 0], mean[..., 0]) <= 1e-5 and err(stats[..., 1], rstd[..., 0]) <= 1e-5
    g = sdm.layer_norm_backward(dy, x, weight, stats, bias=bias is not None)
    ref = od.layer_norm_backward(host(dy), host(x), w64, eps)
    assert set(g) == {"grad_x"} | ({"grad_weight"} if weight is not None else set()) \
        | ({"grad_bias"} if bias is not None else set())
    terms = np.abs(rstd * host(dy) * (1.0 if w64 is None else w64)).max()
    assert np.abs(host(g["grad_x"]) - ref["grad_x"]).max() <= TOL[dtype] * terms
    for name in set(g) - {"grad_x"}:
        assert err(g[name], ref[name]) <= 1e-4, name
    again = sdm.layer_norm_backward(dy, x, weight, stats, bias=bias is not None)
    assert all(torch.equal(g[n], again[n]) for n in g)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,n", [(1, 1), (3, 2), (7, 33), (1, 128), (1000, 128), (65, 96), (5, 512), (33, 513),
                                    (40, 1007), (9, 2048), (3, 4094), (17, 4096), (2, 8191), (4, 8200), (3, 16384),
                                    (2, 16383), (20000, 64), (3000, 250)])
def test_sizes(dtype, rows, n):
    x, dy = draw((rows, n), dtype, rows + n), draw((rows, n), dtype, rows + n + 1, 0.0)
    w = 1 + 0.2 * draw((n,), "f32", 2, 0.0)
    check(x, dy, w, 0.1 * draw((n,), "f32", 3), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,n", [(2, 9), (4001, 33), (2500, 66), (1300, 129), (1300, 1007), (700, 1006), (333, 4099), (170, 4098), (311, 8191)])
def test_many_rows_no_vector_divides(dtype, rows, n):
    """Rows one behind the other that start at any element of a 16-byte piece; more rows than blocks; an input that
    is the result too."""
    x, dy = draw((rows, n), dtype, rows + n), draw((rows, n), dtype, rows + n + 1, 0.0)
    w, b = 1 + 0.2 * draw((n,), "f32", 2, 0.0), 0.1 * draw((n,), "f32", 3)
    check(x, dy, w, b, dtype)
    y = sdm.layer_norm(x, w, b)
    assert torch.equal(sdm.layer_norm(x, w, b, out=x), y) and torch.equal(x, y)


@pytest.mark.parametrize("n", [64, 250, 2048])
@pytest.mark.parametrize("params", ["none", "weight", "bias", "bf16"])
def test_parameters(params, n):
    x, dy = draw((21, n), "bf16", 4), draw((21, n), "bf16", 5)
    wt = "bf16" if params == "bf16" else "f32"
    w = draw((n,), wt, 6) if params in ("weight", "bf16") else None
    b = draw((n,), wt, 7) if params in ("bias", "bf16") else None
    check(x, dy, w, b, "bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,pad,off", [(128, 8, 0), (128, 1, 0), (128, 0, 1), (1007, 1, 3), (2048, 2, 2), (2048, 64, 0)])
def test_strides_and_offsets(dtype, n, pad, off):
    """Rows inside a wider buffer, starting at any element."""
    def view(seed):
        return draw((30 * (n + pad) + off,), dtype, seed)[off:].view(30, n + pad)[:, :n]
    check(view(8), view(9), draw((n,), "f32", 10), draw((n,), "f32", 11), dtype)


def test_leading_dimensions_and_a_broadcast_gradient():
    x = draw((3, 5, 4, 64), "f32", 12)[:, :, 1:3].transpose(0, 0)
    with pytest.raises(ValueError, match="one stride"):
        sdm.layer_norm(x)
    check(draw((3, 5, 64), "f32", 13), draw((1, 1, 64), "f32", 14).expand(3, 5, 64), draw((64,), "f32", 15), None, "f32")


def test_no_rows():
    x = torch.empty((0, 64), device="cuda")
    y, stats = sdm.layer_norm_save(x)
    assert y.shape == (0, 64) and stats.shape == (0, 2)
    g = sdm.layer_norm_backward(x, x, torch.ones(64, device="cuda"), stats)
    assert not g["grad_weight"].any() and not g["grad_bias"].any() and g["grad_x"].shape == (0, 64)


def test_far_from_zero_and_constant_rows():
    """The variance is taken around the mean: a large offset costs no more than float32's spacing."""
    x = draw((16, 1000), "f32", 16, 1000.0)
    ref = od.layer_norm(host(x))[0]
    assert err(sdm.layer_norm(x), ref) <= 1000 * 2.0 ** -23        # the mean's own rounding
    c = torch.full((4, 777), 3.25, device="cuda")
    assert not sdm.layer_norm(c).any()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_row_stays_alone(bad):
    x = draw((300, 130), "bf16", 17)
    y0 = sdm.layer_norm(x)
    x[7, 129] = bad
    y1 = sdm.layer_norm(x)
    keep = torch.arange(300, device="cuda") != 7
    assert torch.equal(y0[keep], y1[keep]) and y1[7].isnan().all()


def test_in_place_and_on_another_stream():
    x = draw((1000, 512), "bf16", 18)
    want = sdm.layer_norm(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = sdm.layer_norm(x, out=x, stream=s)
    s.synchronize()
    assert got is x and torch.equal(x, want)


def test_gradient_against_differences():
    x, dy = draw((6, 100), "f32", 19), draw((6, 100), "f32", 20)
    w, b = draw((100,), "f32", 21), draw((100,), "f32", 22)
    stats = sdm.layer_norm_save(x, w, b)[1]
    g = sdm.layer_norm_backward(dy, x, w, stats)
    for name, a in (("grad_x", x), ("grad_weight", w), ("grad_bias", b)):
        d, h = draw(tuple(a.shape), "f32", 23, 0.0), 1e-2
        moved = [tuple(t + s * h * d if t is a else t for t in (x, w, b)) for s in (1, -1)]
        up, down = ((sdm.layer_norm(*m).double() * dy.double()).sum().item() for m in moved)
        want = (g[name].double() * d.double()).sum().item()
        # third-order term h^2 and the forward's rounding 2^-24 / h
        assert (up - down) / (2 * h) == pytest.approx(want, rel=5e-3, abs=5e-3 * float(dy.norm()))


def test_refusals():
    x = draw((4, 64), "f32", 24)
    st = torch.zeros((4, 2), device="cuda")
    with pytest.raises(TypeError):
        sdm.layer_norm(x.half())
    with pytest.raises(TypeError):
        sdm.layer_norm(x, torch.ones(64, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        sdm.layer_norm(x, torch.ones(63, device="cuda"))
    with pytest.raises(ValueError):
        sdm.layer_norm(x.t())
    with pytest.raises(ValueError):
        sdm.layer_norm(x.cpu())
    with pytest.raises(ValueError):
        sdm.layer_norm(x, out=torch.empty((4, 65), device="cuda"))
    with pytest.raises(sdm.SdmError):
        sdm.layer_norm(x, eps=-1.0)
    with pytest.raises(sdm.SdmError, match="16384"):
        sdm.layer_norm(torch.zeros((1, 16385), device="cuda"))
    with pytest.raises(ValueError):
        sdm.layer_norm_backward(x[:3], x, None, st)
    with pytest.raises(ValueError):
        sdm.layer_norm_backward(x, x, None, st[:3])
    with pytest.raises(sdm.SdmError, match="workspace"):
        sdm.layer_norm_backward(x, x, None, st, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
