"""A NaN or an infinity among the gated delta rule's inputs reaches what the definition says and nothing else: readings
of earlier tokens, other sequences, heads and (for a value) columns are what they are without it. The float64 token
loop says where results are finite; there the usual tolerances hold."""

import numpy as np
import pytest
import torch

import sparse_addressed_delta_gb300 as sdm
from test_gpu_delta import F32_TOL, TOL, call, draw, host, ref

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    sdm.library()


def same(a, want, tol):
    a, live = host(a), np.isfinite(want)
    assert np.array_equal(np.isfinite(a), live)
    assert np.abs(a[live] - want[live]).max(initial=0) <= tol * np.abs(want[live]).max(initial=1e-30)


def check(x, dtype, valid=None):
    with np.errstate(all="ignore"):
        ro, rs = ref(x, valid)
    assert not np.isfinite(ro).all()
    o, state = call(x, valid)
    same(o, ro, TOL[dtype])
    same(state, rs, F32_TOL)
    if o.shape[1] <= sdm.DELTA_STEP_TOKENS:
        return                                # token by token; the saving forward is in chunks
    kept = x["state"].clone()
    vt = None if valid is None else torch.tensor(valid, dtype=torch.int32, device="cuda")
    o2 = sdm.gated_delta_save(kept, x["q"], x["k"], x["v"], x["g"], x["beta"], vt)[0]
    assert torch.equal(torch.nan_to_num(o2, 7.0), torch.nan_to_num(o, 7.0))
    assert torch.equal(torch.nan_to_num(kept, 7.0), torch.nan_to_num(state, 7.0))


WHERE = [("v", NAN), ("v", INF), ("v", -INF), ("k", NAN), ("k", INF), ("g", NAN), ("g", INF), ("beta", NAN), ("beta", -INF), ("q", NAN),
         ("q", INF)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name,value", WHERE)
@pytest.mark.parametrize("t", [0, 5, 15, 16, 31, 45, 63, 64, 98, 99])
def test_a_token(dtype, name, value, t):
    """One token of one sequence and head, at every place of a chunk and its blocks."""
    x = draw(2, 100, 1, 2, 48, 144, dtype, seed=60)
    cell = x[name][1, t, -1]
    if cell.dim():
        cell[7] = value
    else:
        cell.fill_(value)
    check(x, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name,value", [("v", INF), ("k", NAN), ("g", NAN), ("beta", INF)])
@pytest.mark.parametrize("shape", [(1, 1500, 1, 2, 128, 128), (1, 1281, 2, 2, 64, 320)], ids=str)
@pytest.mark.parametrize("t", [0, 3, 700, 1279])
def test_in_segments(dtype, name, value, shape, t):
    x = draw(*shape, dtype, seed=61, decay=0.001)
    cell = x[name][0, t, 0]
    if cell.dim():
        cell[20] = value
    else:
        cell.fill_(value)
    check(x, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [6, 100, 1500])
def test_several_columns_tokens_and_a_state(dtype, T):
    """Columns that go wrong at their own tokens, a state that is so from the start, a short sequence."""
    x = draw(3, T, 1, 2, 64, 128, dtype, seed=62, decay=0.001)
    for i, t in enumerate(range(0, T, max(1, T // 7))):
        x["v"][0, t, 0, 5 * i] = (NAN, INF, -INF)[i % 3]
    x["state"][1, 1, 3, 100] = NAN
    x["state"][2, 0, 0, 0] = INF
    check(x, dtype, [T, T - 1, 3])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_decay_too_large_for_float32(dtype):
    x = draw(1, 90, 1, 2, 32, 32, dtype, seed=63)
    x["g"][0, 41, 1] = 200.0
    o, state = call(x)
    with np.errstate(all="ignore"):
        ro, _ = ref(x)
    assert np.abs(host(o)[0, :, 0] - ro[0, :, 0]).max() <= TOL[dtype] * np.abs(ro[0, :, 0]).max()
    assert np.abs(host(o)[0, :41] - ro[0, :41]).max() <= TOL[dtype] * np.abs(ro[0, :41]).max()
    assert not torch.isfinite(o[0, 41:, 1]).any() and not torch.isfinite(state[0, 1]).any() and torch.isfinite(state[0, 0]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("t", [20, 99])
def test_large_values_are_finite(dtype, t):
    """Near the largest float, and no infinity: every column as the definition has it."""
    x = draw(1, 100, 1, 2, 48, 64, dtype, seed=64)
    x["v"][0, t, 0, 3] = 2e38
    o, state = call(x)
    ro, rs = ref(x)
    for a, want, tol in ((host(o), ro, TOL[dtype]), (host(state), rs, F32_TOL), (host(o)[:, :t], ro[:, :t], TOL[dtype])):
        for part in (np.s_[..., 3], np.s_[..., 4:]):
            assert np.abs(a[part] - want[part]).max() <= tol * np.abs(want[part]).max()
