"""Linear attention and group norm called as the documentation allows and the other tests do not: operands at odd
addresses and shared between arguments, infinite states, one head's NaN, samples in many splits."""

import pytest
import torch

import sparse_addressed_delta_gb300 as sdm
import test_gpu_group_norm as tg
from test_gpu_linear import DT, call, check, draw, lengths
from test_gpu_linear_backward import check as check_back
from test_gpu_linear_backward import grads_of, train

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    sdm.library()


def shifted(t, by=1):
    """The same values `by` elements behind an aligned address."""
    flat = torch.empty(t.numel() + by, dtype=t.dtype, device=t.device)
    flat[by:].copy_(t.reshape(-1))
    return flat[by:].view(t.shape)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 70, 900])
def test_a_gradient_at_an_odd_address(dtype, T):
    """The final state's gradient 4 bytes past a 16-byte address, in one segment and in several."""
    x = draw(2, T, 1, 2, 64, 96, dtype, seed=41)
    do, dS = grads_of(x, dtype, 41)
    want, got = train(x, do, dS)[2], train(x, do, shifted(dS))[2]
    assert all(torch.equal(got[n], want[n]) for n in want)


@pytest.mark.parametrize("T", [1, 70])
def test_odd_addresses_are_refused(T):
    x = draw(1, T, 1, 2, 32, 32, "bf16", seed=42)
    for name in ("q", "k", "v"):
        with pytest.raises((ValueError, sdm.SdmError)):
            call({**x, name: shifted(x[name])})
    state = shifted(x["state"])
    with pytest.raises((ValueError, sdm.SdmError)):
        sdm.linear_attention(state, x["q"], x["k"], x["v"], x["g"])
    with pytest.raises((ValueError, sdm.SdmError)):
        call(x, readings=shifted(x["v"]))
    do, dS = grads_of(x, "bf16", 42)
    with pytest.raises((ValueError, sdm.SdmError)):
        train(x, shifted(do), dS)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 70, 900])
def test_an_infinite_state(dtype, T):
    """An infinity or NaN of the state is in its column's readings and final state, and in no other column."""
    x = draw(2, T, 1, 2, 32, 48, dtype, seed=43)
    want, last = call(x)
    for bad in (torch.inf, -torch.inf, torch.nan):
        x["state"][1, 0, 5, 7] = bad
        o, state = call(x)
        hit = torch.zeros_like(o, dtype=torch.bool)
        hit[1, :, 0, 7] = True
        assert not torch.isfinite(o[hit]).any()
        assert torch.equal(o[~hit], want[~hit])
        hit = torch.zeros_like(state, dtype=torch.bool)
        hit[1, 0, :, 7] = True
        assert not torch.isfinite(state[1, 0, 5, 7])
        assert torch.equal(state[~hit], last[~hit])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [5, 70, 900])
def test_one_heads_nan_decay(dtype, T):
    x = draw(2, T, 3, 3, 32, 32, dtype, seed=44)
    do, dS = grads_of(x, dtype, 44)
    o, state, grads = train(x, do, dS)
    x["g"][1] = torch.nan
    for got, want in ((call(x), call({**x, "g": torch.where(torch.isnan(x["g"]), -0.1, x["g"])})),):
        for a, b in zip(got, want):
            at = 2 if a.dim() == 4 and a is got[0] else 1
            a, b = (t.movedim(at, 0) for t in (a, b))
            assert torch.equal(a[[0, 2]], b[[0, 2]]) and torch.isnan(a[1]).any()
    got = train(x, do, dS)[2]
    for name, heads in (("grad_q", 2), ("grad_k", 2), ("grad_v", 2), ("grad_state", 1), ("grad_log_decay", 0)):
        a, b = (t[name].movedim(heads, 0)[[0, 2]] for t in (got, grads))
        assert torch.equal(a, b), name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_one_tensor_for_all(dtype):
    """q, k and v the same tensor, forward and backward."""
    for T in (7, 130):
        x = draw(2, T, 2, 2, 64, 64, dtype, seed=45)
        x["q"] = x["v"] = x["k"]
        check(x, dtype)
        check_back(x, dtype, 45)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_readings_in_a_wider_buffer(dtype):
    """What lies around them is left as it was."""
    x = draw(3, 40, 2, 2, 32, 32, dtype, seed=46)
    want = call(x)[0]
    buf = torch.full((5, 40, 2, 32), 7.0, dtype=DT[dtype], device="cuda")
    got = call(x, readings=buf[1:4])[0]
    assert torch.equal(got, want) and (buf[0] == 7).all() and (buf[4] == 7).all()


def test_a_saved_buffer_of_another_shape():
    """Too small a one is refused, before anything is queued."""
    x = draw(2, 70, 1, 2, 64, 64, "bf16", seed=47)
    do, dS = grads_of(x, "bf16", 47)
    saved = sdm.linear_attention_save(x["state"][:1].clone(), x["q"][:1], x["k"][:1], x["v"][:1], x["g"])[1]
    with pytest.raises(sdm.SdmError):
        sdm.linear_attention_backward(x["q"], x["k"], x["v"], x["g"], None, saved, do, grad_state=dS)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_ragged_batch_in_segments(dtype):
    """Lengths that leave segments of a long sequence empty, cut inside a chunk, or all of it padding."""
    x = draw(5, 1100, 1, 2, 64, 64, dtype, seed=48)
    valid = [1100, 1, 0, 63, 130]
    check(x, dtype, valid)
    check_back(x, dtype, 48, valid)
    # what stands in the padding is not looked at
    want = call(x, valid)
    for n in ("q", "k", "v"):
        for b, at in enumerate(valid):
            x[n][b, at:] = torch.nan
    got = call(x, valid)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("shape,groups", [((1, 9001, 64), 4), ((2, 57, 8192), 8), ((1, 5000, 24), 24), ((3, 25, 2056), 1), ((500, 9, 40), 5),
                                          ((1, 7, 16384), 16384), ((2, 4099, 6), 3)], ids=str)
def test_group_norm_splits(shape, groups, act, dtype):
    """As many splits as there are blocks, groups as wide as a block and wider, channels of a group each."""
    x, w, b, dy = tg.draw(shape, dtype, seed=sum(shape))
    tg.check(x, groups, w, b, dy, act, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("shape,groups", [((3, 300, 128), 32), ((2, 500, 640), 32), ((1, 130, 2056), 8), ((2, 40, 16384), 4096), ((2, 333, 36), 4),
                                          ((2, 90, 104), 104), ((700, 40, 24), 3), ((1, 3000, 8), 4), ((500, 60, 1032), 24), ((300, 60, 2056), 257), ((2, 9000, 648), 72)], ids=str)
def test_group_norm_groups_that_end_inside_vectors(shape, groups, act, dtype):
    """Groups of a few channels, odd ones and single ones, where 16 bytes of a position hold several or parts of them."""
    x, w, b, dy = tg.draw(shape, dtype, seed=sum(shape))
    tg.check(x, groups, w, b, dy, act, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape,groups", [((31337, 10, 8), 1), ((1500, 6, 40), 5), ((3, 4, 96), 12), ((611, 16, 64), 64), ((305, 2, 510), 6), ((1, 2, 4), 2)],
                         ids=str)
def test_group_norm_small_samples(shape, groups, dtype):
    """Several samples a block, more of them than the blocks take in one turn, the last turn not full."""
    x, w, b, dy = tg.draw(shape, dtype, seed=sum(shape))
    tg.check(x, groups, w, b, dy, "silu", dtype)
    wide = torch.zeros(shape[:-1] + (shape[-1] + 8,), dtype=x.dtype, device="cuda")
    wide[..., :shape[-1]] = x
    wide[..., shape[-1]:] = torch.nan
    assert torch.equal(sdm.group_norm(wide[..., :shape[-1]], groups, w, b), sdm.group_norm(x, groups, w, b))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_group_norm_of_repeated_positions(dtype):
    """One row for all positions and samples (a stride of zero), and parameters and gradients at odd addresses."""
    x, w, b, dy = tg.draw((3, 50, 64), dtype, seed=49)
    row = x[:1, :1].expand(3, 50, 64)
    tg.check(row, 4, w, b, dy, "silu", dtype)
    want = tg.check(x, 4, w, b, dy, "silu", dtype)
    stats = sdm.group_norm_save(x, 4, w, b, activation="silu")[1]
    got = sdm.group_norm_backward(shifted(dy), shifted(x), 4, shifted(w), shifted(b), stats, activation="silu")
    for n in got:                                        # by narrower pieces the sums' order differs
        assert (got[n] - want[1][n]).abs().max() <= 2.0 ** -7 * want[1][n].abs().max()
    mixed = x.expand(3, 50, 64)[:, ::2]
    with pytest.raises(ValueError):
        sdm.group_norm(mixed[:, :7], 4)                  # (positions 2 rows apart, samples 50)


def test_group_norm_without_column_sums():
    """A backward without weight and bias is one with weights of 1 and biases of 0."""
    for shape in ((40, 256), (2, 300, 96)):
        x, _, _, dy = tg.draw(shape, "f32", seed=50)
        one, zero = torch.ones(shape[-1], device="cuda"), torch.zeros(shape[-1], device="cuda")
        stats = sdm.group_norm_save(x, 4, activation="silu")[1]
        a = sdm.group_norm_backward(dy, x, 4, None, None, stats, activation="silu")
        b = sdm.group_norm_backward(dy, x, 4, one, zero, stats, activation="silu")
        assert set(a) == {"grad_x"} and torch.equal(a["grad_x"], b["grad_x"])


def test_lengths_of_one_tensor():
    """The same lengths tensor for two calls in one capture, replayed after it changes."""
    x = draw(3, 100, 1, 2, 32, 32, "bf16", seed=51)
    n = lengths([100, 20, 0])
    state = x["state"].clone()
    args = (x["q"], x["k"], x["v"], x["g"], n)
    sdm.linear_attention(state.clone(), *args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        first = sdm.linear_attention(state, *args)
        second = sdm.linear_attention(state, *args)
    for valid in ([100, 20, 0], [3, 0, 100]):
        n.copy_(torch.tensor(valid))
        state.copy_(x["state"])
        graph.replay()
        want = x["state"].clone()
        for got in (first, second):
            assert torch.equal(got, sdm.linear_attention(want, *args))
        assert torch.equal(state, want)
