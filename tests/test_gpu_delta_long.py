"""The gated delta rule over long sequences of few heads, which are scanned in segments at once, against the
float64 token loop and its reverse mode. The decays are weak, so that a first token's write is still in the
last state. Tolerances are those of the short sequences: a segment's first state is one more float32 product."""

import pytest
import torch

import sparse_addressed_delta_gb300 as sdm
from oracle import delta as od
from test_gpu_delta import call, check, draw, err, host
from test_gpu_delta_backward import GATE, GRAD, GRAD_F32, grads, train
from test_gpu_delta_backward import check as check_train

pytestmark = pytest.mark.gpu

# B, T, Hk, H, Dk, Dv
SHAPES = [(1, 2048, 1, 2, 128, 128), (1, 1500, 1, 1, 64, 80), (2, 1281, 1, 2, 128, 320), (1, 2111, 6, 6, 80, 144),
          (1, 1700, 1, 3, 48, 48), (1, 1800, 8, 32, 64, 128)]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    sdm.library()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(dtype, shape):
    x = draw(*shape, dtype, seed=sum(shape), decay=0.001)
    first, again = check(x, dtype), call(x)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    # the state reaches the end: without it the last one is another
    x["state"].zero_()
    assert not torch.equal(call(x)[1], first[1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES[:-1], ids=str)
def test_backward(dtype, shape):
    x = draw(*shape, dtype, seed=sum(shape), decay=0.001)
    do, dS = grads(shape, dtype)
    o, state, g = check_train(x, do, dS, dtype)
    plain = call(x)
    assert torch.equal(plain[0], o) and torch.equal(plain[1], state)
    again = train(x, do, dS)[2]
    assert all(torch.equal(again[n], g[n]) for n in g)
    check_train(x, do, None, dtype)


def test_backward_of_another_layout():
    """What is saved depends on the shape alone: a forward of queries and keys of one broadcast head, and a backward
    of their contiguous copies; the same with queries broadcast along the tokens, which are laid out first."""
    shape = (1, 1500, 2, 2, 64, 128)
    x = draw(*shape, "bf16", seed=3, decay=0.001)
    do, dS = grads(shape, "bf16")
    x["q"], x["k"] = x["q"][:, :, :1].contiguous().expand(-1, -1, 2, -1), x["k"][:, :, :1].contiguous().expand(-1, -1, 2, -1)
    args = lambda y: (y["q"], y["k"], y["v"], y["g"], y["beta"], None)  # noqa: E731
    y = dict(x, q=x["q"].contiguous(), k=x["k"].contiguous())
    z = dict(x, q=x["q"][:, :1].expand(-1, 1500, -1, -1))
    for one, other in ((x, y), (z, dict(z, q=z["q"].contiguous(), k=y["k"]))):
        saved = sdm.gated_delta_save(one["state"].clone(), *args(one))[1]
        got = sdm.gated_delta_backward(*args(other), saved, do, grad_state=dS)
        want = od.gated_delta_backward(**{n: host(t) for n, t in one.items()}, do=host(do), dS=host(dS), valid=None, scale=64 ** -0.5)
        for n, a in got.items():
            assert err(a, want[n]) <= (GATE if n == "grad_log_decay" else GRAD["bf16"] if a.dtype == torch.bfloat16 else GRAD_F32), n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_valid_tokens(dtype):
    """Lengths from none to all of them: segments of a single chunk, and of none."""
    shape = (6, 1900, 1, 2, 64, 128)
    x = draw(*shape, dtype, seed=5, decay=0.001)
    valid = [1900, 0, 1, 65, 700, 1899]
    o, state = check(x, dtype, valid)
    do, dS = grads(shape, dtype)
    trained = check_train(x, do, dS, dtype, valid)
    assert torch.equal(trained[0], o) and torch.equal(trained[1], state)
    for name in ("q", "k", "v", "g", "beta"):
        for b, n in enumerate(valid):
            x[name][b, n:] = float("nan")
    got = call(x, valid)
    assert torch.equal(got[0], o) and torch.equal(got[1], state)
    assert torch.equal(got[1][1], x["state"][1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_resets(dtype):
    """A reset inside a segment and one at every token."""
    x = draw(1, 1600, 1, 2, 128, 128, dtype, seed=9, decay=0.001)
    x["g"][0, 777, 0] = -torch.inf
    x["g"][0, :, 1] = -torch.inf
    check(x, dtype)
    check_train(x, *grads((1, 1600, 1, 2, 128, 128), dtype), dtype)


def test_nothing_written_stays_nothing():
    """Keys that are too long would blow any state up (each token takes (1 - beta k k^T) = -1.3 of it along
    them); a state of zeros stays one."""
    x = draw(1, 64 * 40, 1, 1, 64, 128, "bf16", seed=4)
    for name in ("state", "v", "g"):
        x[name].zero_()
    x["beta"].fill_(1.0)
    x["k"].fill_((2.3 / 64) ** 0.5)
    o, state = call(x)
    assert not o.any() and not state.any()


def test_gives_up_and_recovers():
    """With a limit of one poll the first launch's waits give up; the second sees that in the status and leaves
    too; the next call with the default limit is right."""
    shape = (1, 2048, 1, 2, 128, 128)
    x, (do, dS) = draw(*shape, "bf16", seed=6, decay=0.001), grads(shape, "bf16")
    args = (x["q"], x["k"], x["v"], x["g"], x["beta"], None)
    packed = sdm._delta_shape(*args, None, do)[0]
    lib = sdm.library()
    fws = torch.empty(lib.sdm_gated_delta_workspace_bytes(packed), dtype=torch.uint8, device="cuda")
    bws = torch.empty(lib.sdm_gated_delta_backward_workspace_bytes(packed), dtype=torch.uint8, device="cuda")
    want, saved = sdm.gated_delta_save(x["state"].clone(), *args, workspace=fws)
    right = sdm.gated_delta_backward(*args, saved, do, grad_state=dS, workspace=bws)
    assert sdm.device_status(fws)["code"] == 0 and sdm.device_status(bws)["code"] == 0
    prev = sdm.set_wait_limit(1)
    try:
        sdm.gated_delta(x["state"].clone(), *args, workspace=fws)
        assert sdm.device_status(fws)["code"] == -4                # SDM_ERR_TIMEOUT
        sdm.gated_delta_backward(*args, saved, do, grad_state=dS, workspace=bws)
        assert sdm.device_status(bws)["code"] == -4
    finally:
        assert sdm.set_wait_limit(prev) == 1
    assert torch.equal(sdm.gated_delta(x["state"].clone(), *args, workspace=fws), want)
    again = sdm.gated_delta_backward(*args, saved, do, grad_state=dS, workspace=bws)
    assert sdm.device_status(fws)["code"] == 0 and sdm.device_status(bws)["code"] == 0
    assert all(torch.equal(again[n], right[n]) for n in right)
