"""The status block of a given workspace is that of the last call, whatever form the call takes."""

import pytest
import torch

import sparse_addressed_delta_gb300 as sdm
from test_gpu_delta import call, draw
from test_gpu_delta_backward import grads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    sdm.library()


def stale(n=1 << 20):
    """A workspace in which an earlier call left something."""
    return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("B,T", [(2, 1), (2, 8), (2, 9), (2, 0), (0, 5)])
def test_cleared_by_every_forward(B, T):
    x = draw(B, T, 1, 2, 32, 32, "bf16", seed=50)
    ws = stale()
    o, state = call(x, workspace=ws)
    assert sdm.device_status(ws) == {"code": 0, "first_bad_token": -1, "bad_slots": 0, "repeated_write_slots": 0}
    want = call(x)
    assert torch.equal(o, want[0]) and torch.equal(state, want[1])


@pytest.mark.parametrize("B,T", [(2, 3), (2, 0), (0, 5)])
def test_cleared_by_every_save_and_backward(B, T):
    shape = (B, T, 1, 2, 32, 32)
    x, (do, dS) = draw(*shape, "f32", seed=51), grads(shape, "f32")
    args = (x["q"], x["k"], x["v"], x["g"], x["beta"], None)
    ws = stale()
    saved = sdm.gated_delta_save(x["state"].clone(), *args, workspace=ws)[1]
    assert sdm.device_status(ws)["code"] == 0
    ws = stale()
    sdm.gated_delta_backward(*args, saved, do, grad_state=dS, workspace=ws)
    assert sdm.device_status(ws)["code"] == 0


def test_a_short_call_takes_a_workspace_too_small_for_a_status():
    x = draw(1, 2, 1, 1, 32, 32, "f32", seed=52)
    ws = stale(64)
    call(x, workspace=ws)
    assert (ws == 0xFF).all()
