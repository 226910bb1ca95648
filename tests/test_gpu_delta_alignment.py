"""The gradient of the final state at any address of a float: it is the caller's own buffer, often a view into
another."""

import pytest
import torch

import sparse_addressed_delta_gb300 as sdm
from test_gpu_delta import draw
from test_gpu_delta_backward import grads, train

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    sdm.library()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1500, 1, 2, 64, 128), (1, 100, 1, 2, 64, 128)], ids=["segments", "one run"])
@pytest.mark.parametrize("offset", [1, 2, 3])
def test_the_final_states_gradient_at_an_odd_address(dtype, shape, offset):
    x, (do, dS) = draw(*shape, dtype, seed=40, decay=0.001), grads(shape, dtype)
    view = torch.empty(dS.numel() + offset, device="cuda")[offset:].view_as(dS)
    view.copy_(dS)
    assert view.data_ptr() % 16 == 4 * offset
    want, got = train(x, do, dS)[2], train(x, do, view)[2]
    assert all(torch.equal(got[n], want[n]) for n in want)
