"""The log-decays' gradient where the decays are strong, against the float64 reverse mode.

The gradient of a log-decay is proportional to the decay itself: everything in it crosses the token. So it has the
file's tolerance (1e-4, a sum over the chunk of float32 products that partly cancel) of the largest of its own
sequence and head, however strong the decays, and is 0 where the state is forgotten whole."""

import numpy as np
import pytest
import torch

import sparse_addressed_delta_gb300 as sdm
from oracle import delta as od
from test_gpu_delta import draw, host
from test_gpu_delta_backward import GATE, grads, train

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    sdm.library()


def check(x, do, dS):
    """The gradient, its errors over the largest of each sequence and head, and the reference."""
    got = host(train(x, do, dS)[2]["grad_log_decay"])
    want = od.gated_delta_backward(**{n: host(t) for n, t in x.items()}, do=host(do), dS=host(dS),
                                   scale=x["q"].shape[-1] ** -0.5)["grad_log_decay"]
    off = np.abs(got - want).max(1) / np.maximum(np.abs(want).max(1), 1e-30)
    assert off.max() <= GATE, off
    return got


# the register kernels' and the tensor cores', more than 128 value columns, shared keys
SHAPES = [(2, 100, 1, 2, 128, 128), (1, 70, 2, 2, 64, 192), (1, 150, 2, 4, 48, 64)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("g", [-6.0, -10.0, -16.0])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_every_token_decays_alike(dtype, g, shape):
    x, (do, dS) = draw(*shape, dtype, seed=30), grads(shape, dtype)
    x["g"].fill_(g)
    check(x, do, dS)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_heads_of_their_own_decay(dtype, shape):
    """One head that keeps, one that forgets: the second's gradient is not the first's rounding."""
    x, (do, dS) = draw(*shape, dtype, seed=31, decay=0.01), grads(shape, dtype)
    x["g"][:, :, 1] = -8.0 + x["g"][:, :, 1]
    check(x, do, dS)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_resets_have_no_gradient(dtype, shape):
    x, (do, dS) = draw(*shape, dtype, seed=32, decay=0.5), grads(shape, dtype)
    reset = torch.rand(x["g"].shape, generator=torch.Generator().manual_seed(33)).cuda() < 0.2
    reset[:, :, 1] = True
    x["g"][reset] = -torch.inf
    got = check(x, do, dS)
    assert not got[host(reset) > 0].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_long_sequences(dtype):
    shape = (1, 1600, 1, 2, 128, 128)
    x, (do, dS) = draw(*shape, dtype, seed=34, decay=0.001), grads(shape, dtype)
    x["g"][:, :, 1] = -9.0
    x["g"][:, 777, 0] = -torch.inf
    assert check(x, do, dS)[0, 777, 0] == 0
