"""bfloat16 results of the gated delta rule are float32 arithmetic's, rounded once.

A result that float32 arithmetic gives with an error e before its rounding to bfloat16 goes the other way than the
exact value with probability |e| / ulp, and is then off by one ulp, at most 2^-7 of the value. So the squared
distance to the exact values rounded once is about sum |e_i| ulp_i <= 2^-7 |e| |x| (2-norms): relative to |x|, the
root of 2^-7 delta where delta is the relative error before the rounding. The float32 form's own results are off by
1.5e-7 to 2.7e-7; 4 x 2^-23 is allowed, which gives 6.1e-5. (Operands of two bfloat16 terms, 2^-18 off, give 1e-4.)"""

import pytest
import torch

import sparse_addressed_delta_gb300 as sdm
from oracle import delta as od
from test_gpu_delta import call, draw, host, ref
from test_gpu_delta_backward import grads, train

pytestmark = pytest.mark.gpu

ROUNDED = (2.0 ** -7 * 4 * 2.0 ** -23) ** 0.5


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    sdm.library()


def apart(a, exact):
    """Relative distance of bfloat16 results to the exact ones rounded once."""
    once = torch.from_numpy(exact).to(torch.bfloat16).double()
    return float((a.double().cpu() - once).norm() / once.norm())


# B, T, Hk, H, Dk, Dv: single chunks and chains, a narrow and a wide state, segments
SHAPES = [(2, 300, 2, 4, 128, 128), (4, 64, 2, 4, 64, 128), (2, 257, 1, 2, 96, 256), (1, 1500, 2, 2, 64, 128)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_readings(shape):
    x = draw(*shape, "bf16", seed=20)
    assert apart(call(x)[0], ref(x)[0]) <= ROUNDED


# many values: a value that rounds the other way is rare
GRADIENT_SHAPES = [(4, 150, 2, 4, 128, 128), (6, 100, 2, 4, 64, 128), (2, 150, 2, 2, 128, 192), (1, 1500, 2, 2, 64, 128)]


@pytest.mark.parametrize("shape", GRADIENT_SHAPES, ids=str)
def test_gradients(shape):
    """The same by sums of |differences|, of which the expectation is sum |e_i| itself: few of a gradient's values are
    large, and a sum of squares would hang on them alone. About n = 2^8 delta (sum |x|)^2 / sum x^2 equal steps make the
    sum, so 3 / sqrt(n) of it is allowed to chance."""
    x, (do, dS) = draw(*shape, "bf16", seed=21), grads(shape, "bf16")
    got = train(x, do, dS)[2]
    want = od.gated_delta_backward(**{n: host(t) for n, t in x.items()}, do=host(do), dS=host(dS), scale=shape[4] ** -0.5)
    for name in ("grad_q", "grad_k", "grad_v"):
        once = torch.from_numpy(want[name]).to(torch.bfloat16).double()
        off, size = float((got[name].double().cpu() - once).abs().sum()), float(once.abs().sum())
        delta = 4 * 2.0 ** -23
        n = 2 ** 8 * delta * size ** 2 / float(once.square().sum())
        assert off / size <= delta * (1 + 3 / n ** 0.5), name
