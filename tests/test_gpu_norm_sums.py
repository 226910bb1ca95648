"""The norm's column sums (the gradients of weight and bias) are as exact as sums in pairs.

A rounding is off by u = 2.4e-8 of the value (root mean square: half a unit over sqrt(3), the unit between 2^-24 and
2^-23 of the value). Sums of independent terms grow as the root of their number, so a run of n terms gives an error of
u sqrt(n / 2), and a level of pairs one of u, of the whole. With 5003 rows: 6 rows a block, 13 blocks a run, 64 runs in
6 levels, u sqrt(3 + 6.5 + 6) = 9.4e-8; the terms' own three roundings add 4.2e-8. That is 1.03e-7, and 1.25e-7 with
a fifth for chance. (64 runs one after the other give 1.6e-7; runs and pairs that keep what their roundings lose, below
1e-7.)"""

import pytest
import torch

import sparse_addressed_delta_gb300 as sdm
from oracle import delta as od

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    sdm.library()


def test_infinite_sums():
    x, dy = torch.randn(700, 40, device="cuda"), torch.randn(700, 40, device="cuda")
    dy[300, 5], dy[10, 7], dy[11, 7], dy[12, 9], dy[13:15, 11] = torch.inf, torch.inf, -torch.inf, torch.nan, 3e38
    got = sdm.layer_norm_backward(dy, x, None, sdm.layer_norm_save(x)[1])["grad_bias"]
    assert got[5] == torch.inf and got[7].isnan() and got[9].isnan() and got[11] == torch.inf
    assert torch.isfinite(got).sum() == 36


@pytest.mark.parametrize("seed", [1, 2, 3])
def test_error_of_the_column_sums(seed):
    gen = torch.Generator().manual_seed(seed)
    x, dy = (torch.randn(5003, 1007, generator=gen) for _ in range(2))
    want = od.layer_norm_backward(dy.double().numpy(), x.double().numpy())
    x, dy = x.cuda(), dy.cuda()
    w = torch.ones(1007, device="cuda")
    got = sdm.layer_norm_backward(dy, x, w, sdm.layer_norm_save(x, w)[1])
    for name in ("grad_weight", "grad_bias"):
        ref = torch.from_numpy(want[name])
        assert float((got[name].double().cpu() - ref).norm() / ref.norm()) <= 1.25e-7, name
