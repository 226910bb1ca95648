"""Group norm of more than 2^23 tokens. Rows need nothing of each other, so they are those of a call of some of them, to the
bit. The column sums are in float32: a thread's sums of up to N / (blocks x 128) rows, a block's 128 threads, then the blocks'
with their lost parts kept; each addition is off by at most 2^-24 of the magnitudes so far. The sums' terms are off by what
xhat is, 4e-6 of max |x| rstd."""

import pytest
import torch

import sparse_addressed_delta_gb300 as sdm

pytestmark = pytest.mark.gpu
N = (1 << 24) + 3


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    sdm.library()


@pytest.mark.parametrize("groups", [1, 2])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_tokens(dtype, groups):
    gen = torch.Generator("cuda").manual_seed(5)
    x, dy = ((torch.randn(N, 4, device="cuda", generator=gen) + 0.3).to(dtype) for _ in range(2))
    w, b = (torch.randn(4, device="cuda", generator=gen) for _ in range(2))
    for act in ("silu", None):
        y, stats = sdm.group_norm_save(x, groups, w, b, activation=act)
        got = sdm.group_norm_backward(dy, x, groups, w, b, stats, activation=act)
        for at in (slice(0, 1000), slice((1 << 23) - 500, (1 << 23) + 500), slice(N - 1000, N)):
            part, st = sdm.group_norm_save(x[at], groups, w, b, activation=act)
            assert torch.equal(y[at], part) and torch.equal(stats[at], st)
            assert torch.equal(got["grad_x"][at], sdm.group_norm_backward(dy[at], x[at], groups, w, b, st, activation=act)["grad_x"])
    # without an activation dz = dy
    h = x.double().unflatten(1, (groups, -1))
    top = h.abs().amax(2, keepdim=True)
    h = h - h.mean(2, keepdim=True)
    rstd = (h.square().mean(2, keepdim=True) + 1e-5).rsqrt()
    h, doubt = (h * rstd).flatten(1), (4e-6 * top * rstd).expand_as(h).flatten(1)
    d = dy.double()
    adds = (N // (152 * 128) + 128 + 64) * 2.0 ** -24
    assert ((got["grad_weight"].double() - (d * h).sum(0)).abs() <= adds * (d * h).abs().sum(0) + (d.abs() * doubt).sum(0)).all()
    assert ((got["grad_bias"].double() - d.sum(0)).abs() <= adds * d.abs().sum(0)).all()


def test_samples_of_several_positions_are_refused():
    x = torch.zeros((1 << 23) + 1, 2, 2, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(sdm.SdmError, match="at most 2"):
        sdm.group_norm(x, 1)
    assert sdm.group_norm(x[:, :0], 1).numel() == 0
