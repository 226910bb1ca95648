"""The norms' launches behind one another: calls one behind the other in one workspace, each with other inputs, are the
same to the bit as calls with a workspace of their own, so none reads what an earlier call left there."""

import pytest
import torch

import sparse_addressed_delta_gb300 as sdm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    sdm.library()


# positions split over many blocks, over few; loaded whole by channels; small samples; rows
@pytest.mark.parametrize("shape,groups", [((2, 4000, 512), 32), ((300, 40, 256), 8), ((2, 9000, 320), 32), ((500, 9, 40), 5), ((2000, 1, 4096), 32)], ids=str)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_one_workspace_for_many_calls(shape, groups, dtype):
    gen = torch.Generator("cuda").manual_seed(sum(shape))
    normal = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    w, b = 1 + 0.1 * normal(shape[-1]), 0.1 * normal(shape[-1])
    calls = [((scale * normal(*shape) + scale).to(dtype), normal(*shape).to(dtype)) for scale in (1.0, 100.0, 0.01)]
    lib = sdm.library()
    N, C = shape[0], shape[-1]
    L = shape[1]
    ws, bws = (torch.full((n(N, L, C, groups),), 0xFF, dtype=torch.uint8, device="cuda")
               for n in (lib.sdm_group_norm_workspace_bytes, lib.sdm_group_norm_backward_workspace_bytes))

    def step(x, dy, ws=None, bws=None):
        y, stats = sdm.group_norm_save(x, groups, w, b, activation="silu", workspace=ws)
        return [y, stats, *sdm.group_norm_backward(dy, x, groups, w, b, stats, activation="silu", workspace=bws).values()]

    want = [step(*c) for c in calls]
    got = [(i, step(*calls[i], ws, bws)) for _ in range(5) for i in range(3)]   # none waited for
    for i, g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want[i]))
