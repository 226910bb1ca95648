"""Norms whose result is their input's memory, and gradients in the place of the result's: the same to the bit as apart."""

import pytest
import torch

import sparse_addressed_delta_gb300 as sdm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    sdm.library()


def stream():
    return torch.cuda.current_stream().cuda_stream


# positions split over blocks, by vectors of groups and whole; a few wide positions; small samples; rows; odd channels
@pytest.mark.parametrize("shape,groups", [((2, 4000, 512), 32), ((2, 9000, 320), 32), ((5, 30, 2048), 16), ((500, 9, 40), 5), ((700, 1, 4096), 32),
                                          ((3, 3000, 33), 3)], ids=str)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_group_norm(shape, groups, dtype):
    gen = torch.Generator("cuda").manual_seed(sum(shape))
    N, L, C = shape
    x, dy = (torch.randn(*shape, device="cuda", generator=gen).to(dtype) for _ in range(2))
    w, b = (torch.randn(C, device="cuda", generator=gen) for _ in range(2))
    y, stats = sdm.group_norm_save(x, groups, w, b, activation="silu")
    want = sdm.group_norm_backward(dy, x, groups, w, b, stats, activation="silu")
    z = x.clone()
    assert sdm.group_norm(z, groups, w, b, activation="silu", out=z) is z and torch.equal(z, y)
    lib = sdm.library()
    n = lib.sdm_group_norm_backward_workspace_bytes(N, L, C, groups)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    d, dw, db = dy.clone(), torch.empty(C, device="cuda"), torch.empty(C, device="cuda")
    code = sdm.SDM_BF16 if dtype == torch.bfloat16 else sdm.SDM_F32
    assert lib.sdm_group_norm_backward(d.data_ptr(), C, x.data_ptr(), C, N, L, C, groups, w.data_ptr(), b.data_ptr(), sdm.SDM_F32, 1, stats.data_ptr(),
                                       code, d.data_ptr(), dw.data_ptr(), db.data_ptr(), ws.data_ptr(), n, stream()) == 0
    assert torch.equal(d, want["grad_x"]) and torch.equal(dw, want["grad_weight"]) and torch.equal(db, want["grad_bias"])


@pytest.mark.parametrize("rows,n", [(300, 16384), (200, 8200), (300, 1007), (3000, 128)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_layer_norm_gradient(rows, n, dtype):
    gen = torch.Generator("cuda").manual_seed(n)
    x, dy = (torch.randn(rows, n, device="cuda", generator=gen).to(dtype) for _ in range(2))
    w = torch.randn(n, device="cuda", generator=gen)
    stats = sdm.layer_norm_save(x, w)[1]
    want = sdm.layer_norm_backward(dy, x, w, stats, bias=False)
    lib = sdm.library()
    size = lib.sdm_layer_norm_workspace_bytes(rows, n)
    ws, d, dw = torch.empty(size, dtype=torch.uint8, device="cuda"), dy.clone(), torch.empty(n, device="cuda")
    code = sdm.SDM_BF16 if dtype == torch.bfloat16 else sdm.SDM_F32
    assert lib.sdm_layer_norm_backward(d.data_ptr(), n, x.data_ptr(), n, rows, n, w.data_ptr(), sdm.SDM_F32, stats.data_ptr(), code, d.data_ptr(),
                                       dw.data_ptr(), None, ws.data_ptr(), size, stream()) == 0
    assert torch.equal(d, want["grad_x"]) and torch.equal(dw, want["grad_weight"])
