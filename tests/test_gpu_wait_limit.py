"""With a limit of one poll every kernel with bounded waits gives up at every call, also where what it waits for has long been
there: sizes at which the copies are fast, data that lies in the cache, many calls."""

import pytest
import torch

import sdm_inputs as si
import sparse_addressed_delta_gb300 as sdm
from sdm_case import run_gpu, small_workload, to_device

pytestmark = pytest.mark.gpu
TIMEOUT = -4


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    sdm.library()


def codes(call, ws, many):
    prev = sdm.set_wait_limit(1)
    try:
        got = []
        for _ in range(many):
            call()
            got.append(sdm.device_status(ws)["code"])
        return got
    finally:
        assert sdm.set_wait_limit(prev) == 1


@pytest.mark.parametrize("T,C,dtype,flags", [(8 * 64, 64, "bf16", 0), (64, 64, "bf16", 0), (2 * 128, 128, "f32", 0), (2 * 128, 128, "bf16", 1)], ids=str)
def test_write_read(T, C, dtype, flags):
    """The pipelined Phase 2 with many steps, with one, and the dual product's kernel."""
    wl = small_workload(P=2, T=T, C=C, S=4096, D=128, W=16, R=16, dtype=dtype, slots="zipf1.1", ragged=False, seed=51)
    dev = to_device(si.generate(wl), wl)
    _, _, ws = run_gpu(wl, dev, flags=flags)
    assert sdm.device_status(ws)["code"] == 0
    got = codes(lambda: run_gpu(wl, dev, workspace=ws, flags=flags), ws, 100)
    assert got == [TIMEOUT] * 100, got
    run_gpu(wl, dev, workspace=ws, flags=flags)
    assert sdm.device_status(ws)["code"] == 0


@pytest.mark.parametrize("T", [65, 2000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_recurrences(T, dtype):
    q, v = torch.randn(1, T, 1, 64, device="cuda").to(dtype) / 8, torch.randn(1, T, 1, 64, device="cuda").to(dtype)
    decay, beta, state = torch.full((1, T, 1), -0.1, device="cuda"), torch.full((1, T, 1), 0.5, device="cuda"), torch.zeros(1, 1, 64, 64, device="cuda")
    lib = sdm.library()
    ws = torch.empty(lib.sdm_linear_attention_workspace_bytes(sdm._linear_shape(q, q, v, decay[0, 0], None, None)[0]), dtype=torch.uint8, device="cuda")
    call = lambda: sdm.linear_attention(state, q, q, v, decay[0, 0], workspace=ws)  # noqa: E731
    call()
    assert sdm.device_status(ws)["code"] == 0 and codes(call, ws, 100) == [TIMEOUT] * 100
    call()
    assert sdm.device_status(ws)["code"] == 0
    if dtype == torch.float32:                 # the delta rule's scan waits on the tensor cores for bfloat16 inputs alone
        return
    ws = torch.empty(lib.sdm_gated_delta_workspace_bytes(sdm._delta_shape(q, q, v, decay, beta, None, None)[0]), dtype=torch.uint8, device="cuda")
    call = lambda: sdm.gated_delta(state, q, q, v, decay, beta, workspace=ws)  # noqa: E731
    call()
    assert sdm.device_status(ws)["code"] == 0 and codes(call, ws, 100) == [TIMEOUT] * 100
    call()
    assert sdm.device_status(ws)["code"] == 0
