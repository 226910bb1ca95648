"""The bounded waits of the gated delta rule's tensor-core kernels: with a limit of one poll they give up,
set SDM_ERR_TIMEOUT in the workspace's status block and return; nothing faults, and the next call with the
default limit is right."""

import ctypes

import pytest
import torch

import sparse_addressed_delta_gb300 as sdm
from test_gpu_delta import call, draw, host, err, TOL, F32_TOL, ref
from test_gpu_delta_backward import grads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    sdm.library()


def test_forward_and_backward_give_up_and_recover():
    shape = (2, 200, 1, 2, 64, 128)
    x, (do, dS) = draw(*shape, "bf16", seed=3), grads(shape, "bf16")
    args = (x["q"], x["k"], x["v"], x["g"], x["beta"], None)
    packed = sdm._delta_shape(*args, None, do)[0]
    lib = sdm.library()
    fws = torch.empty(lib.sdm_gated_delta_workspace_bytes(packed), dtype=torch.uint8, device="cuda")
    bws = torch.empty(lib.sdm_gated_delta_backward_workspace_bytes(packed), dtype=torch.uint8, device="cuda")
    want, saved = sdm.gated_delta_save(x["state"].clone(), *args, workspace=fws)
    assert sdm.device_status(fws)["code"] == 0
    right = sdm.gated_delta_backward(*args, saved, do, grad_state=dS, workspace=bws)
    assert sdm.device_status(bws)["code"] == 0
    prev = sdm.set_wait_limit(1)
    try:
        sdm.gated_delta(x["state"].clone(), *args, workspace=fws)
        assert sdm.device_status(fws)["code"] == -4                # SDM_ERR_TIMEOUT
        sdm.gated_delta_backward(*args, saved, do, grad_state=dS, workspace=bws)
        assert sdm.device_status(bws)["code"] == -4
    finally:
        assert sdm.set_wait_limit(prev) == 1
    o, state = call(x, workspace=fws)
    assert sdm.device_status(fws)["code"] == 0
    ro, rs = ref(x)
    assert torch.equal(o, want) and err(o, ro) <= TOL["bf16"] and err(state, rs) <= F32_TOL
    again = sdm.gated_delta_backward(*args, saved, do, grad_state=dS, workspace=bws)
    assert sdm.device_status(bws)["code"] == 0 and all(torch.equal(again[n], right[n]) for n in right)


def test_workspace_sizes_are_refused_and_host_only():
    """The size queries and the refusals that need no device."""
    lib = sdm.library()
    pack = lambda **kw: sdm._DELTA_SHAPE.pack(*[kw.get(n, d) for n, d in (  # noqa: E731
        ("B", 2), ("T", 100), ("H", 4), ("Hk", 2), ("Dk", 64), ("Dv", 128), ("dtype", sdm.SDM_BF16), ("scale", 1.0))], *kw.get("strides", [0] * 18))
    assert lib.sdm_gated_delta_workspace_bytes(pack()) > 0
    for bad in (dict(B=-1), dict(T=-1), dict(H=3), dict(Hk=0), dict(Dk=24), dict(Dk=144), dict(Dv=8), dict(Dv=1024), dict(dtype=7),
                dict(scale=float("nan")), dict(strides=[4] + [0] * 17), dict(strides=[0] * 9 + [-8] + [0] * 8), dict(B=1 << 30)):
        assert lib.sdm_gated_delta_workspace_bytes(pack(**bad)) == 0, bad
        assert lib.sdm_gated_delta(pack(**bad), *[None] * 8, None, 0, None) < 0
        assert lib.sdm_last_error()
    assert lib.sdm_gated_delta(pack(), *[None] * 8, None, 0, None) == -1
    assert lib.sdm_gated_delta(None, *[None] * 8, None, 0, None) == -1
    assert ctypes.sizeof(ctypes.c_char * sdm._DELTA_SHAPE.size) == 7 * 4 + 4 + 18 * 8
