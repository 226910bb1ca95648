"""Refusals of linear attention's and group norm's C ABI that need no device: the addresses here are never read, every
call returns before anything is queued. And the direct entries take nothing that is not a CUDA tensor."""

import os
import re

import pytest
import torch

import sparse_addressed_delta_gb300 as sdm

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -5
AT = 1 << 20                     # an aligned address that nothing is behind
CSRC = os.path.join(os.path.dirname(sdm.__file__), "csrc")


def shape(**kw):
    """A packed sdm_linear_shape of contiguous bfloat16 inputs."""
    grad = kw.pop("grad", [100 * 4 * 128, 4 * 128, 128])
    q = kw.pop("q", [100 * 2 * 64, 2 * 64, 64])
    order = dict(B=2, T=100, H=4, Hk=2, Dk=64, Dv=128, dtype=sdm.SDM_BF16, scale=1.0) | kw
    return sdm._LINEAR_SHAPE.pack(*order.values(), *q, 100 * 2 * 64, 2 * 64, 64, 100 * 4 * 128, 4 * 128, 128, *grad)


@pytest.mark.parametrize("change,code", [
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(Hk=3), INVALID), (dict(H=0), INVALID), (dict(dtype=7), INVALID),
    (dict(Dk=24), UNSUPPORTED), (dict(Dk=144), UNSUPPORTED), (dict(Dv=528), UNSUPPORTED), (dict(Dk=0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(q=[4, 64, 64]), INVALID), (dict(q=[-64, 64, 64]), INVALID),
    (dict(q=[1 << 40, 64, 64]), UNSUPPORTED), (dict(B=1 << 26, H=64), INVALID)], ids=str)
def test_shapes(change, code):
    lib, s = sdm.library(), shape(**change)
    assert lib.sdm_linear_attention_workspace_bytes(s) == 0 and lib.sdm_linear_attention_saved_bytes(s) == 0
    assert lib.sdm_linear_attention(s, *[AT] * 7, None, 0, None) == code and b"linear attention" in lib.sdm_last_error()
    assert lib.sdm_linear_attention_save(s, *[AT] * 7, None, 0, None, 0, None) == code
    assert lib.sdm_linear_attention_backward(s, *[AT] * 6, 0, *[AT] * 7, None, 0, None) == code


def test_pointers_and_workspaces():
    lib, s = sdm.library(), shape()
    need = lib.sdm_linear_attention_workspace_bytes(s)
    assert need > 0
    for i in (0, 1, 2, 3, 4, 6):              # state, q, k, v, log_decay, readings (valid_tokens may be NULL)
        args = [AT] * 7
        args[i] = None
        assert lib.sdm_linear_attention(s, *args, AT, need, None) == INVALID
        if i != 4:                            # (the decays' address is any float's)
            args[i] = AT + 8
            assert lib.sdm_linear_attention(s, *args, AT, need, None) == INVALID and b"aligned" in lib.sdm_last_error()
    for ws, n in ((None, need), (AT, 100), (AT + 16, need)):
        assert lib.sdm_linear_attention(s, *[AT] * 7, ws, n, None) == WORKSPACE
    assert lib.sdm_linear_attention_save(s, *[AT] * 7, AT, 64, AT, need, None) == WORKSPACE and b"saved" in lib.sdm_last_error()
    back = lib.sdm_linear_attention_backward_workspace_bytes(s)
    assert lib.sdm_linear_attention_backward(s, *[AT] * 6, 64, *[AT] * 7, AT, back, None) == WORKSPACE
    # the forward does not look at the gradient's strides
    for bad in ([-8, -8, -8], [3, 5, 7], [1 << 60, 1 << 50, 1 << 45]):
        t = shape(grad=bad)
        assert lib.sdm_linear_attention_workspace_bytes(t) == need and lib.sdm_linear_attention_backward_workspace_bytes(t) == 0


def test_group_norm():
    lib = sdm.library()

    def call(stride=64, N=4, L=9, C=64, G=4, wdt=0, eps=1e-5, act=0, dt=0, y=AT, stats=AT, ws=None, n=0, x=AT):
        return lib.sdm_group_norm(x, stride, N, L, C, G, AT, AT, wdt, eps, act, dt, y, stats, ws, n, None)

    def back(stride=64, grad=64, N=4, L=9, C=64, G=4, wdt=0, act=0, dt=0, stats=AT, ws=None, n=0, dx=AT):
        return lib.sdm_group_norm_backward(AT, grad, AT, stride, N, L, C, G, AT, AT, wdt, act, stats, dt, dx, AT, AT, ws, n, None)

    for fn in (call, back):
        for bad in (dict(N=-1), dict(L=-1), dict(C=0), dict(G=0), dict(G=5), dict(stride=-1), dict(act=2), dict(dt=9), dict(wdt=1), dict(stats=AT + 4)):
            assert fn(**bad) == INVALID, bad
        for bad in (dict(C=16400), dict(N=1 << 24), dict(L=1 << 31)):
            assert fn(**bad) == UNSUPPORTED, bad
        for bad in (dict(), dict(ws=AT, n=16), dict(ws=AT + 8, n=1 << 20)):
            assert fn(**bad) == WORKSPACE
    assert call(eps=-1.0) == INVALID and call(eps=float("nan")) == INVALID and call(x=None) == INVALID and call(y=None) == INVALID
    assert back(grad=-1) == INVALID and back(stats=None) == INVALID and back(dx=None) == INVALID
    for query in (lib.sdm_group_norm_workspace_bytes, lib.sdm_group_norm_backward_workspace_bytes):
        assert query(4, 9, 64, 4) > 0 and query(4, 9, 64, 5) == 0 and query(-1, 9, 64, 4) == 0


def test_direct_entries_take_only_device_tensors():
    sdm.library()
    x, z = torch.randn(3, 8), torch.zeros(1, 1, 1, 16)
    assert sdm._fast.group_norm(x, 2, None, None, None, 1e-5, False) is None and sdm._fast.group_norm() is None
    assert sdm._fast.group_norm_backward(x, x, 2, None, None, x, None) is None
    assert sdm._fast.linear_attention(torch.zeros(1, 1, 16, 16), z, z, z, z[0, 0, 0, :1], None, None, None, False) is None
    assert sdm._fast.linear_attention(*range(9)) is None and sdm._fast.linear_attention_backward(*range(10)) is None


def test_step_tokens_are_the_kernels():
    src = open(os.path.join(CSRC, "linear_internal.cuh")).read()
    assert int(re.search(r"kLinearStepTokens = (\d+)", src).group(1)) == sdm.LINEAR_STEP_TOKENS
