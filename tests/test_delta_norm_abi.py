"""Refusals of the layer norm's and the gated delta rule's C ABI that need no device: the addresses here are never
read, every call returns before anything is queued."""

import pytest
import torch

import sparse_addressed_delta_gb300 as sdm

INVALID, WORKSPACE = -1, -5
AT = 1 << 20                     # an aligned address that nothing is behind


def test_stats_alignment():
    """A row's (mean, rstd) is one 8-byte value."""
    lib = sdm.library()
    for off in (1, 2, 4, 12):
        assert lib.sdm_layer_norm(AT, 3, 64, 64, None, None, sdm.SDM_F32, 1e-5, sdm.SDM_F32, AT, AT + off, None) == INVALID
        assert b"8-byte" in lib.sdm_last_error()
        assert lib.sdm_layer_norm_backward(AT, 64, AT, 64, 3, 64, None, sdm.SDM_F32, AT + off, sdm.SDM_F32, AT, None, None, None,
                                           0, None) == INVALID
        assert b"8-byte" in lib.sdm_last_error()


def shape(**kw):
    """A packed sdm_delta_shape of contiguous bfloat16 inputs."""
    order = dict(B=2, T=100, H=4, Hk=2, Dk=64, Dv=128, dtype=sdm.SDM_BF16, scale=1.0) | {n: kw.pop(n) for n in list(kw) if n != "grad"}
    qk, v, gate = [100 * 2 * 64, 2 * 64, 64], [100 * 4 * 128, 4 * 128, 128], [400, 4, 1]
    return sdm._DELTA_SHAPE.pack(*order.values(), *qk, *qk, *v, *gate, *gate, *kw.get("grad", v))


def test_the_forward_ignores_the_gradients_strides():
    """They may be unset: the forward, its size queries and what it saves do not depend on them; the backward refuses."""
    lib = sdm.library()
    for bad in ([-8, -8, -8], [3, 5, 7], [1 << 60, 1 << 50, 1 << 45]):
        s = shape(grad=bad)
        assert lib.sdm_gated_delta_workspace_bytes(s) == lib.sdm_gated_delta_workspace_bytes(shape()) > 0
        assert lib.sdm_gated_delta_saved_bytes(s) == lib.sdm_gated_delta_saved_bytes(shape()) > 0
        # past the shape's check, to the missing workspace's
        assert lib.sdm_gated_delta(s, *[AT] * 8, None, 0, None) == WORKSPACE and b"workspace" in lib.sdm_last_error()
        assert lib.sdm_gated_delta_save(s, *[AT] * 8, None, 0, None, 0, None) == WORKSPACE
        assert lib.sdm_gated_delta_backward_workspace_bytes(s) == 0
        assert lib.sdm_gated_delta_backward(s, *[AT] * 6, AT, 0, *[AT] * 8, None, 0, None) < 0


class DeviceLike(torch.Tensor):
    """A tensor without storage that says it is on a device."""
    is_cuda = True


@pytest.mark.parametrize("n", [2 ** 31, 2 ** 32 + 128])
def test_more_columns_than_an_int(n):
    """Refused as too many columns are, not taken as what an int keeps of them (128)."""
    x = torch.empty((1, n), device="meta").as_subclass(DeviceLike)
    for fn in (sdm.layer_norm, sdm.layer_norm_save):
        with pytest.raises(sdm.SdmError, match="columns"):
            fn(x)
    with pytest.raises(sdm.SdmError, match="columns"):
        sdm.layer_norm_backward(x, x, None, torch.empty((1, 2), device="meta"))
