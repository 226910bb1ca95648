"""Refusals of the layer norm's and the gated delta rule's C ABI that need no device: the addresses here are never
read, every call returns before anything is queued."""

import sparse_addressed_delta_gb300 as sdm

INVALID = -1
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
