"""The module of the everyday calls without a device: it loads with the library and takes nothing that is not a
CUDA tensor; the number of tokens that go one by one is the kernels'."""

import os
import re

import torch

import sparse_addressed_delta_gb300 as sdm

CSRC = os.path.join(os.path.dirname(sdm.__file__), "csrc")


def test_takes_only_device_tensors():
    sdm.library()
    x = torch.randn(3, 8)
    assert sdm._fast.layer_norm(x, None, None, 1e-5, False) is None
    assert sdm._fast.layer_norm(None, None, None, 1e-5, False) is None
    assert sdm._fast.layer_norm() is None
    assert sdm._fast.layer_norm_backward(x, x, None, x, True) is None
    z = torch.zeros(1, 1, 1, 16)
    assert sdm._fast.gated_delta(torch.zeros(1, 1, 16, 16), z, z, z, z[..., 0], z[..., 0], None, None, None) is None
    assert sdm._fast.gated_delta(*range(9)) is None


def test_step_tokens_are_the_kernels():
    src = open(os.path.join(CSRC, "delta_internal.cuh")).read()
    assert int(re.search(r"kDeltaStepTokens = (\d+)", src).group(1)) == sdm.DELTA_STEP_TOKENS
