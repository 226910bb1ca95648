"""The norms' and linear attention's launches, read from the source: every launch's result is looked at before the next one is
made, so that none follows one that failed (it would read what that one has not written)."""

import os
import re

import pytest

import sparse_addressed_delta_gb300 as sdm

CSRC = os.path.join(os.path.dirname(sdm.__file__), "csrc")
FILES = ["group_norm.cu", "norm.cu", "linear.cu", "linear_step.cu", "linear_scan_tc.cu", "linear_carry_tc.cu", "linear_decay_tc.cu"]


@pytest.mark.parametrize("name", FILES)
def test_every_launch_is_looked_at(name):
    src = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    statements = re.split(r"[;{}]", src)
    for i, s in enumerate(statements):
        if "<<<" in s:
            # the last launch of a branch may be looked at behind it
            rest = [t.strip() for t in statements[i + 1:i + 7] if t.strip()]
            looked = next((k for k, t in enumerate(rest) if "cudaGetLastError()" in t), None)
            assert looked is not None and all("launch" not in t for t in rest[:looked]), s
        for call in re.finditer(r"\b(chain_launch|launch_linear_\w+)\(", s):
            before = s[:call.start()].rstrip()
            assert "cudaError_t" in before or before.endswith(("return", "=", "?", ":")), s
