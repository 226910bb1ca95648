"""Which loads the norms' kernels may use, read from the source: the read-only path (__ldg) holds only for memory that nobody
writes while the reading kernel lives, and compilers move such loads across waits."""

import os
import re

import pytest

import sparse_addressed_delta_gb300 as sdm

CSRC = os.path.join(os.path.dirname(sdm.__file__), "csrc")


def body(name):
    """The source of the one function of that name, from its name to the brace that closes it."""
    src = "".join(re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, f)).read()) for f in ("norm_rows.cuh", "group_norm.cu", "norm.cu"))
    found = re.findall(rf"\b{name}\((?:const |[A-Z]\w* |int |bool )", src)
    assert len(found) == 1, f"{name}: {len(found)} definitions"
    at = src.index(found[0])
    at = end = src.index("{", at)
    depth = 0
    while True:
        depth += {"{": 1, "}": -1}.get(src[end], 0)
        end += 1
        if depth == 0:
            return src[at:end]


@pytest.mark.parametrize("name", ["k_group_join", "k_group_terms", "norm_cols"])
def test_behind_another_launch(name):
    """These begin while the launch that writes what they read still runs."""
    text = body(name)
    assert "__ldcg(" in text and "__ldg(" not in text


@pytest.mark.parametrize("name", ["k_group_apply", "k_group_apply_bwd", "k_group_small", "k_group_small_bwd", "load_row"])
def test_of_what_the_kernel_may_overwrite(name):
    """y may be x, and x's gradient y's: such a kernel stores where it has read."""
    assert "__ldg(" not in body(name)
