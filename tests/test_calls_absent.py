"""The module of the everyday calls saves host time and nothing else: without it, or without Python's headers, the
package builds and loads, and the binding makes those calls by itself."""

import os
import subprocess
import sys
import sysconfig

import pytest
import torch

import sparse_addressed_delta_gb300 as sdm
from sparse_addressed_delta_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_package_loads_without_it():
    code = ("import sparse_addressed_delta_gb300 as sdm\n"
            "sdm._calls_path = '/nonexistent'\n"
            "sdm.library()\n"
            "assert sdm.version() and sdm._fast.layer_norm(1, 2, 3, 4, 5) is None and sdm._fast.gated_delta() is None\n")
    subprocess.run([sys.executable, "-c", code], cwd=ROOT, check=True)


def test_it_is_built_where_pythons_headers_are(monkeypatch, tmp_path):
    target = str(tmp_path / "calls.so")
    monkeypatch.setattr(_build, "CALLS", target)
    monkeypatch.setattr(_build, "_headers", lambda: None)
    assert _build.build_calls() is None and not os.listdir(tmp_path)
    # nothing is stale for want of it
    lib = tmp_path / "libsdm.so"
    lib.write_bytes(b"")
    monkeypatch.setattr(_build, "LIB", str(lib))
    assert _build.build() == str(lib)


def test_it_is_named_for_the_interpreter():
    suffix = sysconfig.get_config_var("EXT_SUFFIX")
    assert sdm._calls_path == _build.CALLS and _build.CALLS.endswith("_calls" + suffix) and "cpython" in suffix


@pytest.mark.gpu
def test_the_same_results_without_it(monkeypatch):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from test_gpu_delta import call, draw
    sdm.library()
    x = draw(2, 20, 1, 2, 32, 48, "bf16", seed=70)
    w = torch.randn(48, device="cuda")

    def all_of_it():
        o, state = call(x)
        y, stats = sdm.layer_norm_save(o, w)
        return [o, state, y, stats, sdm.layer_norm(o, w), *sdm.layer_norm_backward(o, o, w, stats, bias=False).values()]

    want = all_of_it()
    monkeypatch.setattr(sdm, "_fast", sdm._NoCalls)
    assert all(torch.equal(a, b) for a, b in zip(all_of_it(), want, strict=True))
