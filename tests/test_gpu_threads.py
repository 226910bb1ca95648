"""Host threads that call at once. A kernel's limit of dynamic shared memory belongs to the kernel, so to all threads: a
call of narrow rows must not lower it between another thread's setting of it and that thread's launch."""

import threading

import pytest
import torch

import sparse_addressed_delta_gb300 as sdm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    sdm.library()


def group(n, gen):
    """Rows of one group: a block's threads, and its shared memory, by their width."""
    x, dy = (torch.randn(48, n, device="cuda", generator=gen) for _ in range(2))
    w = torch.randn(n, device="cuda", generator=gen)

    def call():
        y, stats = sdm.group_norm_save(x, 1, w, w, activation="silu")
        return [y, stats, *sdm.group_norm_backward(dy, x, 1, w, w, stats, activation="silu").values()]

    return call


def group_split(n, gen):
    """Positions split over blocks, a block's shared memory by the channels."""
    x, dy = (torch.randn(2, 80, n, device="cuda", generator=gen) for _ in range(2))

    def call():
        y, stats = sdm.group_norm_save(x, 1)
        return [y, stats, sdm.group_norm_backward(dy, x, 1, None, None, stats)["grad_x"]]

    return call


def layer(n, gen):
    x, dy = (torch.randn(48, n, device="cuda", generator=gen) for _ in range(2))
    w = torch.randn(n, device="cuda", generator=gen)

    def call():
        y, stats = sdm.layer_norm_save(x, w, w)
        return [y, stats, *sdm.layer_norm_backward(dy, x, w, stats).values()]

    return call


@pytest.mark.parametrize("make,widths", [(group, (8192, 2624)), (layer, (8192, 3008)), (group_split, (16381, 7001))],
                         ids=["group norm rows", "layer norm rows", "group norm maps"])
def test_widths_of_two_threads(make, widths):
    gen = torch.Generator("cuda").manual_seed(1)
    calls = [make(n, gen) for n in widths]
    want = [call() for call in calls]
    torch.cuda.synchronize()
    wrong = []

    def loop(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(1500):
                try:
                    got = calls[i]()
                except sdm.SdmError as e:
                    wrong.append(str(e))
                    continue
                if _ % 50 == 0 and not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    wrong.append(f"results of width {widths[i]}")

    threads = [threading.Thread(target=loop, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong, (len(wrong), wrong[:3])
