"""Linear attention's status block: cleared by every call with a workspace, and set by bounded waits that give up (a limit
of one poll), after which nothing has faulted and the next call with the default limit is right. And calls at once."""

import pytest
import torch

import sparse_addressed_delta_gb300 as sdm
from test_gpu_linear import draw, lengths
from test_gpu_linear_backward import grads_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    sdm.library()


def spaces(x, do):
    """Workspaces of the forward and the backward in which an earlier call left something."""
    packed = sdm._linear_shape(x["q"], x["k"], x["v"], x["g"], None, None, do)[0]
    lib = sdm.library()
    return [torch.full((n(packed),), 0xFF, dtype=torch.uint8, device="cuda")
            for n in (lib.sdm_linear_attention_workspace_bytes, lib.sdm_linear_attention_backward_workspace_bytes)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [100, 900])
def test_waits_give_up_and_recover(dtype, T):
    """T = 900: in segments, so that a carry gives up and the launches behind it find that it has."""
    x = draw(2, T, 1, 2, 64, 128, dtype, seed=30)
    do, dS = grads_of(x, dtype, 31)
    args = (x["q"], x["k"], x["v"], x["g"], None)
    fws, bws = spaces(x, do)
    want, saved = sdm.linear_attention_save(x["state"].clone(), *args, workspace=fws)
    assert sdm.device_status(fws)["code"] == 0
    right = sdm.linear_attention_backward(*args, saved, do, grad_state=dS, workspace=bws)
    assert sdm.device_status(bws)["code"] == 0
    prev = sdm.set_wait_limit(1)
    try:
        sdm.linear_attention(x["state"].clone(), *args, workspace=fws)
        assert sdm.device_status(fws)["code"] == -4                # SDM_ERR_TIMEOUT
        sdm.linear_attention_backward(*args, saved, do, grad_state=dS, workspace=bws)
        assert sdm.device_status(bws)["code"] == -4
    finally:
        assert sdm.set_wait_limit(prev) == 1
    assert torch.equal(sdm.linear_attention(x["state"].clone(), *args, workspace=fws), want)
    assert sdm.device_status(fws)["code"] == 0
    again = sdm.linear_attention_backward(*args, saved, do, grad_state=dS, workspace=bws)
    assert sdm.device_status(bws)["code"] == 0 and all(torch.equal(again[n], right[n]) for n in right)


@pytest.mark.parametrize("B,T", [(2, 1), (2, 12), (2, 13), (2, 0), (0, 5)])
def test_cleared(B, T):
    x = draw(B, T, 1, 2, 32, 32, "bf16", seed=32)
    do, dS = grads_of(x, "bf16", 33)
    args = (x["q"], x["k"], x["v"], x["g"], lengths([T, T // 2][:B]))
    fws, bws = spaces(x, do)
    state = x["state"].clone()
    o = sdm.linear_attention(state, *args, workspace=fws)
    assert sdm.device_status(fws) == {"code": 0, "first_bad_token": -1, "bad_slots": 0, "repeated_write_slots": 0}
    other = x["state"].clone()
    assert torch.equal(o, sdm.linear_attention(other, *args)) and torch.equal(state, other)
    saved = sdm.linear_attention_save(x["state"].clone(), *args, workspace=fws)[1]
    sdm.linear_attention_backward(*args, saved, do, grad_state=dS, workspace=bws)
    assert sdm.device_status(fws)["code"] == 0 and sdm.device_status(bws)["code"] == 0


def test_calls_at_once():
    """Two training steps on two streams, and two graphs of steps replayed at once."""
    xs = [draw(2, 700, 1, 2, 64, 128, "bf16", seed=s) for s in (34, 35)]
    sides = [torch.cuda.Stream() for _ in xs]

    def step(x, do, dS):
        args = (x["q"], x["k"], x["v"], x["g"], None)
        state = x["state"].clone()
        o, saved = sdm.linear_attention_save(state, *args)
        return [o, state, *sdm.linear_attention_backward(*args, saved, do, grad_state=dS).values()]

    ins = [(x, *grads_of(x, "bf16", 36)) for x in xs]
    want = [step(*i) for i in ins]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(3):
        for i, side in enumerate(sides):
            with torch.cuda.stream(side):
                got[i] = step(*ins[i])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))
    graphs, outs = [], []
    for i in ins:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(step(*i))
    for graph, side in zip(graphs, sides):
        with torch.cuda.stream(side):
            graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g, w in zip(outs, want) for a, b in zip(g, w))


def test_deterministic_and_repeated():
    x = draw(3, 300, 2, 4, 128, 256, "bf16", seed=37)
    do, dS = grads_of(x, "bf16", 38)
    args = (x["q"], x["k"], x["v"], x["g"], lengths([300, 200, 65]))
    saved = sdm.linear_attention_save(x["state"].clone(), *args)[1]
    first = sdm.linear_attention_backward(*args, saved, do, grad_state=dS)
    for _ in range(5):
        again = sdm.linear_attention_backward(*args, saved, do, grad_state=dS)
        assert all(torch.equal(again[n], first[n]) for n in first)
