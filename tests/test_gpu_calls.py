"""The everyday calls' own entry (csrc/calls.cpp) beside the Python binding's checked path, which a call with a
workspace, an output or rows out of order takes: the same results to the bit, on any stream."""

import pytest
import torch

import sparse_addressed_delta_gb300 as sdm
from test_gpu_delta import draw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    sdm.library()


def taken(name, *args):
    """What the direct entry answers; it has to take the call."""
    out = getattr(sdm._fast, name)(*args)
    assert out is not None
    return out


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 16, 17, 90])
def test_gated_delta(dtype, T):
    x = draw(3, T, 2, 4, 64, 96, dtype, seed=T)
    wide = torch.zeros(3, T, 8, 96, dtype=x["v"].dtype, device="cuda")       # values inside wider rows, gates by head
    wide[:, :, 2:6] = x["v"]
    args = (x["q"], x["k"], wide[:, :, 2:6], x["g"].transpose(1, 2).contiguous().transpose(1, 2), x["beta"])
    valid = torch.tensor([T, 0, T // 2], dtype=torch.int32, device="cuda")
    shape = sdm._delta_shape(*args, valid, None)[0]
    ws = torch.empty(sdm.library().sdm_gated_delta_workspace_bytes(shape), dtype=torch.uint8, device="cuda")
    want_state, want = x["state"].clone(), None
    want = sdm.gated_delta(want_state, *args, valid, workspace=ws)
    for given in (None, torch.empty(3, T, 4, 96, dtype=want.dtype, device="cuda")):
        state = x["state"].clone()
        got = taken("gated_delta", state, *args, valid, None, given)
        assert got.is_contiguous() and (given is None or got is given)
        assert torch.equal(got, want) and torch.equal(state, want_state)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    state = x["state"].clone()
    side.wait_stream(torch.cuda.current_stream())
    got = sdm.gated_delta(state, *args, valid, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(state, want_state)


def test_gated_delta_out_of_order():
    """None of these is taken; the checked path names what is wrong (and nothing has been written)."""
    x = draw(2, 3, 1, 2, 32, 48, "bf16")
    args = [x["state"], x["q"], x["k"], x["v"], x["g"], x["beta"], None, None, None]
    before = x["state"].clone()
    wrong = {0: [x["state"][:, :1], x["state"].double(), x["state"].transpose(2, 3).contiguous().transpose(2, 3)], 1: [x["q"][..., :16], x["q"].float(), 3],
             2: [x["k"].cpu(), x["k"][:, :2], None], 3: [x["v"][..., ::2], x["v"][:1], "v"], 4: [x["g"].bfloat16(), x["g"][..., :1]],
             5: [x["beta"][:1], x["beta"].double()], 6: [torch.zeros(2, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda"), 7],
             7: ["scale"], 8: [torch.empty(2, 3, 2, 32, dtype=torch.bfloat16, device="cuda"), x["v"].float()]}
    for i, values in wrong.items():
        for value in values:
            assert sdm._fast.gated_delta(*args[:i], value, *args[i + 1:]) is None, (i, value)
    assert sdm._fast.gated_delta(*args[:-1]) is None and torch.equal(x["state"], before)
    with pytest.raises((TypeError, ValueError)):
        sdm.gated_delta(x["state"], x["q"], x["k"].cpu(), x["v"], x["g"], x["beta"])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("weight,bias", [(None, None), (torch.float32, torch.float32), ("x", None), (None, "x")])
@pytest.mark.parametrize("shape", [(1, 1), (5, 33), (2, 3, 128)])
def test_layer_norm(dtype, weight, bias, shape):
    gen = torch.Generator().manual_seed(1)
    x, dy = (torch.randn(*shape, generator=gen).to(dtype).cuda() for _ in range(2))
    param = lambda kind: None if kind is None else torch.nn.Parameter(  # noqa: E731
        torch.randn(shape[-1], generator=gen).to(dtype if kind == "x" else kind).cuda())
    w, b = param(weight), param(bias)
    want = sdm.layer_norm(x, w, b, out=torch.empty_like(x))
    assert torch.equal(taken("layer_norm", x, w, b, 1e-5, False), want)
    y, stats = taken("layer_norm", x, w, b, 1e-5, True)
    assert torch.equal(y, want) and stats.shape == shape[:-1] + (2,)
    n = sdm.library().sdm_layer_norm_workspace_bytes(x.numel() // shape[-1], shape[-1])
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    back = sdm.layer_norm_backward(dy, x, w, stats, bias=b is not None, workspace=ws)
    got = taken("layer_norm_backward", dy, x, w, stats, b is not None)
    assert set(got) == set(back) and all(torch.equal(got[k], back[k]) for k in back)
    # what is not in order is left to the checked path
    for bad in ((x.double(), w, b), (x.cpu(), w, b), (x, torch.ones(shape[-1] + 1, device="cuda"), b), (x, torch.ones(shape[-1]), b),
                (x[..., :0], None, None), (None, w, b)):
        assert sdm._fast.layer_norm(*bad, 1e-5, False) is None
    assert sdm._fast.layer_norm_backward(dy[..., :0], x, w, stats, True) is None
    assert sdm._fast.layer_norm_backward(dy, x, w, stats.double(), True) is None


def test_a_refusal_is_raised():
    x = torch.zeros(2, 16385, device="cuda")
    with pytest.raises(sdm.SdmError):
        sdm.layer_norm(x)
    with pytest.raises(sdm.SdmError):
        sdm.gated_delta(torch.zeros(1, 1, 24, 16, device="cuda"), *(torch.zeros(1, 1, 1, 24, device="cuda"),) * 2,
                        torch.zeros(1, 1, 1, 16, device="cuda"), *(torch.zeros(1, 1, 1, device="cuda"),) * 2)
