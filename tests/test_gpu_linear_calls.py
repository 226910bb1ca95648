"""The direct entries of linear attention and group norm (csrc/calls.cpp) beside the binding's checked path: the same
results to the bit, and calls out of order left to the checks."""

import pytest
import torch

import sparse_addressed_delta_gb300 as sdm
from test_gpu_linear import draw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    sdm.library()


def both(monkeypatch, call):
    """The call's results by the direct entry, which has to take it, and without it."""
    took = []

    class Watch:
        def __getattr__(self, name):
            def entry(*args):
                out = getattr(fast, name)(*args)
                took.append(out is not None)
                return out
            return entry

    fast = sdm._fast
    monkeypatch.setattr(sdm, "_fast", Watch())
    got = call()
    assert took and all(took)
    monkeypatch.setattr(sdm, "_fast", sdm._NoCalls)
    want = call()
    monkeypatch.setattr(sdm, "_fast", fast)
    assert len(got) == len(want) and all(a.dtype == b.dtype and a.shape == b.shape and torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 12, 13, 90])
@pytest.mark.parametrize("options", [{}, dict(scale=0.3)], ids=str)
def test_linear_attention(monkeypatch, dtype, T, options):
    x = draw(3, T, 2, 4, 64, 96, dtype, seed=T)
    wide = torch.zeros(3, T, 8, 96, dtype=x["v"].dtype, device="cuda")
    wide[:, :, 2:6] = x["v"]
    args = (x["q"], x["k"], wide[:, :, 2:6], x["g"], torch.tensor([T, 0, T // 2], dtype=torch.int32, device="cuda"))
    end = torch.randn_like(x["state"])

    def call():
        state, again = x["state"].clone(), x["state"].clone()
        o = sdm.linear_attention(state, *args, **options)
        given = torch.empty_like(o)
        assert sdm.linear_attention(x["state"].clone(), *args, readings=given, **options) is given
        p, saved = sdm.linear_attention_save(again, *args, **options)
        out = [o, given, state, p, again, saved[:x["state"].numel() * 4].view(torch.float32)]
        for kw in (dict(grad_state=end), dict(decay=False)):
            got = sdm.linear_attention_backward(*args, saved, wide[:, :, 2:6], **kw, **options)
            assert ("grad_log_decay" in got) == kw.get("decay", True)
            out += [got[n] for n in sorted(got)]
        return out

    both(monkeypatch, call)


@pytest.mark.parametrize("shape", [(40, 64), (3, 1, 96), (2, 70, 64)], ids=str)
@pytest.mark.parametrize("act", [None, "silu"])
def test_group_norm(monkeypatch, shape, act):
    x, dy = (torch.randn(*shape, device="cuda").bfloat16() for _ in range(2))
    for w, b in ((None, None), (torch.randn(shape[-1], device="cuda"), None), tuple(torch.nn.Parameter(torch.randn(shape[-1], device="cuda").bfloat16()) for _ in range(2))):
        def call():
            y, stats = sdm.group_norm_save(x, 4, w, b, activation=act)
            got = sdm.group_norm_backward(dy, x, 4, w, b, stats, activation=act)
            assert set(got) == {"grad_x"} | ({"grad_weight"} if w is not None else set()) | ({"grad_bias"} if b is not None else set())
            return [sdm.group_norm(x, 4, w, b, activation=act), y, stats, *(got[n] for n in sorted(got))]

        both(monkeypatch, call)


def test_out_of_order():
    """None of these is taken (the checked path names what is wrong)."""
    x = draw(2, 9, 1, 2, 32, 48, "bf16")
    args = [x["state"], x["q"], x["k"], x["v"], x["g"], None, None, None, False]
    before = x["state"].clone()
    wrong = {0: [x["state"][:, :1], x["state"].double()], 1: [x["q"][..., :16], x["q"].float(), 3], 2: [x["k"].cpu(), x["k"][:, :2], None],
             3: [x["v"][..., ::2], x["v"][:1], "v"], 4: [x["g"].bfloat16(), x["g"][:1], x["g"][:, None]],
             5: [torch.zeros(2, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda"), 7], 6: ["scale"],
             7: [torch.empty(2, 9, 2, 32, dtype=torch.bfloat16, device="cuda"), x["v"].float()]}
    for i, values in wrong.items():
        for value in values:
            assert sdm._fast.linear_attention(*args[:i], value, *args[i + 1:]) is None, (i, value)
    assert sdm._fast.linear_attention(*args[:-1]) is None and torch.equal(x["state"], before)
    saved = sdm.linear_attention_save(x["state"].clone(), *args[1:5])[1]
    back = [*args[1:5], None, saved, x["v"], None, None, True]
    for i, value in ((5, saved.float()), (5, None), (6, x["v"].float()), (6, x["v"][:, :3]), (7, x["state"].double()), (8, "scale"), (3, None)):
        assert sdm._fast.linear_attention_backward(*back[:i], value, *back[i + 1:]) is None, i
    y = torch.randn(3, 5, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    for bad in ((y.double(), 4, w, w, None), (y.cpu(), 4, w, w, None), (y, 5, w, w, None), (y, True, w, w, None), (y, 4, w[:32], w, None), (y, 4, w, w, "gelu"),
                (y.transpose(0, 1), 4, w, w, None), (y[0, 0], 4, w, w, None), (y[..., :0], 1, None, None, None), (None, 4, w, w, None), (y, 0, w, w, None)):
        assert sdm._fast.group_norm(*bad, 1e-5, False) is None
    stats = sdm.group_norm_save(y, 4, w, w)[1]
    for bad in ((y[:2], y, 4, w, w, stats, None), (y, y, 8, w, w, stats, None), (y, y, 4, w, w, stats.double(), None), (y.bfloat16(), y, 4, w, w, stats, None)):
        assert sdm._fast.group_norm_backward(*bad) is None


def test_a_refusal_is_raised():
    with pytest.raises(sdm.SdmError):
        sdm.group_norm(torch.zeros(2, 16400, device="cuda"), 4)
    for T in (1, 20):
        with pytest.raises(sdm.SdmError):
            sdm.linear_attention(torch.zeros(1, 1, 24, 16, device="cuda"), *(torch.zeros(1, T, 1, 24, device="cuda"),) * 2,
                                 torch.zeros(1, T, 1, 16, device="cuda"), torch.zeros(1, device="cuda"))
