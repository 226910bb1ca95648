"""Linear attention and group norm as a layer uses them: the readings of a token's heads normed in groups, with an
activation, in training (against autograd through the definitions in float64) and in serving (a prompt, then single
tokens); and both at sizes whose offsets pass 32 bits."""

import numpy as np
import pytest
import torch

import sparse_addressed_delta_gb300 as sdm
from test_gpu_linear import DT, draw, host, lengths

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    sdm.library()


def reference(x, w, b, valid, dy):
    """y and the gradients by autograd in float64, token by token, on the CPU."""
    p = {n: t.cpu().double().requires_grad_() for n, t in {**x, "w": w, "b": b}.items()}
    rep = p["v"].shape[2] // p["q"].shape[2]
    q, k = (p[n].repeat_interleave(rep, 2) for n in ("q", "k"))
    S, out = p["state"], []
    for t in range(q.shape[1]):
        new = p["g"].exp()[:, None, None] * S + k[:, t, :, :, None] * p["v"][:, t, :, None]
        on = (t < valid).double()[:, None, None, None]
        S = on * new + (1 - on) * S
        out.append(on[..., 0] * q.shape[-1] ** -0.5 * (q[:, t, :, :, None] * new).sum(-2))
    o = torch.stack(out, 1)
    h = (o - o.mean(-1, keepdim=True)) / (o.var(-1, unbiased=False, keepdim=True) + 1e-5).sqrt()
    z = h.flatten(2) * p["w"] + p["b"]
    y = z * torch.sigmoid(z)
    names = list(p)
    return y, dict(zip(names, torch.autograd.grad((y * dy.cpu().double()).sum(), [p[n] for n in names])))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_layers_gradients(dtype):
    """float32: 1e-4 in the 2-norm (the norm divides by the readings' deviation, a tenth of their size and more). bfloat16:
    readings, y and the gradients between them are rounded to 2^-9 each, four times on the way, and the norm's division
    makes up to ten times as much of the readings' own: 4 x 10 x 2^-9 = 8e-2 at most."""
    x = draw(2, 150, 1, 2, 32, 48, dtype, seed=40)
    valid = torch.tensor([150, 97])
    gen = torch.Generator().manual_seed(41)
    w, b = (1 + 0.1 * torch.randn(96, generator=gen)).cuda(), (0.1 * torch.randn(96, generator=gen)).cuda()
    dy = torch.randn(2, 150, 96, generator=gen)
    dy[1, 97:] = 0                                       # what stands behind a sequence has no gradient to give
    dy = dy.to(DT[dtype]).cuda()
    state = x["state"].clone()
    args = (x["q"], x["k"], x["v"], x["g"], lengths(valid.tolist()))
    o, saved = sdm.linear_attention_save(state, *args)
    tokens = o.flatten(0, 1).flatten(1)                  # a token a sample, its heads the groups
    y, stats = sdm.group_norm_save(tokens, 2, w, b, activation="silu")
    n = sdm.group_norm_backward(dy.flatten(0, 1), tokens, 2, w, b, stats, activation="silu")
    d = sdm.linear_attention_backward(*args, saved, n["grad_x"].view_as(o))
    want_y, want = reference(x, w, b, valid, dy)
    got = {"state": d["grad_state"], "q": d["grad_q"], "k": d["grad_k"], "v": d["grad_v"], "g": d["grad_log_decay"], "w": n["grad_weight"],
           "b": n["grad_bias"]}
    tol = 1e-4 if dtype == "f32" else 8e-2
    live = (torch.arange(150)[None] < valid[:, None])[..., None]
    off = lambda a, r: float((a.cpu().double() - r).norm() / r.norm())  # noqa: E731
    assert off(y.view(2, 150, 96).cpu() * live, want_y.detach() * live) <= tol
    for name, g in got.items():
        assert off(g, want[name]) <= tol, name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_layer_served(dtype):
    """A prompt of unequal lengths, then token by token, is the whole sequence through the layer: the readings differ by
    the order of their sums (2e-5 of the largest), which the norm's division makes up to ten times as much; bfloat16
    readings round to neighbours then (2^-8 of the value, and as much of y)."""
    x = draw(2, 90, 2, 4, 64, 64, dtype, seed=42)
    w, b = torch.ones(256, device="cuda"), torch.zeros(256, device="cuda")
    norm = lambda o: sdm.group_norm(o.flatten(2).flatten(0, 1), 4, w, b, activation="silu").view(*o.shape[:2], 256)  # noqa: E731
    whole = norm(sdm.linear_attention(x["state"].clone(), x["q"], x["k"], x["v"], x["g"]))
    state, valid = x["state"].clone(), [70, 33]
    sdm.linear_attention(state, x["q"], x["k"], x["v"], x["g"], lengths(valid))
    for step in range(20):
        cut = {n: torch.stack([x[n][i, valid[i] + step] for i in range(2)])[:, None] for n in ("q", "k", "v")}
        y = norm(sdm.linear_attention(state, cut["q"], cut["k"], cut["v"], x["g"]))
        want = torch.stack([whole[i, valid[i] + step] for i in range(2)])[:, None]
        tol = 1e-3 if dtype == "f32" else 11 * 2.0 ** -8
        assert np.abs(host(y) - host(want)).max() <= tol * np.abs(host(want)).max()


def test_offsets_past_32_bits():
    """Values of 2^31 elements and more, the last tokens against a call on them alone: heads that forget 95 % at a token
    have nothing left of what was 200 tokens before (e^-600)."""
    T, H = 34000, 512
    q, k = (torch.nn.functional.normalize(torch.randn(1, T, 1, 16, device="cuda"), dim=-1).bfloat16() for _ in range(2))
    v = torch.empty(1, T, H, 128, device="cuda", dtype=torch.bfloat16).normal_()
    assert v.numel() > 2 ** 31
    g = torch.full((H,), -3.0, device="cuda")
    state = torch.zeros(1, H, 16, 128, device="cuda")
    o = sdm.linear_attention(state, q, k, v, g)
    first = T - T % 64 - 256                             # the chunks are the same ones
    alone = torch.zeros_like(state)
    tail = sdm.linear_attention(alone, q[:, first:], k[:, first:], v[:, first:], g)
    assert torch.equal(o[:, -56:], tail[:, -56:]) and torch.equal(state, alone)
    tokens = o.view(T, H * 128)[:, :16384].contiguous() if H * 128 > 16384 else o.view(T, -1)
    del o, v
    x = tokens.repeat(4, 1)
    del tokens
    assert x.numel() > 2 ** 31
    y, stats = sdm.group_norm_save(x, 128, activation="silu")
    assert torch.equal(y[-T:], sdm.group_norm(x[-T:], 128, activation="silu"))
    dx = sdm.group_norm_backward(y, x, 128, None, None, stats, activation="silu")["grad_x"]
    want = sdm.group_norm_backward(y[-500:].contiguous(), x[-500:], 128, None, None, stats[-500:].contiguous(), activation="silu")["grad_x"]
    assert torch.equal(dx[-500:], want)
    maps = x.view(2, -1, 16384)                          # two samples of half the positions each
    y = sdm.group_norm(maps, 128, activation="silu")
    want = sdm.group_norm(maps[1:], 128, activation="silu")
    # (another number of splits for another number of samples: sums in another order)
    assert (y[1:].float() - want.float()).abs().max() <= 2.0 ** -7 * want.float().abs().max()
