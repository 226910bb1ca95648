"""The memory block of examples/delta_block.py: its gradients against autograd through the definitions in
float64, and serving (a prompt, then single tokens) against the whole sequence."""

import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


def reference(block, x, target, valid):
    """The same loss by autograd in float64, token by token, on the CPU."""
    hk, h, dk, dv = block.shape
    p = {n: t.cpu().double().requires_grad_() for n, t in block.p.items()}
    x, target = x.cpu().double().requires_grad_(), target.cpu()

    def norm(t, w, b=0.0):
        m = t.mean(-1, keepdim=True)
        return (t - m) / ((t - m).square().mean(-1, keepdim=True) + 1e-5).sqrt() * w + b

    n = norm(x, p["norm_w"], p["norm_b"])
    q, k, v = (n @ p["w_in"]).split(block.cuts, -1)
    a, b = (n @ p["w_gate"]).split(h, -1)
    q, k = (torch.nn.functional.normalize(t.unflatten(-1, (hk, dk)), dim=-1).repeat_interleave(h // hk, 2) for t in (q, k))
    v, g, beta = v.unflatten(-1, (h, dv)), -0.1 * torch.nn.functional.softplus(a), torch.sigmoid(b)
    S, out = torch.zeros(x.shape[0], h, dk, dv, dtype=torch.float64), []
    for t in range(x.shape[1]):
        d = g[:, t, :, None, None].exp() * S
        r = v[:, t] - (k[:, t, :, :, None] * d).sum(-2)
        new = d + (beta[:, t, :, None] * k[:, t])[..., None] * r[:, :, None]
        on = (t < valid).double()[:, None, None, None] if valid is not None else 1.0
        S = on * new + (1 - on) * S
        out.append((on if valid is None else on[..., 0]) * dk ** -0.5 * (q[:, t, :, :, None] * new).sum(-2))
    y = x + norm(torch.stack(out, 1), p["head_w"]).flatten(2) @ p["w_out"]
    loss = (y - target.double()).square().mean()
    names = list(p)
    grads = torch.autograd.grad(loss, [p[n] for n in names] + [x])
    return y, loss, dict(zip(names + ["x"], grads))


@pytest.mark.parametrize("dtype,tol", [(torch.float32, 2e-3), (torch.bfloat16, 5e-2)])
def test_gradients(dtype, tol):
    """float32: the projections may run in TF32 (10 bits). bfloat16: a chain of six roundings of 2^-9 each
    way, carried through a recurrence and three products; in the 2-norm."""
    from delta_block import DeltaBlock
    block = DeltaBlock(96, 1, 2, 32, 80, dtype=dtype, seed=3)
    gen = torch.Generator("cuda").manual_seed(4)
    x, target = (torch.randn(2, 70, 96, device="cuda", generator=gen).to(dtype) for _ in range(2))
    loss, grads = block.gradients(x, target)
    _, want_loss, want = reference(block, x, target, None)
    assert loss.item() == pytest.approx(want_loss.item(), rel=tol)
    for name, g in grads.items():
        assert float((g.cpu().double() - want[name]).norm() / want[name].norm()) <= tol, name


def test_training_lowers_the_loss():
    from delta_block import DeltaBlock
    block = DeltaBlock(128, 2, 4, 64, 64, seed=5)
    x = torch.randn(2, 100, 128, device="cuda", generator=torch.Generator("cuda").manual_seed(6)).bfloat16()
    target = torch.roll(x, 2, 1)
    losses = [block.train(x, target, 20.0).item() for _ in range(6)]
    assert all(b < a for a, b in zip(losses, losses[1:])), losses


def test_serving_continues_a_prompt():
    """In float32, so that nothing but the order of sums differs: tokens one by one after a prompt, and a
    prompt of unequal lengths."""
    from delta_block import DeltaBlock
    block = DeltaBlock(96, 2, 4, 48, 80, dtype=torch.float32, seed=7)
    x = torch.randn(3, 90, 96, device="cuda", generator=torch.Generator("cuda").manual_seed(8))
    whole = block.prompt(x, block.state(3))
    state = block.state(3)
    first = block.prompt(x[:, :64], state)
    rest = torch.stack([block.token(x[:, t], state) for t in range(64, 90)], 1)
    got = torch.cat([first, rest], 1)
    assert float((got - whole).norm() / whole.norm()) <= 1e-3          # TF32 projections of other shapes
    valid = torch.tensor([64, 10, 0], dtype=torch.int32, device="cuda")
    state = block.state(3)
    block.prompt(x[:, :64], state, valid)
    alone = block.state(1)
    block.prompt(x[1:2, :10], alone)
    assert float((state[1:2] - alone).norm() / alone.norm()) <= 1e-3 and not state[2].any()
