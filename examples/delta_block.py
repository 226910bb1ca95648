"""A memory block of the gated delta rule, trained and then served.

    python examples/delta_block.py

The block is y = x + merge(norm(delta(split(norm(x) W_in)))) W_out: layer norm, a projection to queries,
keys and values and one to the gates, the gated delta rule over the sequence, layer norm of every head's
readings, and a projection back with a residual. The projections are plain matrix products; the norms and
the delta rule, forward and backward, are this package's kernels. ``train`` takes one gradient step by
hand; ``prompt`` and ``token`` serve the block with the state carried along, one token at a time.
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import sparse_addressed_delta_gb300 as sdm  # noqa: E402


class DeltaBlock:
    def __init__(self, width, key_heads, heads, dk, dv, dtype=torch.bfloat16, seed=0, device="cuda"):
        self.shape = (key_heads, heads, dk, dv)
        self.dtype = dtype
        self.cuts = [key_heads * dk, key_heads * dk, heads * dv]         # q, k, v
        gen = torch.Generator(device).manual_seed(seed)

        def normal(*size, scale):
            return (scale * torch.randn(*size, device=device, generator=gen)).to(dtype)

        f32 = dict(device=device, dtype=torch.float32)
        self.p = {"w_in": normal(width, sum(self.cuts), scale=width ** -0.5),
                  "w_gate": normal(width, 2 * heads, scale=width ** -0.5),          # decay, beta
                  "w_out": normal(heads * dv, width, scale=(heads * dv) ** -0.5),
                  "norm_w": torch.ones(width, **f32), "norm_b": torch.zeros(width, **f32),
                  "head_w": torch.ones(dv, **f32)}

    def state(self, sequences):
        hk, h, dk, dv = self.shape
        return torch.zeros((sequences, h, dk, dv), dtype=torch.float32, device=self.p["norm_w"].device)

    def _heads(self, y):
        """The projections' columns as heads (views), unit keys and queries, and float32 gates."""
        hk, h, dk, dv = self.shape
        q, k, v = (y @ self.p["w_in"]).split(self.cuts, -1)
        a, b = (y @ self.p["w_gate"]).split(h, -1)
        q, k, v = q.unflatten(-1, (hk, dk)), k.unflatten(-1, (hk, dk)), v.unflatten(-1, (h, dv))
        unit = [t.float().norm(dim=-1, keepdim=True).clamp_min(1e-6) for t in (q, k)]
        gates = -0.1 * torch.nn.functional.softplus(a.float()), torch.sigmoid(b.float())
        return (q.float() / unit[0]).to(self.dtype), (k.float() / unit[1]).to(self.dtype), v, gates, unit, a

    def prompt(self, x, state, valid=None):
        """x [B, T, width] -> [B, T, width]; ``state`` is advanced in place."""
        x = x.contiguous()
        y = sdm.layer_norm(x, self.p["norm_w"], self.p["norm_b"])
        q, k, v, (g, beta) = self._heads(y)[:4]
        o = sdm.gated_delta(state, q, k, v, g, beta, valid)
        return x + sdm.layer_norm(o, self.p["head_w"]).flatten(2) @ self.p["w_out"]

    def token(self, x, state):
        """One token of every sequence, x [B, width]."""
        return self.prompt(x[:, None], state)[:, 0]

    def gradients(self, x, target, valid=None):
        """(loss, gradients of the parameters and of x) of the squared error of one training step."""
        p, (hk, h, dk, dv) = self.p, self.shape
        y, stats = sdm.layer_norm_save(x, p["norm_w"], p["norm_b"])
        q, k, v, (g, beta), unit, a = self._heads(y)
        o, saved = sdm.gated_delta_save(self.state(x.shape[0]), q, k, v, g, beta, valid)
        n, head_stats = sdm.layer_norm_save(o, p["head_w"])
        out = x + n.flatten(2) @ p["w_out"]
        err = (out - target).float()
        loss = err.square().mean()
        dout = (2 / err.numel() * err).to(self.dtype)
        flat = lambda t: t.flatten(0, 1)  # noqa: E731
        dn = (dout @ p["w_out"].T).unflatten(-1, (h, dv))
        hn = sdm.layer_norm_backward(dn, o, p["head_w"], head_stats, bias=False)
        d = sdm.gated_delta_backward(q, k, v, g, beta, valid, saved, hn["grad_x"])

        def through_unit(grad, value, size):
            grad, value = grad.float(), value.float()
            return ((grad - value * (grad * value).sum(-1, keepdim=True)) / size).flatten(2)

        dz = torch.cat([through_unit(d["grad_q"], q, unit[0]), through_unit(d["grad_k"], k, unit[1]),
                        d["grad_v"].flatten(2).float()], -1).to(self.dtype)
        dgate = torch.cat([-0.1 * torch.sigmoid(a.float()) * d["grad_log_decay"], beta * (1 - beta) * d["grad_beta"]], -1).to(self.dtype)
        nn = sdm.layer_norm_backward(dz @ p["w_in"].T + dgate @ p["w_gate"].T, x, p["norm_w"], stats)
        return loss, {"w_in": flat(y).T @ flat(dz), "w_gate": flat(y).T @ flat(dgate),
                      "w_out": flat(n.flatten(2)).T @ flat(dout),
                      "norm_w": nn["grad_weight"], "norm_b": nn["grad_bias"], "head_w": hn["grad_weight"],
                      "x": nn["grad_x"] + dout}

    def train(self, x, target, rate, valid=None):
        loss, grads = self.gradients(x, target, valid)
        for name, t in self.p.items():
            t -= (rate * grads[name]).to(t.dtype)
        return loss


def main():
    block = DeltaBlock(width=512, key_heads=4, heads=8, dk=64, dv=128)
    gen = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(4, 300, 512, device="cuda", generator=gen).bfloat16()
    # the sequence shifted by a few tokens, to be remembered
    target = torch.roll(x, 3, 1)
    for step in range(10):
        print(f"step {step}: loss {block.train(x, target, 20.0).item():.5f}")
    state = block.state(4)
    block.prompt(x[:, :200], state)
    served = torch.stack([block.token(x[:, t], state) for t in range(200, 300)], 1)
    whole = block.prompt(x, block.state(4))[:, 200:]
    off = (served - whole).float().norm() / whole.float().norm()
    print(f"served token by token after a prompt of 200: {off.item():.1e} off the whole sequence's outputs")


if __name__ == "__main__":
    main()
