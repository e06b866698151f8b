"""A residual block around the gated delta rule, trained and run token by token on the library's operators:

    one-hot tokens -> 1x1 convolution -> h
    h + 1x1 convolution of (layer norm -> 1x1 convolution to q, k, v -> causal convolution (SiLU) -> delta rule -> layer norm of each head)
      -> 1x1 convolution to logits

Queries, keys and values are slices of one tensor, and their gradients are written into slices of one tensor; the gates
(log decays and strengths) come from a 1x1 convolution of the normed rows.  ``AdamW`` steps the float32 weights and writes the
bf16 ones that the next forward pass reads.  The task and the 1x1 convolutions are those of ``sequence_block``.  Afterwards the
model answers token by token (``causal_conv_step``, ``delta_rule_step``).

    python examples/delta_block.py [--steps 100]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from sequence_block import B, BF16, batch, linear, linear_backward  # noqa: E402

BF16_WEIGHTS = ("w_in", "w_qkv", "w_conv", "w_gates", "w_o", "w_out")


class DeltaBlock:
    """The model, its optimiser, and the state it carries from token to token."""

    def __init__(self, symbols=16, width=64, heads=2, taps=4, lr=1e-2, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.symbols, self.width, self.heads, self.taps, self.dim = symbols, width, heads, taps, width // heads

        def normal(*shape, std):
            return torch.randn(*shape, generator=gen, device="cuda") * std

        one, s = (lambda n: torch.ones(n, device="cuda")), 1 / math.sqrt(width)
        self.master = {"w_in": normal(width, symbols, 1, 1, std=0.5), "norm1": one(width), "shift1": 0 * one(width),
                       "w_qkv": normal(3 * width, width, 1, 1, std=s), "w_conv": normal(3 * width, taps, std=1 / math.sqrt(taps)),
                       "bias": 0 * one(3 * width), "w_gates": normal(2 * heads, width, 1, 1, std=s), "norm2": one(self.dim),
                       "shift2": 0 * one(self.dim), "w_o": normal(width, width, 1, 1, std=s), "w_out": normal(symbols, width, 1, 1, std=s)}
        self.copies = {n: p.to(BF16) for n, p in self.master.items() if n in BF16_WEIGHTS}
        self.w = {**self.master, **self.copies}
        self.optimizer = B.AdamW(list(self.master.values()), [torch.zeros_like(p) for p in self.master.values()],
                                 copies=[self.copies.get(n) for n in self.master], lr=lr)

    def split(self, c):
        """Queries, keys and values, (..., heads, dim) each, as slices of the convolution's rows."""
        return [c[..., i * self.width:(i + 1) * self.width].unflatten(-1, (self.heads, self.dim)) for i in range(3)]

    def gates(self, n):
        a = linear(n, self.w["w_gates"]).float()
        g = -torch.nn.functional.softplus(a[..., :self.heads] - 2)
        return a, g, torch.sigmoid(a[..., self.heads:])

    def head_norm(self, y, **kw):
        return B.layer_norm(y.reshape(-1, self.dim), self.w["norm2"], self.w["shift2"], **kw)

    def forward(self, ids):
        """Logits (B, T, symbols) in float32, and what the backward pass reads."""
        w = self.w
        x = torch.nn.functional.one_hot(ids, self.symbols).to(BF16)
        h = linear(x, w["w_in"])
        n, m1, r1 = B.layer_norm(h, w["norm1"], w["shift1"], with_stats=True)
        u = linear(n, w["w_qkv"])
        c = B.causal_conv(u, w["w_conv"], w["bias"], silu=True)
        q, k, v = self.split(c)
        a, g, beta = self.gates(n)
        y, _, states = B.delta_rule(q, k, v, g.contiguous(), beta.contiguous(), unit=True, with_states=True)
        z, m2, r2 = self.head_norm(y, with_stats=True)
        h2 = h + linear(z.reshape(h.shape), w["w_o"])
        return linear(h2, w["w_out"]).float(), (x, h, n, m1, r1, u, c, a, g.contiguous(), beta.contiguous(), y, states, z, m2, r2, h2)

    def backward(self, dlogits, saved):
        """The gradients of all weights, by name, for upstream dlogits (bf16)."""
        x, h, n, m1, r1, u, c, a, g, beta, y, states, z, m2, r2, h2 = saved
        w, d = self.w, {}
        dh2, d["w_out"] = linear_backward(h2, w["w_out"], dlogits)
        dz, d["w_o"] = linear_backward(z.reshape(h.shape), w["w_o"], dh2.to(BF16))
        dy, d["norm2"], d["shift2"] = B.layer_norm_backward(y.reshape(-1, self.dim), w["norm2"], dz.to(BF16).reshape(-1, self.dim), m2, r2)
        q, k, v = self.split(c)
        dc = torch.empty_like(c)
        _, _, _, dg, dbeta, _ = B.delta_rule_backward(q, k, v, g, beta, dy.reshape(y.shape), states, unit=True, out=(*self.split(dc), None, None))
        da = torch.cat([-dg * torch.sigmoid(a[..., :self.heads] - 2), dbeta * beta * (1 - beta)], -1)
        dn1, d["w_gates"] = linear_backward(n, w["w_gates"], da.to(BF16))
        du, d["w_conv"], d["bias"], _ = B.causal_conv_backward(u, w["w_conv"], dc, w["bias"], silu=True)
        dn2, d["w_qkv"] = linear_backward(n, w["w_qkv"], du)
        dh, d["norm1"], d["shift1"] = B.layer_norm_backward(h, w["norm1"], (dn1 + dn2).to(BF16), m1, r1)
        _, d["w_in"] = linear_backward(x, w["w_in"], (dh + dh2).to(BF16))
        return d

    def loss(self, logits, targets, weight):
        """The mean cross entropy over the tokens of weight 1, and its gradient in bf16."""
        logp, onehot = torch.log_softmax(logits, -1), torch.nn.functional.one_hot(targets, self.symbols)
        share = (weight / weight.sum())[..., None]
        return -(logp * onehot * share).sum(), ((logp.exp() - onehot) * share).to(BF16)

    def step(self, ids, targets, weight):
        logits, saved = self.forward(ids)
        loss, dlogits = self.loss(logits, targets, weight)
        grads = self.backward(dlogits, saved)
        self.optimizer.step([grads[n] for n in self.master])
        return loss

    def start(self, sequences):
        """The state of `sequences` answers that have seen nothing."""
        return (torch.zeros(sequences, self.taps - 1, 3 * self.width, dtype=BF16, device="cuda"),
                torch.zeros(sequences, self.heads, self.dim, self.dim, device="cuda"))

    def answer(self, ids, state):
        """Logits (B, symbols) after one more token of each sequence; the state moves on."""
        w = self.w
        h = linear(torch.nn.functional.one_hot(ids, self.symbols).to(BF16), w["w_in"])
        n = B.layer_norm(h, w["norm1"], w["shift1"])
        c = B.causal_conv_step(linear(n, w["w_qkv"]), w["w_conv"], state[0], w["bias"], silu=True)
        _, g, beta = self.gates(n)
        y = B.delta_rule_step(*self.split(c), g.contiguous(), beta.contiguous(), state[1], unit=True)
        h2 = h + linear(self.head_norm(y).reshape(h.shape), w["w_o"])
        return linear(h2, w["w_out"]).float()


def train(steps=100, sequences=16, tokens=96, seed=0):
    model = DeltaBlock(seed=seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    losses = [model.step(*batch(gen, sequences, tokens, model.symbols)) for _ in range(steps)]
    return model, torch.stack(losses).tolist()


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=100)
    a = ap.parse_args()
    model, losses = train(a.steps)
    for k in range(0, a.steps, max(1, a.steps // 10)):
        print("step %4d  loss %.4f" % (k, losses[k]))
    ids, targets, _ = batch(torch.Generator(device="cuda").manual_seed(99), 4, 40, model.symbols)
    state = model.start(4)
    right = sum(int((model.answer(ids[:, t], state).argmax(-1) == targets[:, t]).sum()) * (t >= 2) for t in range(40))
    print("token by token: %d of %d right" % (right, 4 * 38))


if __name__ == "__main__":
    main()
