"""A small sequence model trained and run on the library's operators:

    one-hot tokens -> 1x1 convolution -> causal convolution (SiLU) -> 1x1 convolution to two gates
                   -> gated recurrence -> 1x1 convolution to logits

The 1x1 convolutions over tokens are ``conv_ex`` (channels-last, bf16 out) forward and
``conv_backward`` backward; the gates are column slices of one tensor, and their gradients are
written into slices of one tensor; ``AdamW`` steps the float32 weights and writes the bf16 ones
that the next forward pass reads.  The task: name the symbol seen two tokens ago.  Afterwards the
model answers token by token (``causal_conv_step``, ``gated_scan_step``).

    python examples/sequence_block.py [--steps 150] [--bits 8]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from cnn_convolution_forward_amd import binding as B  # noqa: E402

BF16 = torch.bfloat16


def linear(x, w):
    """Rows x (..., D) times w (C, D, 1, 1), as a 1x1 convolution of one channels-last image; bf16."""
    y = B.conv_ex(x.reshape(1, 1, -1, x.shape[-1]), w, layout="nhwc", out_dtype="bf16")
    return y.view(BF16).reshape(*x.shape[:-1], w.shape[0])


def linear_backward(x, w, dy):
    """(dx, dw) of linear, float32: every row is an image of one pixel."""
    n = x.numel() // x.shape[-1]
    dx, dw, _ = B.conv_backward(x.reshape(n, -1, 1, 1), w, dy.reshape(n, -1, 1, 1), with_db=False)
    return dx.reshape(x.shape), dw


class SequenceBlock:
    """The model, its optimiser, and the state it carries from token to token."""

    def __init__(self, symbols=16, width=64, taps=4, bits=32, lr=1e-2, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std):
            return torch.randn(*shape, generator=gen, device="cuda") * std

        self.symbols, self.width, self.taps = symbols, width, taps
        self.master = [normal(width, symbols, 1, 1, std=0.5), normal(width, taps, std=1 / math.sqrt(taps)),
                       torch.zeros(width, device="cuda"), normal(2 * width, width, 1, 1, std=1 / math.sqrt(width)),
                       torch.linspace(-5.0, -1.0, width, device="cuda"), normal(symbols, width, 1, 1, std=1 / math.sqrt(width))]
        reads_bf16 = (True, True, False, True, False, True)       # bias and decay are read in float32
        self.copies = [p.to(BF16) if b else None for p, b in zip(self.master, reads_bf16)]
        self.w_in, self.w_conv, self.bias, self.w_gates, self.decay, self.w_out = (
            p if c is None else c for p, c in zip(self.master, self.copies))
        self.grads = [torch.zeros_like(p) for p in self.master]
        self.optimizer = B.AdamW(self.master, self.grads, copies=self.copies, bits=bits, lr=lr)

    def forward(self, ids):
        """Logits (B, T, symbols) in float32, and what the backward pass reads."""
        x = torch.nn.functional.one_hot(ids, self.symbols).to(BF16)
        u = linear(x, self.w_in)
        c = B.causal_conv(u, self.w_conv, self.bias, silu=True)
        gates = linear(c, self.w_gates)
        g, i = gates[..., :self.width], gates[..., self.width:]
        y, _, states = B.gated_scan(c, g, i, self.decay, with_states=True)
        return linear(y, self.w_out).float(), (x, u, c, g, i, y, states)

    def step(self, ids, targets, weight):
        """One training step on the mean cross entropy over the tokens of weight 1; returns the loss."""
        logits, (x, u, c, g, i, y, states) = self.forward(ids)
        logp = torch.log_softmax(logits, -1)
        onehot = torch.nn.functional.one_hot(targets, self.symbols)
        loss = -(logp * onehot).sum(-1).mul(weight).sum() / weight.sum()
        dlogits = ((logp.exp() - onehot) * (weight / weight.sum())[..., None]).to(BF16)
        dy, d_out = linear_backward(y, self.w_out, dlogits)
        dgates = torch.empty(*g.shape[:-1], 2 * self.width, dtype=BF16, device="cuda")
        dc = torch.empty_like(c)
        _, _, _, d_decay, _ = B.gated_scan_backward(
            c, g, i, self.decay, dy.to(BF16), states, out=(dc, dgates[..., :self.width], dgates[..., self.width:]))
        dc2, d_gates = linear_backward(c, self.w_gates, dgates)
        du, d_conv, d_bias, _ = B.causal_conv_backward(u, self.w_conv, (dc + dc2).to(BF16), self.bias, silu=True)
        _, d_in = linear_backward(x, self.w_in, du)
        self.optimizer.step([d_in, d_conv, d_bias, d_gates, d_decay, d_out])
        return loss

    def start(self, sequences):
        """The state of `sequences` answers that have seen nothing."""
        return (torch.zeros(sequences, self.taps - 1, self.width, dtype=BF16, device="cuda"),
                torch.zeros(sequences, self.width, device="cuda"))

    def answer(self, ids, state):
        """Logits (B, symbols) after one more token of each sequence; the state moves on."""
        x = torch.nn.functional.one_hot(ids, self.symbols).to(BF16)
        c = B.causal_conv_step(linear(x, self.w_in), self.w_conv, state[0], self.bias, silu=True)
        gates = linear(c, self.w_gates)
        y = B.gated_scan_step(c, gates[:, :self.width], gates[:, self.width:], self.decay, state[1])
        return linear(y, self.w_out).float()


def batch(gen, sequences, tokens, symbols, delay=2):
    ids = torch.randint(symbols, (sequences, tokens), generator=gen, device="cuda")
    weight = torch.ones(sequences, tokens, device="cuda")
    weight[:, :delay] = 0
    return ids, torch.roll(ids, delay, 1), weight


def train(steps=150, bits=32, sequences=16, tokens=96, seed=0):
    model = SequenceBlock(bits=bits, seed=seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    losses = [model.step(*batch(gen, sequences, tokens, model.symbols)) for _ in range(steps)]
    return model, torch.stack(losses).tolist()


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=150)
    ap.add_argument("--bits", type=int, default=32, choices=(8, 32))
    a = ap.parse_args()
    model, losses = train(a.steps, a.bits)
    for k in range(0, a.steps, max(1, a.steps // 10)):
        print("step %4d  loss %.4f" % (k, losses[k]))
    ids, targets, _ = batch(torch.Generator(device="cuda").manual_seed(99), 4, 40, model.symbols)
    state = model.start(4)
    right = 0
    for t in range(40):
        got = model.answer(ids[:, t], state).argmax(-1)
        right += int((got == targets[:, t]).sum()) if t >= 2 else 0
    print("token by token: %d of %d right" % (right, 4 * 38))


if __name__ == "__main__":
    main()
