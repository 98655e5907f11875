"""A transformer block from one attention's output to the inputs of the next.

    attention output -> projection -> gated residual, norm, modulation
      -> MLP up, GELU -> MLP down -> gated residual, norm, modulation
      -> q, k, v in one projection -> rotary positions of q and k

Every linear is the block-scaled e4m3 one; where a norm feeds a linear it writes
that linear's packed input, so the normalized activations never exist in 16
bits. ``input_gradient`` is the way back through frozen weights, as training an
adapter on them needs it.

    python examples/between_attentions.py [--tokens 4096] [--width 5120] [--heads 40]

runs it on synthetic weights and prints the time of one pass.
"""

from __future__ import annotations

import argparse
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from int8_hadamard_rotated_convrot_gb300 import block as bl  # noqa: E402


@dataclass
class Linear:
    """Frozen weights with their transposed form for the input gradient."""

    w: bl.Fp8Weights
    bias: torch.Tensor
    wt: bl.Fp8Weights

    @staticmethod
    def random(n: int, k: int, g: torch.Generator) -> "Linear":
        w = bl.convrot_fp8_quantize_weights(torch.randn(n, k, generator=g, device="cuda") * k**-0.5)
        return Linear(w, torch.randn(n, generator=g, device="cuda") * 0.01, w.transposed())


class Stretch:
    """The stretch between two attentions for [batch, tokens, width] activations in bf16."""

    def __init__(self, width: int, heads: int, hidden: int, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.width, self.heads, self.head_dim = width, heads, width // heads
        self.proj, self.up = Linear.random(width, width, g), Linear.random(hidden, width, g)
        self.down, self.qkv = Linear.random(width, hidden, g), Linear.random(3 * width, width, g)
        self.norms = [1 + 0.1 * torch.randn(width, generator=g, device="cuda") for _ in range(2)]

    def tables(self, tokens: int, scale: float = 1.0):
        """cos and sin for the tokens; past the trained length by `scale`, YaRN's frequencies."""
        freq, factor = bl.rotary_frequencies(self.head_dim // 2, scaling="yarn" if scale > 1 else "none", factor=scale,
                                             original_length=int(tokens / scale))
        return bl.convrot_rotary_table(tokens, freq, factor=factor)

    def forward(self, x, attention, modulation, tables):
        """x, attention [batch, tokens, width]; modulation: two (gate, scale, shift) of [batch, width] float32.
        Returns (residual stream, rotated q, rotated k, v) and what input_gradient needs."""
        b, t, d = x.shape
        (gate1, scale1, shift1), (gate2, scale2, shift2) = modulation
        rows = x.view(-1, d)
        y1 = bl.convrot_fp8_pack_linear(attention.reshape(-1, d), self.proj.w, self.proj.bias)
        h1, n1 = bl.convrot_gated_norm_pack(rows, y1, gate=gate1, scale=scale1, shift=shift1, rows_per_batch=t,
                                            pre=bl.NORM_RMS, pre_weight=self.norms[0])
        hidden = bl.convrot_fp8_linear(n1, self.up.w, self.up.bias, bl.ACT_GELU_TANH)
        y2 = bl.convrot_fp8_pack_linear(hidden, self.down.w, self.down.bias)
        h2, n2 = bl.convrot_gated_norm_pack(h1, y2, gate=gate2, scale=scale2, shift=shift2, rows_per_batch=t,
                                            pre=bl.NORM_RMS, pre_weight=self.norms[1])
        qkv = bl.convrot_fp8_linear(n2, self.qkv.w, self.qkv.bias).view(b, t, 3 * self.heads, self.head_dim)
        q, k, v = qkv.split(self.heads, 2)
        q, k = bl.convrot_rotary(q, k, *tables, out_q=q, out_k=k)  # in place
        return (h2.view(b, t, d), q, k, v), (h1, y1, h2, y2, n1)

    def input_gradient(self, saved, modulation, tables, dh, dq, dk, dv):
        """The gradients of x and of the attention's output, from those of forward's results."""
        h1, y1, h2, y2, n1 = saved
        b, t, d = dh.shape
        (gate1, scale1, shift1), (gate2, scale2, shift2) = modulation
        dqkv = torch.empty(b, t, 3 * self.heads, self.head_dim, dtype=dh.dtype, device=dh.device)
        parts = dqkv.split(self.heads, 2)
        bl.convrot_rotary(dq, dk, *tables, inverse=True, out_q=parts[0], out_k=parts[1])
        parts[2].copy_(dv)
        dn = bl.convrot_fp8_pack_linear(dqkv.view(b * t, -1), self.qkv.wt)
        second = bl.convrot_gated_norm_backward(h2, y2, dh.reshape(-1, d), dn, gate=gate2, scale=scale2, shift=shift2,
                                                rows_per_batch=t, pre=bl.NORM_RMS, pre_weight=self.norms[1])
        # GELU's input was not kept: the up projection is run again for it, without the activation
        u = bl.convrot_fp8_linear(n1, self.up.w, self.up.bias).float().requires_grad_()
        dhidden = bl.convrot_fp8_pack_linear(second["dy"], self.down.wt)
        (du,) = torch.autograd.grad(torch.nn.functional.gelu(u, approximate="tanh"), u, dhidden.float())
        dn = bl.convrot_fp8_pack_linear(du.to(dh.dtype), self.up.wt)
        first = bl.convrot_gated_norm_backward(h1, y1, second["dx"], dn, gate=gate1, scale=scale1, shift=shift1,
                                               rows_per_batch=t, pre=bl.NORM_RMS, pre_weight=self.norms[0])
        dattention = bl.convrot_fp8_pack_linear(first["dy"], self.proj.wt)
        return first["dx"].view(b, t, d), dattention.view(b, t, d)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--batch", type=int, default=1)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--width", type=int, default=5120)
    ap.add_argument("--heads", type=int, default=40)
    ap.add_argument("--hidden", type=int, default=13824)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    net = Stretch(a.width, a.heads, a.hidden)
    x, attention = (torch.randn(a.batch, a.tokens, a.width, device="cuda").bfloat16() for _ in range(2))
    modulation = [[0.3 * torch.randn(a.batch, a.width, device="cuda") for _ in range(3)] for _ in range(2)]
    tables = net.tables(a.tokens)
    (h, q, k, v), saved = net.forward(x, attention, modulation, tables)
    grads = [torch.randn_like(z) * 0.1 for z in (h, q, k, v)]
    for name, run in (("forward", lambda: net.forward(x, attention, modulation, tables)),
                      ("input gradient", lambda: net.input_gradient(saved, modulation, tables, *grads))):
        for _ in range(3):
            run()
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        for _ in range(a.steps):
            run()
        end.record()
        torch.cuda.synchronize()
        print(f"{name}: {start.elapsed_time(end) / a.steps * 1e3:.0f} us for {a.batch * a.tokens} tokens")


if __name__ == "__main__":
    main()
