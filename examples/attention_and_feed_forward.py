"""The second half of a transformer block: attention to a prompt, then the gated feed-forward.

    norm -> q;  prompt -> k, v in one projection
      -> attention of the tokens to the prompt's states, padding masked -> projection
      -> residual, norm -> gate and up projections, SiLU, product -> projection -> residual

The frozen projections are block-scaled e4m3 linears; the gated feed-forward's own
two are 16-bit weights, and are trained: ``gradient`` gives their gradients and
those of the tokens and the prompt.

    python examples/attention_and_feed_forward.py [--tokens 4096] [--prompt 512] [--width 5120] [--heads 40]

runs it on synthetic weights and prints the time of one pass.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from examples.between_attentions import Linear  # noqa: E402
from int8_hadamard_rotated_convrot_gb300 import block as bl  # noqa: E402


class Half:
    """For [batch, tokens, width] activations and [batch, prompt, width] states in bf16."""

    def __init__(self, width: int, heads: int, hidden: int, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.width, self.heads, self.head_dim, self.hidden = width, heads, width // heads, hidden
        self.q, self.kv = Linear.random(width, width, g), Linear.random(2 * width, width, g)
        self.proj, self.down = Linear.random(width, width, g), Linear.random(width, hidden, g)
        self.norms = [1 + 0.1 * torch.randn(width, generator=g, device="cuda") for _ in range(2)]
        # one tensor, as checkpoints have it: the gate's rows, then the up projection's
        self.w = (torch.randn(2 * hidden, width, generator=g, device="cuda") * width**-0.5).bfloat16()
        self.b = torch.randn(2 * hidden, generator=g, device="cuda") * 0.01

    def forward(self, x, prompt, mask):
        """x, prompt; mask [batch, prompt]: which states are there. Returns the residual stream and what gradient needs."""
        b, t, d = x.shape
        p, n = prompt.shape[1], self.hidden
        rows = x.view(-1, d)
        _, n1 = bl.convrot_gated_norm(rows, pre=bl.NORM_RMS, pre_weight=self.norms[0])
        q = bl.convrot_fp8_pack_linear(n1, self.q.w, self.q.bias).view(b, t, self.heads, self.head_dim)
        kv = bl.convrot_fp8_pack_linear(prompt.reshape(-1, d), self.kv.w, self.kv.bias).view(b, p, 2, self.heads, self.head_dim)
        a, lse = bl.convrot_attention(q, kv[:, :, 0], kv[:, :, 1], mask)
        y1 = bl.convrot_fp8_pack_linear(a.view(-1, d), self.proj.w, self.proj.bias)
        h1, n2 = bl.convrot_gated_norm(rows, y1, pre=bl.NORM_RMS, pre_weight=self.norms[1])
        y, gate, up = bl.convrot_gated_linear(n2, self.w[:n], self.w[n:], self.b[:n], self.b[n:], bl.ACT_SILU, keep=True)
        y2 = bl.convrot_fp8_pack_linear(y, self.down.w, self.down.bias)
        h2, _ = bl.convrot_gated_norm(h1, y2, pre=bl.NORM_NONE)
        return h2.view(b, t, d), (q, kv, a, lse, y1, h1, n2, gate, up)

    def gradient(self, x, saved, mask, dh):
        """The gradients of x, the prompt, the gated weights and their biases, from that of forward's residual stream."""
        q, kv, a, lse, y1, h1, n2, gate, up = saved
        b, t, d = dh.shape
        n, rows = self.hidden, dh.reshape(-1, d)
        dy = bl.convrot_fp8_pack_linear(rows, self.down.wt)
        ff = bl.convrot_gated_linear_backward(n2, self.w[:n], self.w[n:], gate, up, dy, bl.ACT_SILU, biases=True)
        second = bl.convrot_gated_norm_backward(h1, y1, rows, ff["dx"], pre=bl.NORM_RMS, pre_weight=self.norms[1])
        da = bl.convrot_fp8_pack_linear(second["dy"], self.proj.wt).view(b, t, self.heads, self.head_dim)
        at = bl.convrot_attention_backward(q, kv[:, :, 0], kv[:, :, 1], a, lse, da, mask)
        dkv = torch.stack([at["dk"], at["dv"]], 2)
        dprompt = bl.convrot_fp8_pack_linear(dkv.view(-1, 2 * d), self.kv.wt)
        dn1 = bl.convrot_fp8_pack_linear(at["dq"].view(-1, d), self.q.wt)
        first = bl.convrot_gated_norm_backward(x.view(-1, d), None, second["dx"], dn1, pre=bl.NORM_RMS, pre_weight=self.norms[0])
        return {"x": first["dx"].view(b, t, d), "prompt": dprompt.view(b, -1, d), "w": torch.cat([ff["dw_gate"], ff["dw_up"]]),
                "b": torch.cat([ff["db_gate"], ff["db_up"]])}


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--batch", type=int, default=1)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--prompt", type=int, default=512)
    ap.add_argument("--width", type=int, default=5120)
    ap.add_argument("--heads", type=int, default=40)
    ap.add_argument("--hidden", type=int, default=13824)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    net = Half(a.width, a.heads, a.hidden)
    x, prompt = (torch.randn(a.batch, n, a.width, device="cuda").bfloat16() for n in (a.tokens, a.prompt))
    mask = (torch.arange(a.prompt, device="cuda") < a.prompt * 3 // 4).expand(a.batch, a.prompt)
    h, saved = net.forward(x, prompt, mask)
    dh = torch.randn_like(h) * 0.1
    for name, run in (("forward", lambda: net.forward(x, prompt, mask)), ("gradient", lambda: net.gradient(x, saved, mask, dh))):
        for _ in range(3):
            run()
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        for _ in range(a.steps):
            run()
        end.record()
        torch.cuda.synchronize()
        print(f"{name}: {start.elapsed_time(end) / a.steps * 1e3:.0f} us for {a.batch * a.tokens} tokens and {a.batch * a.prompt} of the prompt")


if __name__ == "__main__":
    main()
