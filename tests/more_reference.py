"""Plain 64-bit forms of the gated feed-forward's projections and of attention to
other states, for their tests: from the formulas in include/convrot_block.h,
sharing no code with the package. Each comes with bounds on how far a result may
be off, elementwise, from the arithmetic alone:

* a rounding to a type is off by half a step, rounding(dtype) of the value (and
  2^-25 absolutely in float16, where values are subnormal);
* the tensor cores add 16 products at a time to an fp32 sum, each addition off by
  at most 2^-23 of the sizes added so far (they may cut off instead of rounding):
  SUM(k) = (k / 16 + 8) 2^-23 of the sum of the products' sizes;
* an activation or exponential in fp32: APPROX = 2^-20 of its factors' sizes (two
  approximate instructions of 2 units each and a few roundings; the erf form's
  1.5e-7 is below that too).
"""

import math

import torch

from . import block_reference

APPROX = 2.0**-20
SILU = 3


def rounding(dtype):
    return 0.0 if dtype == torch.float64 else block_reference.rounding(dtype)


def total(k):
    return (k / 16 + 8) * 2.0**-23


def half_step(v, dtype):
    return rounding(dtype) * v.abs() * (1 + 1e-6) + (2.0**-25 if dtype == torch.float16 else 0.0)


def act(v, kind):
    if kind == SILU:
        return v * torch.sigmoid(v)
    if kind == 1:
        return 0.5 * v * torch.special.erfc(-v / math.sqrt(2.0))
    if kind == 2:
        return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v**3))
    return v


def gated(x, wg, wu, bg=None, bu=None, kind=SILU):
    """((y, gate, up), their bounds) in float64."""
    dtype = x.dtype
    x, wg, wu = x.double(), wg.double(), wu.double()
    g, u = x @ wg.t(), x @ wu.t()
    eg, eu = ((x.abs() @ w.abs().t()) * total(x.shape[1]) for w in (wg, wu))
    if bg is not None:
        g = g + bg.double()
    if bu is not None:
        u = u + bu.double()
    eg, eu = eg + 2.0**-23 * g.abs(), eu + 2.0**-23 * u.abs()
    y = act(g, kind) * u
    ey = 1.2 * eg * (u.abs() + eu) + act(g, kind).abs() * eu + APPROX * g.abs() * u.abs()
    return (y, g, u), (half_step(y, dtype) + 1.01 * ey, half_step(g, dtype) + eg, half_step(u, dtype) + eu)


def gated_gradient(x, wg, wu, gate, up, dy, kind=SILU):
    """(gradients, bounds) as dicts in float64."""
    dtype = x.dtype
    m, k = x.shape
    n = wg.shape[0]
    x, wg, wu, d, u = (t.double() for t in (x, wg, wu, dy, up))
    g = gate.double().requires_grad_()
    a = act(g, kind)
    (slope,) = torch.autograd.grad(a.sum(), g)
    g, a = g.detach(), a.detach()
    dg, du = d * u * slope, d * a
    eg, eu = 2 * APPROX * (d * u).abs() * (1 + g.abs()), 2 * APPROX * (d * g).abs()
    rg, ru = half_step(dg, dtype) + eg, half_step(du, dtype) + eu  # as operands
    out = {"dx": dg @ wg + du @ wu, "dw_gate": dg.t() @ x, "dw_up": du.t() @ x, "db_gate": dg.sum(0), "db_up": du.sum(0)}
    size = {"dx": dg.abs() @ wg.abs() + du.abs() @ wu.abs(), "dw_gate": dg.abs().t() @ x.abs(), "dw_up": du.abs().t() @ x.abs()}
    bound = {"dx": rg @ wg.abs() + ru @ wu.abs() + total(2 * n) * size["dx"],
             "dw_gate": rg.t() @ x.abs() + total(m) * size["dw_gate"], "dw_up": ru.t() @ x.abs() + total(m) * size["dw_up"]}
    bound = {name: 1.01 * b + half_step(out[name], dtype) for name, b in bound.items()}
    # sums over rows in fp32: every addition is off by half a step of what is there, and no more than m of them follow each other
    bound |= {"db_gate": eg.sum(0) + min(m, 2000) * 2.0**-24 * dg.abs().sum(0) + 1e-30, "db_up": eu.sum(0) + min(m, 2000) * 2.0**-24 * du.abs().sum(0) + 1e-30}
    return out, bound


def _heads(t, heads):
    return t.double().transpose(1, 2).repeat_interleave(heads // t.shape[2], 1)


class Attention:
    """out, lse and the gradients, with bounds, by sample and query head in float64."""

    def __init__(self, q, k, v, mask=None, scale=None):
        self.dtype, heads, d = q.dtype, q.shape[2], q.shape[3]
        self.kv_heads, self.scale = k.shape[2], d**-0.5 if scale is None else scale
        there = torch.ones(k.shape[:2], dtype=torch.bool, device=k.device) if mask is None else mask.bool()
        clean = lambda t: torch.where(there[:, :, None, None], t, torch.zeros((), dtype=t.dtype, device=t.device))  # noqa: E731
        self.q, self.k, self.v = q.double().transpose(1, 2), _heads(clean(k), heads), _heads(clean(v), heads)
        s = self.scale * self.q @ self.k.transpose(2, 3)
        s = s.masked_fill(~there[:, None, None], -math.inf)
        self.lse = torch.logsumexp(s, 3) if k.shape[1] else torch.full(s.shape[:3], -math.inf, device=q.device, dtype=torch.float64)
        self.p = torch.where(there[:, None, None], torch.exp(s - self.lse[..., None]), 0.0).nan_to_num(0.0)
        out = self.p @ self.v
        # what a score, and so a probability's exponent, may be off by
        self.e = self.scale * total(d) * (self.q.abs() @ self.k.abs().transpose(2, 3)) + 2.0**-21 * s.masked_fill(~there[:, None, None], 0.0).abs() + APPROX
        worst = self.e.amax(3, keepdim=True) if k.shape[1] else torch.zeros_like(self.q[..., :1])
        self.worst = worst
        size = self.p @ self.v.abs()
        tiny = 2.0**-30 if self.dtype == torch.float16 else 0.0  # probabilities whose float16 is subnormal
        # (a factor of 1.1: e^x - 1 for the exponents above, up to 0.1)
        bound = (rounding(self.dtype) + 2.2 * worst + total(k.shape[1])) * size + tiny * self.v.abs().sum(2, keepdim=True)
        self.out, self.out_bound = out.transpose(1, 2), (bound + half_step(out, self.dtype)).transpose(1, 2)
        self.lse_bound = 1.1 * worst[..., 0] + 2.0**-22 * self.lse.abs().nan_to_num(0.0, posinf=0.0) + 2.0**-20

    def gradient(self, dout):
        b, h = self.q.shape[:2]
        g, h2 = dout.double().transpose(1, 2), rounding(self.dtype)
        e = 1.1 * self.e + 1.1 * self.worst  # a probability's: its own score's and the sum's
        dp = g @ self.v.transpose(2, 3)
        delta = (self.p * dp).sum(3, keepdim=True)
        ds = self.p * (dp - delta)
        edp = total(g.shape[3]) * (g.abs() @ self.v.abs().transpose(2, 3))
        edelta = (g.abs() * self.out_bound.transpose(1, 2)).sum(3, keepdim=True) + 2.0**-20 * (g.abs() * self.out.transpose(1, 2).abs()).sum(3, keepdim=True)
        eds = ds.abs() * (h2 + 2 * e) + 1.1 * self.p * (edp + edelta)
        tiny_p = 0.0
        if self.dtype == torch.float16 and dout.numel():
            tiny_p = 2.0**-39
            eds = eds + 2.0**-21 * g.abs().amax()
        # a query without keys has no part in anything
        some = self.lse[..., None].isfinite()
        eds, nq = torch.where(some & (self.p > 0) | (eds > 0) & some, eds, 0.0), self.q.shape[2]
        out = {"dq": self.scale * ds @ self.k, "dk": self.scale * ds.transpose(2, 3) @ self.q, "dv": self.p.transpose(2, 3) @ g}
        bound = {"dq": self.scale * (eds @ self.k.abs() + total(self.p.shape[3]) * ds.abs() @ self.k.abs()),
                 "dk": self.scale * (eds.transpose(2, 3) @ self.q.abs() + total(nq) * ds.abs().transpose(2, 3) @ self.q.abs()),
                 "dv": (self.p * (h2 + 2 * e) + tiny_p).transpose(2, 3) @ g.abs() + total(nq) * self.p.transpose(2, 3) @ g.abs()}
        for name in ("dk", "dv"):
            out[name], bound[name] = (t.reshape(b, self.kv_heads, -1, *t.shape[2:]).sum(2) for t in (out[name], bound[name]))
        out = {name: t.transpose(1, 2) for name, t in out.items()}
        return out, {name: 1.01 * bound[name].transpose(1, 2) + half_step(out[name], self.dtype) for name in out}
