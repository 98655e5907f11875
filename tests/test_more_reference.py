"""The 64-bit forms that the GPU tests compare with (more_reference.py), against autograd and central differences of the
formulas written once more, on the CPU."""

import math

import pytest
import torch

from . import more_reference as ref

F64 = torch.float64


def attention(q, k, v, mask, scale):
    """sum_j softmax_j(scale q_i k_j) v_j, head by head."""
    out = []
    for h in range(q.shape[2]):
        hk = h // (q.shape[2] // k.shape[2])
        s = scale * torch.einsum("btd,bsd->bts", q[:, :, h], k[:, :, hk]).masked_fill(~mask[:, None], -math.inf)
        out.append(torch.softmax(s, 2) @ v[:, :, hk])
    return torch.stack(out, 2)


def inputs(b, tq, tk, hq, hk, d, seed=1):
    g = torch.Generator().manual_seed(seed)
    q, k, v, dout = (torch.randn(b, t, h, d, generator=g, dtype=F64) for t, h in ((tq, hq), (tk, hk), (tk, hk), (tq, hq)))
    mask = torch.rand(b, tk, generator=g) < 0.6
    mask[:, 0] = True  # something is there in each sample
    return 1.5 * q, k, v, dout, mask


@pytest.mark.parametrize("b,tq,tk,hq,hk,d", [(2, 5, 9, 4, 2, 16), (1, 1, 1, 1, 1, 1), (3, 7, 20, 6, 1, 8), (2, 16, 3, 2, 2, 33)])
def test_attention_and_its_gradient(b, tq, tk, hq, hk, d):
    q, k, v, dout, mask = inputs(b, tq, tk, hq, hk, d)
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    want = attention(*leaves, mask, 0.4)
    got = ref.Attention(q, k, v, mask, scale=0.4)
    assert torch.allclose(got.out, want.detach(), rtol=1e-12, atol=1e-12)
    grads, _ = got.gradient(dout)
    for name, t in zip(("dq", "dk", "dv"), torch.autograd.grad(want, leaves, dout)):
        assert torch.allclose(grads[name], t, rtol=1e-9, atol=1e-9), name


def test_attention_gradient_against_differences():
    q, k, v, dout, mask = inputs(2, 4, 6, 4, 2, 8)
    grads, _ = ref.Attention(q, k, v, mask, scale=0.4).gradient(dout)
    for i, name in enumerate(("dq", "dk", "dv")):
        for at in range(0, (q, k, v)[i].numel(), 7):
            step = torch.zeros_like((q, k, v)[i])
            step.view(-1)[at] = 1e-5
            up, down = (float((attention(*(t + s * step if j == i else t for j, t in enumerate((q, k, v))), mask, 0.4) * dout).sum()) for s in (1, -1))
            # the third derivative's part is under 1e-10 times a few, the rounding's under 1e-14 / 1e-5
            assert abs(float(grads[name].reshape(-1)[at]) - (up - down) / 2e-5) <= 1e-7, (name, at)


def test_attention_of_no_keys():
    q, k, v, dout, mask = inputs(2, 3, 4, 2, 1, 8)
    mask[0] = False
    k[0], v[0] = math.nan, math.nan
    got = ref.Attention(q, k, v, mask)
    grads, bounds = got.gradient(dout)
    assert not got.out[0].any() and torch.all(got.lse[0] == -math.inf) and torch.isfinite(got.lse[1]).all()
    assert all(not t[0].any() and torch.isfinite(t).all() for t in grads.values())
    assert all(torch.isfinite(t).all() for t in bounds.values())


def plain_act(v, kind):
    if kind == ref.SILU:
        return v / (1 + torch.exp(-v))
    if kind == 1:
        return 0.5 * v * (1 + torch.erf(v / math.sqrt(2)))
    if kind == 2:
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v**3)))
    return v


@pytest.mark.parametrize("kind", [0, 1, 2, 3])
def test_gated_and_its_gradient(kind):
    g = torch.Generator().manual_seed(kind)
    x, wg, wu, dy = (torch.randn(*s, generator=g, dtype=F64) for s in ((7, 12), (10, 12), (10, 12), (7, 10)))
    bg, bu = (torch.randn(10, generator=g, dtype=F64) for _ in range(2))
    leaves = [t.clone().requires_grad_() for t in (x, wg, wu, bg, bu)]
    gate, up = leaves[0] @ leaves[1].t() + leaves[3], leaves[0] @ leaves[2].t() + leaves[4]
    y = plain_act(gate, kind) * up
    want = torch.autograd.grad(y, leaves, dy)
    (got, got_gate, got_up), _ = ref.gated(x, wg, wu, bg, bu, kind)
    for a, b in ((got, y), (got_gate, gate), (got_up, up)):
        assert torch.allclose(a, b.detach(), rtol=1e-12, atol=1e-12)
    grads, _ = ref.gated_gradient(x, wg, wu, gate.detach(), up.detach(), dy, kind)
    for name, t in zip(("dx", "dw_gate", "dw_up", "db_gate", "db_up"), want):
        assert torch.allclose(grads[name], t, rtol=1e-9, atol=1e-9), name
