"""Plain 64-bit forms of the operators around the linears, for their tests:
torch float64 on the CPU or the GPU, from the formulas in
include/convrot_block.h, sharing no code with the package."""

import math

import torch

NONE, RMS, LAYER = range(3)
EPS = 1e-6


def e4m3_codes(v):
    """e4m3 bit patterns of float32 values, nearest with ties to even, +-448 past the end."""
    return v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def block_scales(X, weights=False):
    """(scales, 448 * (1 / maximum)) of the float32 definition, one for 128 features of each row
    (weights: of 128 rows too), in float32 as the definition has them."""
    r, k = X.shape
    kb = -(-k // 128)
    X = torch.nn.functional.pad(X.float().abs(), (0, kb * 128 - k))
    amax = X.view(r, kb, 128).amax(2)
    if weights:
        rb = -(-r // 128)
        amax = torch.nn.functional.pad(amax, (0, 0, 0, rb * 128 - r)).view(rb, 128, kb).amax(1)
    amax = amax.clamp_min(2.0**-96)
    top = torch.full_like(amax, 448.0)  # tensors: a division by a number is a product with its reciprocal on the GPU
    return amax / top, (torch.ones_like(amax) / amax) * top


def spread(per_block, rows, cols, weights=False):
    if weights:
        per_block = per_block.repeat_interleave(128, 0)[:rows]
    return per_block.repeat_interleave(128, 1)[:, :cols]


def act(v, kind):
    if kind == 1:
        return 0.5 * v * (1 + torch.erf(v / math.sqrt(2.0)))
    if kind == 2:
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v**3)))
    return v


def norm(v, kind, weight=None, bias=None, eps=EPS):
    if kind == LAYER:
        v = v - v.mean(1, keepdim=True)
    if kind != NONE:
        v = v / torch.sqrt((v**2).mean(1, keepdim=True) + eps)
    if weight is not None:
        v = v * weight
    return v if bias is None else v + bias


def gated_norm(x, y=None, gate=None, scale=None, shift=None, rows=None, res_scale=1.0, post=NONE, post_weight=None,
               post_bias=None, pre=RMS, pre_weight=None, pre_bias=None, eps=EPS):
    """(h, n) in the type of x (float64 in the tests); differentiable."""
    sample = torch.arange(x.shape[0], device=x.device) // (rows or max(1, x.shape[0]))
    h = res_scale * x
    if y is not None:
        u = norm(y, post, post_weight, post_bias, eps)
        h = h + (u if gate is None else gate[sample] * u)
    n = norm(h, pre, pre_weight, pre_bias, eps)
    if scale is not None:
        n = n * (1 + scale[sample])
    if shift is not None:
        n = n + shift[sample]
    return h, n


def rotary(v, cos, sin, at, layout, inverse=False):
    """v [b, t, h, d] float64 with the angles of table rows at [b, t]."""
    pairs = cos.shape[1]
    c, s = cos.double()[at][:, :, None], sin.double()[at][:, :, None]
    s = -s if inverse else s
    out = v.clone()
    for i in range(pairs):
        p, q = (i, i + pairs) if layout == 0 else (2 * i, 2 * i + 1)
        a, b = v[..., p], v[..., q]
        out[..., p] = a * c[..., i] - b * s[..., i]
        out[..., q] = b * c[..., i] + a * s[..., i]
    return out


def rounding(dtype):
    """Half a unit in the last place of the type, relative to the value."""
    return {torch.float32: 2.0**-24, torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11}[dtype]
