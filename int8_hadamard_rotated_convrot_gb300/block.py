"""Python binding of the operators around the linears (``include/convrot_block.h``).

What stands between two linears of a transformer block, as CUDA kernels of
libconvrot: a linear on e4m3 codes with block scales, the gated norm with its
gradient, and rotary positions. As in ``convrot``, this is argument handling
only; there is no fallback, and a refused call raises ``ConvrotError`` (or
TypeError / ValueError for tensors that the C side, which sees pointers and
sizes, cannot check). The tensors are taken apart in native code
(``csrc/block_py.cpp``), because the smallest calls take a few microseconds.
"""

from __future__ import annotations

import importlib.util
import math
import os
from dataclasses import dataclass

import torch

from . import build as _build
from . import convrot as _cr
from .convrot import ACT_GELU_ERF, ACT_GELU_TANH, ACT_NONE, ConvrotError  # noqa: F401

F32, BF16, F16 = range(3)
NORM_NONE, NORM_RMS, NORM_LAYER = range(3)
ROTARY_HALF, ROTARY_INTERLEAVED = range(2)
FP8_BLOCK = 128
NORM_MAX_D = 16384
ROTARY_MAX_D = 4096

_DTYPE = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
_E4M3 = torch.float8_e4m3fn

_native = None


def load():
    """The native marshalling module, loaded (with libconvrot) on first use."""
    global _native
    if _native is None:
        _cr.load()
        path = _build.BLOCK_MODULE
        if not os.path.exists(path):
            raise RuntimeError(f"the block module is not built ({path}); run __graft_entry__.build()")
        spec = importlib.util.spec_from_file_location("_block", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        _native = module
    return _native


def _check(status: int, what: str):
    if status:
        raise ConvrotError(status, what)


def _stream(device: torch.device, stream) -> int:
    return (torch.cuda.current_stream(device) if stream is None else stream).cuda_stream


# ---------------------------------------------------------------- the block-scaled linear


@dataclass
class Fp8Rows:
    """Packed activations: codes q [m, k] (e4m3, rows 16-byte aligned) and scale [ceil(k / 128), >= m]
    with scale[j, r] the scale of row r's block j."""

    q: torch.Tensor
    scale: torch.Tensor

    def dequantize(self) -> torch.Tensor:
        """The fp32 values that the codes stand for (a copy, for checks)."""
        m, k = self.q.shape
        return self.q.float() * self.scale[:, :m].t().repeat_interleave(FP8_BLOCK, 1)[:, :k]


@dataclass
class Fp8Weights:
    """A weight in blocks of 128 x 128: codes q [n, k] (e4m3, rows 16-byte aligned) and scale
    [ceil(n / 128), ceil(k / 128)], as block-scaled checkpoints store them."""

    q: torch.Tensor
    scale: torch.Tensor

    def dequantize(self) -> torch.Tensor:
        n, k = self.q.shape
        return self.q.float() * self.scale.repeat_interleave(FP8_BLOCK, 0)[:n].repeat_interleave(FP8_BLOCK, 1)[:, :k]

    def transposed(self) -> "Fp8Weights":
        """The weight of the linear's input gradient, dX = dY W: the transposed codes under the
        transposed scales (a block is square, so nothing is quantized again). A copy, made once."""
        n, k = self.q.shape
        t = fp8_codes(k, n, self.q.device)
        t.view(torch.uint8).copy_(self.q.view(torch.uint8).t())
        return Fp8Weights(t, self.scale.t().contiguous())


def _blocks(v: int) -> int:
    return -(-v // FP8_BLOCK)


def fp8_codes(rows: int, k: int, device=None, stream=None) -> torch.Tensor:
    """An uninitialized [rows, k] code tensor whose rows start on 16 bytes."""
    return _cr._empty((rows, -(-k // 16) * 16), _E4M3, device or "cuda", stream)[:, :k]


def empty_fp8_rows(m: int, k: int, device=None, stream=None) -> Fp8Rows:
    """Allocates (with torch) the buffers that a pack fills."""
    scale = _cr._empty((_blocks(k), -(-m // 4) * 4), torch.float32, device or "cuda", stream)
    return Fp8Rows(fp8_codes(m, k, device, stream), scale[:, :m])


def fp8_weights_from_codes(q: torch.Tensor, scale: torch.Tensor) -> Fp8Weights:
    """A checkpoint's codes [n, k] and scales as Fp8Weights, copied only if the rows of q do not
    start on 16 bytes. Codes are torch.float8_e4m3fn (bytes: viewed as that)."""
    if q.dtype != _E4M3 or q.dim() != 2:
        raise TypeError("codes must be a 2-D float8_e4m3fn tensor")
    n, k = q.shape
    if q.stride(1) != 1 or q.stride(0) % 16 or q.data_ptr() % 16:
        codes = fp8_codes(n, k, q.device)
        codes.view(torch.uint8).copy_(q.view(torch.uint8))
        q = codes
    return Fp8Weights(q, scale.to(torch.float32).contiguous())


def convrot_fp8_pack_activations(X: torch.Tensor, out: Fp8Rows | None = None, stream=None) -> Fp8Rows:
    """Codes and scales of X [m, k] (float32, bfloat16 or float16), one scale for 128 features of a row."""
    if out is None:
        out = empty_fp8_rows(*X.shape, X.device, stream)
    _check(load().pack_activations(X, out.q, out.scale, stream), "convrot_fp8_pack_activations")
    return out


def convrot_fp8_quantize_weights(W: torch.Tensor, stream=None) -> Fp8Weights:
    """Offline: codes and scales of W [n, k], one scale for each block of 128 x 128."""
    if W.dtype not in _DTYPE or not W.is_cuda or W.dim() != 2 or (W.shape[1] > 1 and W.stride(1) != 1):
        raise TypeError("W must be a 2-D row-major float32, bfloat16 or float16 CUDA tensor")
    n, k = W.shape
    q = fp8_codes(n, k, W.device, stream)
    scale = _cr._empty((_blocks(n), _blocks(k)), torch.float32, W.device, stream)
    with torch.cuda.device(W.device):
        _check(_cr.load().convrot_fp8_quantize_weights(W.data_ptr(), _DTYPE[W.dtype], n, k, W.stride(0) if n > 1 else k,
                                                       q.data_ptr(), -(-k // 16) * 16, scale.data_ptr(), _blocks(k),
                                                       _stream(W.device, stream)), "convrot_fp8_quantize_weights")
    return Fp8Weights(q, scale)


def convrot_fp8_linear(x: Fp8Rows, w: Fp8Weights, bias: torch.Tensor | None = None, act: int = ACT_NONE,
                       out: torch.Tensor | None = None, out_dtype: torch.dtype = torch.bfloat16,
                       dev_status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y [m, n] = act(x w^T + b) from packed activations; bias fp32 [n]. Y has out's or out_dtype's type."""
    if out is None:
        out = _cr._empty((x.q.shape[0], w.q.shape[0]), out_dtype, x.q.device, stream)
    _check(load().linear(x.q, x.scale, w.q, w.scale, bias, act, out, None, dev_status, stream), "convrot_fp8_linear")
    return out


def fp8_pack_linear_work_bytes(m: int, n: int, k: int) -> int:
    """Bytes of the workspace that convrot_fp8_pack_linear needs (0 where it packs on chip)."""
    return _cr.load().convrot_fp8_pack_linear_work_bytes(m, n, k)


def convrot_fp8_pack_linear(X: torch.Tensor, w: Fp8Weights, bias: torch.Tensor | None = None, act: int = ACT_NONE,
                            out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
                            work: torch.Tensor | None = None, dev_status: torch.Tensor | None = None,
                            stream=None) -> torch.Tensor:
    """Y [m, n] = act(pack(X) w^T + b): convrot_fp8_pack_activations and convrot_fp8_linear in one call.
    Y has out's, out_dtype's or X's type. ``work`` (uint8) is allocated here when not given."""
    if out is None:
        out = _cr._empty((X.shape[0], w.q.shape[0]), out_dtype or X.dtype, X.device, stream)
    _check(load().linear(X, None, w.q, w.scale, bias, act, out, work, dev_status, stream), "convrot_fp8_pack_linear")
    return out


# ---------------------------------------------------------------- the gated norm


def convrot_gated_norm(x: torch.Tensor, y: torch.Tensor | None = None, *, gate: torch.Tensor | None = None,
                       scale: torch.Tensor | None = None, shift: torch.Tensor | None = None,
                       rows_per_batch: int | None = None, res_scale: float = 1.0, post: int = NORM_NONE,
                       post_weight: torch.Tensor | None = None, post_bias: torch.Tensor | None = None,
                       pre: int = NORM_RMS, pre_weight: torch.Tensor | None = None,
                       pre_bias: torch.Tensor | None = None, eps: float = 1e-6, out_h: torch.Tensor | None = None,
                       out_n: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """(h, n) with h = res_scale x + gate post(y) and n = pre(h) (1 + scale) + shift, for rows x, y [m, d].

    gate, scale and shift are [batches, d], row r taking sample r // rows_per_batch (default: one sample); norms
    are NORM_NONE, NORM_RMS or NORM_LAYER with optional weight and bias [d]. All parameters have one type, float32
    or x's. Without y there is no gate and no post norm's weight or bias (ValueError); without y and with res_scale 1
    and no out_h, the returned h is x itself. out_h may be x (in place)."""
    if out_h is None:
        out_h = x if y is None and res_scale == 1.0 else _cr._empty(x.shape, x.dtype, x.device, stream)
    if out_n is None:
        out_n = _cr._empty(x.shape, x.dtype, x.device, stream)
    write_h = None if out_h is x and y is None and res_scale == 1.0 else out_h
    _check(load().gated_norm(x, y, gate, scale, shift, rows_per_batch, res_scale, post, post_weight, post_bias, pre,
                                 pre_weight, pre_bias, eps, write_h, out_n, None, None, stream),
           "convrot_gated_norm")
    return out_h, out_n


def convrot_gated_norm_pack(x: torch.Tensor, y: torch.Tensor | None = None, *, gate: torch.Tensor | None = None,
                            scale: torch.Tensor | None = None, shift: torch.Tensor | None = None,
                            rows_per_batch: int | None = None, res_scale: float = 1.0, post: int = NORM_NONE,
                            post_weight: torch.Tensor | None = None, post_bias: torch.Tensor | None = None,
                            pre: int = NORM_RMS, pre_weight: torch.Tensor | None = None,
                            pre_bias: torch.Tensor | None = None, eps: float = 1e-6,
                            out_h: torch.Tensor | None = None, out: Fp8Rows | None = None,
                            stream=None) -> tuple[torch.Tensor, Fp8Rows]:
    """convrot_gated_norm with n written as the packed input of convrot_fp8_linear instead: (h, packed n)."""
    if out_h is None:
        out_h = x if y is None and res_scale == 1.0 else _cr._empty(x.shape, x.dtype, x.device, stream)
    if out is None:
        out = empty_fp8_rows(*x.shape, x.device, stream)
    write_h = None if out_h is x and y is None and res_scale == 1.0 else out_h
    _check(load().gated_norm(x, y, gate, scale, shift, rows_per_batch, res_scale, post, post_weight, post_bias, pre,
                                 pre_weight, pre_bias, eps, write_h, None, out.q, out.scale, stream),
           "convrot_gated_norm")
    return out_h, out


def convrot_gated_norm_backward(h: torch.Tensor, y: torch.Tensor | None, dh: torch.Tensor | None,
                                dn: torch.Tensor | None, *, gate: torch.Tensor | None = None,
                                scale: torch.Tensor | None = None, shift: torch.Tensor | None = None,
                                rows_per_batch: int | None = None, res_scale: float = 1.0, post: int = NORM_NONE,
                                post_weight: torch.Tensor | None = None, post_bias: torch.Tensor | None = None,
                                pre: int = NORM_RMS, pre_weight: torch.Tensor | None = None,
                                pre_bias: torch.Tensor | None = None, eps: float = 1e-6,
                                work: torch.Tensor | None = None, stream=None) -> dict[str, torch.Tensor | None]:
    """The gradients of convrot_gated_norm's inputs, from its output h, its input y and the gradients dh and dn
    of its outputs (None: zero). A dict with dx, dy (of h's type) and, in float32, dgate, dscale, dshift [batches, d]
    and dpost_weight, dpost_bias, dpre_weight, dpre_bias [d]: None for each input that was not given."""
    got = load().gated_norm_backward(h, y, dh, dn, gate, scale, shift, rows_per_batch, res_scale, post, post_weight,
                                         post_bias, pre, pre_weight, pre_bias, eps, work, stream)
    if not isinstance(got, dict):
        raise ConvrotError(got, "convrot_gated_norm_backward")
    return got


# ---------------------------------------------------------------- rotary positions


def convrot_rotary(q: torch.Tensor, k: torch.Tensor | None, cos: torch.Tensor, sin: torch.Tensor,
                   positions: torch.Tensor | None = None, *, layout: int = ROTARY_HALF, inverse: bool = False,
                   out_q: torch.Tensor | None = None, out_k: torch.Tensor | None = None,
                   dev_status: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor | None]:
    """Queries [batch, tokens, heads, head_dim] and keys (k: same, with their own number of heads; or None) with the
    first 2 * cos.shape[1] values of each head turned by the angles of the token's position.

    cos, sin: [rows, pairs] (rotary_table); positions: int32 or int64 [batch, tokens] or [tokens], rows of the table
    (default: token t uses row t). A position outside the table gives NaN and ERR_INVALID_ARG in dev_status.
    inverse turns by the opposite angles (the gradient). Any batch, token and head strides; out_q may be q itself."""
    if out_q is None:
        out_q = _cr._empty(q.shape, q.dtype, q.device, stream)
    if k is None:
        out_k = None
    elif out_k is None:
        out_k = _cr._empty(k.shape, k.dtype, k.device, stream)
    _check(load().rotary(q, k, cos, sin, positions, layout, inverse, out_q, out_k, dev_status, stream), "convrot_rotary")
    return out_q, out_k


def rotary_frequencies(pairs: int, base: float = 10000.0, *, scaling: str = "none", factor: float = 1.0,
                       original_length: int = 0, beta_fast: float = 32.0,
                       beta_slow: float = 1.0) -> tuple[list[float], float]:
    """(frequencies [pairs], attention factor) for rotary_table, in 64 bits.

    Pair i turns by base^(-i / pairs) radians a position. For contexts longer than the ``original_length`` that a
    model was trained on, by ``factor``:
      "linear"  every frequency divided by factor (positions interpolated)
      "ntk"     the base raised by factor^(pairs / (pairs - 1)): the fastest pair keeps its frequency and the slowest
                is divided by factor
      "yarn"    pairs that turn more than beta_fast times over original_length keep their frequency, those that turn
                less than beta_slow times are divided by factor, with a linear ramp over the pair index in between
                (from pair 0 on, where even that one turns less than beta_fast times); the attention factor is
                0.1 ln(factor) + 1. The method, its two limits and the factor are Peng et al.'s, "YaRN: Efficient
                Context Window Extension of Large Language Models", sections 3.2 to 3.4. Their text's ramp is linear
                in the number of turns; the one over the pair index, between the whole indices around both limits, is
                that of their released models, whose checkpoints need it."""
    if pairs < 1 or base <= 0 or factor < 1:
        raise ValueError("pairs >= 1, base > 0 and factor >= 1 are needed")
    if scaling == "ntk" and pairs > 1:
        base = base * factor ** (pairs / (pairs - 1))
    freq = [base ** (-i / pairs) for i in range(pairs)]
    if scaling in ("none", "ntk"):
        return freq, 1.0
    if scaling == "linear":
        return [f / factor for f in freq], 1.0
    if scaling != "yarn":
        raise ValueError(f"unknown scaling {scaling!r}")
    if original_length < 1:
        raise ValueError("yarn needs the original length")

    def pair_of(turns: float) -> float:  # the (real) pair index that turns this often over original_length
        return pairs * math.log(original_length / (turns * 2 * math.pi)) / math.log(base)

    # the ramp's ends, not cut off at the last pair: where even that one turns more than beta_slow times it is part way up
    start, end = max(math.floor(pair_of(beta_fast)), 0), math.ceil(pair_of(beta_slow))

    def divided(i: int) -> float:  # 0: kept, 1: divided by factor
        return min(max(i - start, 0) / (end - start), 1.0) if end > start else float(i > start)

    return [f * (1 - divided(i)) + f / factor * divided(i) for i, f in enumerate(freq)], 0.1 * math.log(factor) + 1.0


def convrot_rotary_table(rows: int | torch.Tensor, freq, axis=None, factor: float = 1.0, device=None,
                         stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """cos and sin [rows, pairs] of position * freq, times factor, the angles taken in 64 bits.

    rows: a count (row p is position p), or positions [rows] or [rows, axes] (one for each axis of an image or a
    video; integer or floating point). freq: [pairs] (rotary_frequencies); axis: the axis of each pair."""
    if isinstance(rows, torch.Tensor):
        device = rows.device
    device = torch.device(device or "cuda")
    if device.type != "cuda":
        raise TypeError("positions must be a CUDA tensor")
    # what is converted here is converted, read and freed on the one stream
    with torch.cuda.device(device), torch.cuda.stream(stream):
        positions = None
        if isinstance(rows, torch.Tensor):
            positions = rows.to(torch.float64).reshape(rows.shape[0], math.prod(rows.shape[1:])).contiguous()
            count, axes = positions.shape
        else:
            count, axes = int(rows), 1
        freq = torch.as_tensor(freq, dtype=torch.float64).to(device).contiguous()
        pairs = freq.numel()
        if axis is not None:
            axis = torch.as_tensor(axis, dtype=torch.int32).to(device).contiguous()
            if axis.numel() != pairs:
                raise ValueError("axis must name one axis for each frequency")
    cos, sin = (_cr._empty((count, pairs), torch.float32, device, stream) for _ in range(2))
    with torch.cuda.device(device):
        _check(_cr.load().convrot_rotary_table(_cr._ptr(positions), count, axes, freq.data_ptr(), _cr._ptr(axis), pairs,
                                               float(factor), cos.data_ptr(), sin.data_ptr(), pairs,
                                               _stream(device, stream)), "convrot_rotary_table")
    return cos, sin
