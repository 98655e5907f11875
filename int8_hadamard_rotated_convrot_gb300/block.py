"""Python binding of the operators around the linears (``include/convrot_block.h``).

What stands between two linears of a transformer block, as CUDA kernels of
libconvrot: a linear on e4m3 codes with block scales, the gated norm with its
gradient, and rotary positions. As in ``convrot``, this module only checks and
marshals arguments; there is no fallback, and a refused call raises
``ConvrotError`` (or TypeError / ValueError for tensors that the C side, which
sees pointers and sizes, cannot check).

The arguments of a call travel as one C struct, packed here in one step.
"""

from __future__ import annotations

import ctypes
import math
import struct
from dataclasses import dataclass

import torch

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

_LINEAR = struct.Struct("@8P3q5qq4i")
_NORM = struct.Struct("@13P3q9q2f4i")
_NORM_BACKWARD = struct.Struct("@20Pq3q8q2f4i")
_ROTARY = struct.Struct("@8P4q12q3q6i")

_lib = None


def _library() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        _lib = _cr.load()
    return _lib


def _stream(device: torch.device, stream) -> int:
    return (torch.cuda.current_stream(device) if stream is None else stream).cuda_stream


def _check(status: int, what: str):
    if status:
        raise ConvrotError(status, what)


def _code(t: torch.Tensor, name: str) -> int:
    code = _DTYPE.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, not {t.dtype}")
    return code


def _matrix(t: torch.Tensor, name: str, dtype, rows: int, cols: int) -> tuple[int, int]:
    """(address, leading dimension) of a [rows, cols] tensor with contiguous rows on the GPU."""
    if t.dtype != dtype or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor of {dtype}")
    if t.shape != (rows, cols):
        raise ValueError(f"{name} has shape {list(t.shape)}; expected [{rows}, {cols}]")
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return t.data_ptr(), ld if rows > 1 else max(ld, cols)


def _vector(t: torch.Tensor | None, name: str, dtype, n: int) -> int:
    if t is None:
        return 0
    if t.dtype != dtype or not t.is_cuda or t.shape != (n,) or (n > 1 and t.stride(0) != 1):
        raise TypeError(f"{name} must be a contiguous CUDA tensor of {dtype} with {n} elements")
    return t.data_ptr()


def _status_ptr(t: torch.Tensor | None) -> int:
    return _vector(t, "dev_status", torch.int32, 1)


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


def fp8_codes(rows: int, k: int, device=None) -> torch.Tensor:
    """An uninitialized [rows, k] code tensor whose rows start on 16 bytes."""
    return torch.empty((rows, -(-k // 16) * 16), dtype=_E4M3, device=device or "cuda")[:, :k]


def empty_fp8_rows(m: int, k: int, device=None) -> Fp8Rows:
    """Allocates (with torch) the buffers that a pack fills."""
    scale = torch.empty((_blocks(k), -(-m // 4) * 4), dtype=torch.float32, device=device or "cuda")
    return Fp8Rows(fp8_codes(m, k, device), scale[:, :m])


def fp8_weights_from_codes(q: torch.Tensor, scale: torch.Tensor) -> Fp8Weights:
    """A checkpoint's codes [n, k] and scales as Fp8Weights, copied only if the rows of q do not
    start on 16 bytes."""
    n, k = q.shape
    if q.stride(1) != 1 or q.stride(0) % 16 or q.data_ptr() % 16:
        codes = fp8_codes(n, k, q.device)
        codes.view(torch.uint8).copy_(q.view(torch.uint8))
        q = codes
    return Fp8Weights(q, scale.to(torch.float32).contiguous())


def _rows_in(X: torch.Tensor, name: str) -> tuple[int, int, int, int, int]:
    if X.dim() != 2:
        raise TypeError(f"{name} must be a 2-D tensor")
    m, k = X.shape
    return _code(X, name), m, k, *_matrix(X, name, X.dtype, m, k)


def _rows_of(x: Fp8Rows, m: int, k: int) -> tuple[int, int, int, int]:
    q, ldq = _matrix(x.q, "q", _E4M3, m, k)
    s, lds = _matrix(x.scale, "scale", torch.float32, _blocks(k), m)
    return q, -(-ldq // 16) * 16 if m <= 1 else ldq, s, lds


def convrot_fp8_pack_activations(X: torch.Tensor, out: Fp8Rows | None = None, stream=None) -> Fp8Rows:
    """Codes and scales of X [m, k] (float32, bfloat16 or float16), one scale for 128 features of a row."""
    dtype, m, k, x, ldx = _rows_in(X, "X")
    out = out or empty_fp8_rows(m, k, X.device)
    q, ldq, s, lds = _rows_of(out, m, k)
    _check(_library().convrot_fp8_pack_activations(x, dtype, m, k, ldx, q, ldq, s, lds, _stream(X.device, stream)),
           "convrot_fp8_pack_activations")
    return out


def convrot_fp8_quantize_weights(W: torch.Tensor, stream=None) -> Fp8Weights:
    """Offline: codes and scales of W [n, k], one scale for each block of 128 x 128."""
    dtype, n, k, w, ldw = _rows_in(W, "W")
    q = fp8_codes(n, k, W.device)
    scale = torch.empty((_blocks(n), _blocks(k)), dtype=torch.float32, device=W.device)
    _check(_library().convrot_fp8_quantize_weights(w, dtype, n, k, ldw, q.data_ptr(), -(-k // 16) * 16,
                                                   scale.data_ptr(), _blocks(k), _stream(W.device, stream)),
           "convrot_fp8_quantize_weights")
    return Fp8Weights(q, scale)


def _weights_of(w: Fp8Weights, k: int) -> tuple[int, int, int, int, int]:
    n = w.q.shape[0]
    q, ldq = _matrix(w.q, "w.q", _E4M3, n, k)
    s, lds = _matrix(w.scale, "w.scale", torch.float32, _blocks(n), _blocks(k))
    return n, q, -(-ldq // 16) * 16 if n <= 1 else ldq, s, lds


def convrot_fp8_linear(x: Fp8Rows, w: Fp8Weights, bias: torch.Tensor | None = None, act: int = ACT_NONE,
                       out: torch.Tensor | None = None, out_dtype: torch.dtype = torch.bfloat16,
                       dev_status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y [m, n] = act(x w^T + b) from packed activations; bias fp32 [n]. Y has out's or out_dtype's type."""
    m, k = x.q.shape
    xq, ldx, xs, ldxs = _rows_of(x, m, k)
    n, wq, ldw, ws, ldws = _weights_of(w, k)
    if out is None:
        out = torch.empty((m, n), dtype=out_dtype, device=x.q.device)
    y, ldy = _matrix(out, "out", out.dtype, m, n)
    args = _LINEAR.pack(xq, xs, wq, ws, _vector(bias, "bias", torch.float32, n), y, 0, _status_ptr(dev_status), m, n,
                        k, ldx, ldxs, ldw, ldws, ldy, 0, 0, _code(out, "out"), act, 0)
    _check(_library().convrot_fp8_linear(args, _stream(out.device, stream)), "convrot_fp8_linear")
    return out


def fp8_pack_linear_work_bytes(m: int, n: int, k: int) -> int:
    """Bytes of the workspace that convrot_fp8_pack_linear needs (0 where it packs on chip)."""
    return int(_library().convrot_fp8_pack_linear_work_bytes(m, n, k))


def convrot_fp8_pack_linear(X: torch.Tensor, w: Fp8Weights, bias: torch.Tensor | None = None, act: int = ACT_NONE,
                            out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
                            work: torch.Tensor | None = None, dev_status: torch.Tensor | None = None,
                            stream=None) -> torch.Tensor:
    """Y [m, n] = act(pack(X) w^T + b): convrot_fp8_pack_activations and convrot_fp8_linear in one call.
    Y has out's, out_dtype's or X's type. ``work`` (uint8) is allocated here when not given."""
    dtype, m, k, x, ldx = _rows_in(X, "X")
    n, wq, ldw, ws, ldws = _weights_of(w, k)
    if out is None:
        out = torch.empty((m, n), dtype=out_dtype or X.dtype, device=X.device)
    y, ldy = _matrix(out, "out", out.dtype, m, n)
    need = _library().convrot_fp8_pack_linear_work_bytes(m, n, k)
    if need and work is None:
        work = torch.empty(need, dtype=torch.uint8, device=X.device)
    elif need and (work.dtype != torch.uint8 or not work.is_cuda or work.dim() != 1 or not work.is_contiguous()
                   or work.numel() < need):
        raise ValueError(f"work must be a contiguous 1-D uint8 CUDA tensor of at least {need} bytes")
    args = _LINEAR.pack(x, 0, wq, ws, _vector(bias, "bias", torch.float32, n), y, work.data_ptr() if need else 0,
                        _status_ptr(dev_status), m, n, k, ldx, 0, ldw, ldws, ldy, work.numel() if need else 0, dtype,
                        _code(out, "out"), act, 0)
    _check(_library().convrot_fp8_pack_linear(args, _stream(X.device, stream)), "convrot_fp8_pack_linear")
    return out


# ---------------------------------------------------------------- the gated norm


def _param_dtype(dtype: torch.dtype, *params) -> torch.dtype:
    """The one type of the parameters given (float32 or the tensors' own)."""
    for p in params:
        if p is not None:
            if p.dtype != torch.float32 and p.dtype != dtype:
                raise TypeError(f"parameters must be float32 or {dtype}, not {p.dtype}")
            return p.dtype
    return torch.float32


def _rows_by_sample(t: torch.Tensor | None, name: str, dtype, batches: int, d: int) -> tuple[int, int]:
    return (0, d) if t is None else _matrix(t, name, dtype, batches, d)


def _gated_norm(x, y, gate, scale, shift, rows_per_batch, res_scale, post, post_weight, post_bias, pre, pre_weight,
                pre_bias, eps, out_h, out_n, packed, stream):
    code, m, d, xp, ldx = _rows_in(x, "x")
    dtype = x.dtype
    rows = rows_per_batch or max(m, 1)
    batches = -(-m // rows)
    p = _param_dtype(dtype, gate, scale, shift, post_weight, post_bias, pre_weight, pre_bias)
    yp, ldy = (0, d) if y is None else _matrix(y, "y", dtype, m, d)
    gp, ldg = _rows_by_sample(gate, "gate", p, batches, d)
    cp, ldc = _rows_by_sample(scale, "scale", p, batches, d)
    fp, ldf = _rows_by_sample(shift, "shift", p, batches, d)
    hp, ldh = (0, d) if out_h is None else _matrix(out_h, "out_h", dtype, m, d)
    np_, ldn = (0, d) if out_n is None else _matrix(out_n, "out_n", dtype, m, d)
    qp, ldq, qs, ldqs = (0, 0, 0, 0) if packed is None else _rows_of(packed, m, d)
    args = _NORM.pack(xp, yp, gp, cp, fp, _vector(post_weight, "post_weight", p, d), _vector(post_bias, "post_bias", p, d),
                      _vector(pre_weight, "pre_weight", p, d), _vector(pre_bias, "pre_bias", p, d), hp, np_, qp, qs, m, d,
                      rows, ldx, ldy, ldg, ldc, ldf, ldh, ldn, ldq, ldqs, res_scale, eps, post, pre, code, _DTYPE[p])
    _check(_library().convrot_gated_norm(args, _stream(x.device, stream)), "convrot_gated_norm")


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
    or x's. Without y and with res_scale 1 and no out_h, the returned h is x itself. out_h may be x (in place)."""
    if out_h is None:
        out_h = x if y is None and res_scale == 1.0 else torch.empty(x.shape, dtype=x.dtype, device=x.device)
    if out_n is None:
        out_n = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    write_h = None if out_h is x and y is None and res_scale == 1.0 else out_h
    _gated_norm(x, y, gate, scale, shift, rows_per_batch, res_scale, post, post_weight, post_bias, pre, pre_weight,
                pre_bias, eps, write_h, out_n, None, stream)
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
        out_h = x if y is None and res_scale == 1.0 else torch.empty(x.shape, dtype=x.dtype, device=x.device)
    out = out or empty_fp8_rows(*x.shape, x.device)
    write_h = None if out_h is x and y is None and res_scale == 1.0 else out_h
    _gated_norm(x, y, gate, scale, shift, rows_per_batch, res_scale, post, post_weight, post_bias, pre, pre_weight,
                pre_bias, eps, write_h, None, out, stream)
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
    code, m, d, hp, ldh = _rows_in(h, "h")
    dtype, dev = h.dtype, h.device
    rows = rows_per_batch or max(m, 1)
    batches = -(-m // rows)
    p = _param_dtype(dtype, gate, scale, shift, post_weight, post_bias, pre_weight, pre_bias)
    yp, ldy = (0, d) if y is None else _matrix(y, "y", dtype, m, d)
    dhp, lddh = (0, d) if dh is None else _matrix(dh, "dh", dtype, m, d)
    dnp, lddn = (0, d) if dn is None else _matrix(dn, "dn", dtype, m, d)
    gp, ldg = _rows_by_sample(gate, "gate", p, batches, d)
    cp, ldc = _rows_by_sample(scale, "scale", p, batches, d)
    _rows_by_sample(shift, "shift", p, batches, d)
    if y is None and not (gate is None and post_weight is None and post_bias is None):
        raise ValueError("gate, post_weight and post_bias belong to a branch y")
    out = {"dx": torch.empty((m, d), dtype=dtype, device=dev),
           "dy": None if y is None else torch.empty((m, d), dtype=dtype, device=dev)}
    # one buffer for the small gradients, cut into views
    wanted = [("dgate", gate, batches), ("dscale", scale, batches), ("dshift", shift, batches),
              ("dpost_weight", post_weight, 1), ("dpost_bias", post_bias, 1), ("dpre_weight", pre_weight, 1),
              ("dpre_bias", pre_bias, 1)]
    small = torch.empty((sum(n for _, t, n in wanted if t is not None), d), dtype=torch.float32, device=dev)
    base, at, addresses = small.data_ptr(), 0, []
    for name, t, n in wanted:
        if t is None:
            out[name] = None
            addresses.append(0)
            continue
        out[name] = small[at:at + n] if t.dim() == 2 else small[at]
        addresses.append(base + at * d * 4)
        at += n
    need = _library().convrot_gated_norm_backward_work_bytes(m, d, rows)
    if work is None:
        work = torch.empty(need, dtype=torch.uint8, device=dev)
    elif work.dtype != torch.uint8 or not work.is_cuda or work.dim() != 1 or not work.is_contiguous() or work.numel() < need:
        raise ValueError(f"work must be a contiguous 1-D uint8 CUDA tensor of at least {need} bytes")
    args = _NORM_BACKWARD.pack(
        hp, yp, dhp, dnp, gp, cp, _vector(post_weight, "post_weight", p, d), _vector(post_bias, "post_bias", p, d),
        _vector(pre_weight, "pre_weight", p, d), _vector(pre_bias, "pre_bias", p, d), out["dx"].data_ptr(),
        0 if y is None else out["dy"].data_ptr(), *addresses, work.data_ptr(), work.numel(), m, d, rows, ldh, ldy, lddh,
        lddn, ldg, ldc, d, d, res_scale, eps, post, pre, code, _DTYPE[p])
    _check(_library().convrot_gated_norm_backward(args, _stream(dev, stream)), "convrot_gated_norm_backward")
    return out


# ---------------------------------------------------------------- rotary positions


def _heads(t: torch.Tensor | None, name: str, like: torch.Tensor) -> tuple[int, int, tuple[int, int, int]]:
    """(address, heads, (batch, token, head) strides) of a [batch, tokens, heads, head_dim] tensor."""
    if t is None:
        return 0, 0, (0, 0, 0)
    if t.dim() != 4 or t.dtype != like.dtype or not t.is_cuda:
        raise TypeError(f"{name} must be a 4-D CUDA tensor of {like.dtype}")
    b, n, h, d = t.shape
    if (b, n, d) != (like.shape[0], like.shape[1], like.shape[3]):
        raise ValueError(f"{name} has shape {list(t.shape)}; expected [{like.shape[0]}, {like.shape[1]}, heads, {like.shape[3]}]")
    *strides, step = t.stride()
    if step != 1 and d > 1:
        raise ValueError(f"{name} must have a contiguous last dimension")
    return t.data_ptr(), h, strides


def convrot_rotary(q: torch.Tensor, k: torch.Tensor | None, cos: torch.Tensor, sin: torch.Tensor,
                   positions: torch.Tensor | None = None, *, layout: int = ROTARY_HALF, inverse: bool = False,
                   out_q: torch.Tensor | None = None, out_k: torch.Tensor | None = None,
                   dev_status: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor | None]:
    """Queries [batch, tokens, heads, head_dim] and keys (k: same, with their own number of heads; or None) with the
    first 2 * cos.shape[1] values of each head turned by the angles of the token's position.

    cos, sin: [rows, pairs] (rotary_table); positions: int32 or int64 [batch, tokens] or [tokens], rows of the table
    (default: token t uses row t). A position outside the table gives NaN and ERR_INVALID_ARG in dev_status.
    inverse turns by the opposite angles (the gradient). Any batch, token and head strides; out_q may be q itself."""
    if q.dim() != 4:
        raise TypeError("q must be [batch, tokens, heads, head_dim]")
    b, t, _, d = q.shape
    if out_q is None:
        out_q = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    if k is not None and out_k is None:
        out_k = torch.empty(k.shape, dtype=k.dtype, device=k.device)
    qp, qh, qs = _heads(q, "q", q)
    kp, kh, ks = _heads(k, "k", q)
    oq, oqh, oqs = _heads(out_q, "out_q", q)
    ok, okh, oks = _heads(out_k if k is not None else None, "out_k", q)
    if (oqh, okh) != (qh, kh):
        raise ValueError("outputs must have as many heads as their inputs")
    rows, pairs = cos.shape
    cp, ldt = _matrix(cos, "cos", torch.float32, rows, pairs)
    sp, ldt_sin = _matrix(sin, "sin", torch.float32, rows, pairs)
    if ldt_sin != ldt:
        raise ValueError("cos and sin must have the same leading dimension")
    pp = stride = bits = 0
    if positions is not None:
        if positions.dtype not in (torch.int32, torch.int64) or not positions.is_cuda:
            raise TypeError("positions must be an int32 or int64 CUDA tensor")
        if positions.shape != (b, t) and positions.shape != (t,):
            raise ValueError(f"positions has shape {list(positions.shape)}; expected [{b}, {t}] or [{t}]")
        if t > 1 and positions.stride(-1) != 1:
            raise ValueError("positions must be contiguous along tokens")
        pp, bits = positions.data_ptr(), positions.element_size() * 8
        stride = positions.stride(0) if positions.dim() == 2 else 0
    args = _ROTARY.pack(qp, kp, oq, ok, cp, sp, pp, _status_ptr(dev_status), b, t, qh, kh, *qs, *ks, *oqs, *oks, rows,
                        ldt, stride, d, 2 * pairs, layout, inverse, _code(q, "q"), bits)
    _check(_library().convrot_rotary(args, _stream(q.device, stream)), "convrot_rotary")
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
                less than beta_slow times are divided by factor, a linear ramp over the pair index in between; the
                attention factor is 0.1 ln(factor) + 1 (Peng et al., "YaRN: Efficient Context Window Extension of
                Large Language Models", sections 3.2 to 3.4)."""
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

    low = max(math.floor(pair_of(beta_fast)), 0)
    high = min(math.ceil(pair_of(beta_slow)), pairs - 1)
    ramp = [min(max((i - low) / max(high - low, 1e-3), 0.0), 1.0) for i in range(pairs)]
    return [f * (1 - r) + f / factor * r for f, r in zip(freq, ramp)], 0.1 * math.log(factor) + 1.0


def convrot_rotary_table(rows: int | torch.Tensor, freq, axis=None, factor: float = 1.0, device=None,
                         stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """cos and sin [rows, pairs] of position * freq, times factor, the angles taken in 64 bits.

    rows: a count (row p is position p), or positions [rows] or [rows, axes] (one for each axis of an image or a
    video; integer or floating point). freq: [pairs] (rotary_frequencies); axis: the axis of each pair."""
    positions = None
    if isinstance(rows, torch.Tensor):
        device = rows.device
        positions = rows.to(torch.float64).reshape(rows.shape[0], -1).contiguous()
        count, axes = positions.shape
    else:
        count, axes = int(rows), 1
    device = torch.device(device or "cuda")
    if device.type != "cuda":
        raise TypeError("positions must be a CUDA tensor")
    freq = torch.as_tensor(freq, dtype=torch.float64).to(device).contiguous()
    pairs = freq.numel()
    if axis is not None:
        axis = torch.as_tensor(axis, dtype=torch.int32).to(device).contiguous()
        if axis.numel() != pairs:
            raise ValueError("axis must name one axis for each frequency")
    cos, sin = (torch.empty((count, pairs), dtype=torch.float32, device=device) for _ in range(2))
    _check(_library().convrot_rotary_table(_cr._ptr(positions), count, axes, freq.data_ptr(), _cr._ptr(axis), pairs,
                                           float(factor), cos.data_ptr(), sin.data_ptr(), pairs, _stream(device, stream)),
           "convrot_rotary_table")
    return cos, sin
