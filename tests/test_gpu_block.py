"""GPU tests of the operators around the linears against plain 64-bit forms.

Tolerances follow from the arithmetic, before any run:

* a result rounded once to its type is off by half a unit in its last place
  (rounding(dtype) of its size) plus the error of the 32-bit value behind it;
* a 32-bit value that is a sum of terms is off by at most a small multiple of
  2^-24 of the sum of the terms' sizes: C32 = 64 times, for values that went
  through a norm's statistics first (a few roundings each, and sums over a row
  in a tree of at most 16 levels) and were then added up over rows;
* the tensor cores add up products of e4m3 codes, which are exact in fp32, at
  no less than 2^-21 of the sum of the products' sizes in a block of 128
  (CTC), and blocks are added up in fp32.
"""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from int8_hadamard_rotated_convrot_gb300 import block as bl  # noqa: E402
from int8_hadamard_rotated_convrot_gb300 import convrot as cr  # noqa: E402

from . import block_reference as ref  # noqa: E402

U = 2.0**-24
C32 = 64 * U
CTC = 2.0**-21
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from int8_hadamard_rotated_convrot_gb300 import build

    build.build()
    cr.load()
    yield
    torch.cuda.synchronize()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=F32, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def framed(rows, cols, dtype, pad=0, fill=-3.0):
    """(a [rows, cols] view with a larger leading dimension, check that nothing around it was written)"""
    big = torch.full((rows + 2, cols + pad), fill, dtype=dtype, device="cuda")
    view = big[1:rows + 1, :cols]

    def intact():
        assert torch.all(big[0] == fill) and torch.all(big[-1] == fill) and torch.all(big[:, cols:] == fill)

    return view, intact


def close(got, want, bound, what=""):
    """|got - want| <= bound elementwise, both finite."""
    assert got.shape == want.shape, what
    off = (got.double() - want).abs()
    assert torch.isfinite(off).all(), f"{what}: not finite"
    bad = off > bound
    if bad.any():
        at = torch.nonzero(bad)[0].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; first at {at}: got {float(got[tuple(at)])}, "
                             f"want {float(want[tuple(at)])}, off by {float(off[tuple(at)]):.3g}")


def rounded(want, dtype, error32):
    return ref.rounding(dtype) * want.abs() * (1 + 1e-6) + error32 + (2.0**-25 if dtype == F16 else 0.0)


# ---------------------------------------------------------------- quantizers


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=["f32", "bf16", "f16"])
@pytest.mark.parametrize("m,k", [(1, 1), (1, 128), (3, 127), (5, 129), (130, 1000), (64, 2056), (33, 5120), (2, 13824)])
def test_pack_activations(m, k, dtype):
    g = gen(m * 100003 + k)
    big = randn(g, m, k + 3, dtype=dtype)
    big[:, k // 2] *= 50
    if m > 2:
        big[1] = 0
        big[2, :] *= 2.0**-40 if dtype != F16 else 2.0**-10
    for X in (big[:, :k], big[:, :k].contiguous()):  # rows that start anywhere, and aligned ones
        out = bl.empty_fp8_rows(m, k)
        out.q.view(torch.uint8).fill_(0x55)
        bl.convrot_fp8_pack_activations(X, out=out)
        scale, up = ref.block_scales(X)
        assert torch.equal(out.scale.t(), scale)
        assert torch.equal(out.q.view(torch.uint8), ref.e4m3_codes(X.float() * ref.spread(up, m, k)))


@pytest.mark.parametrize("n,k,dtype", [(1, 1, F32), (128, 128, BF16), (200, 300, F16), (300, 1000, F32), (1024, 513, BF16)])
def test_quantize_weights(n, k, dtype):
    W = randn(gen(n + k), n, k, dtype=dtype, std=0.02)
    w = bl.convrot_fp8_quantize_weights(W)
    scale, up = ref.block_scales(W, weights=True)
    assert torch.equal(w.scale, scale)
    assert torch.equal(w.q.view(torch.uint8), ref.e4m3_codes(W.float() * ref.spread(up, n, k, weights=True)))


def test_rows_that_overlap_are_refused():
    one = torch.ones(1, 64, device="cuda").expand(4, 64)
    w = bl.convrot_fp8_quantize_weights(torch.ones(8, 64, device="cuda"))
    for call in (lambda: bl.convrot_fp8_quantize_weights(one), lambda: bl.convrot_fp8_pack_activations(one),
                 lambda: bl.convrot_fp8_pack_linear(one, w), lambda: bl.convrot_gated_norm(one)):
        with pytest.raises(cr.ConvrotError) as e:
            call()
        assert e.value.status == cr.ERR_INVALID_ARG


def test_nan_and_infinity_stay_in_their_rows():
    g = gen(3)
    X = randn(g, 130, 384, dtype=BF16)
    W = bl.convrot_fp8_quantize_weights(randn(g, 200, 384, std=0.02))
    clean = bl.convrot_fp8_pack_linear(X, W)
    X[7, 5] = float("nan")
    X[100, 300] = float("inf")
    for m in (130, 8):  # many rows, and few
        y = bl.convrot_fp8_pack_linear(X[:m], W)
        bad = torch.tensor([r for r in (7, 100) if r < m], device="cuda")
        assert not torch.isfinite(y[bad]).any()
        keep = torch.ones(m, dtype=torch.bool, device="cuda")
        keep[bad] = False
        assert torch.equal(y[keep], bl.convrot_fp8_pack_linear(torch.nan_to_num(X[:m], 0, 0, 0), W)[keep])
    assert torch.isfinite(clean).all()


# ---------------------------------------------------------------- the block-scaled linear


def check_linear(y, x, w, bias, act, dtype):
    """y against the 64-bit sum over the same codes and scales."""
    xd, wd = x.q.double() * ref.spread(x.scale.t()[:x.q.shape[0]].double(), *x.q.shape), w.q.double() * ref.spread(
        w.scale.double(), *w.q.shape, weights=True)
    z = xd @ wd.t()
    blocks = -(-x.q.shape[1] // 128)
    err = (CTC + (blocks + 4) * U) * (xd.abs() @ wd.abs().t())
    if bias is not None:
        z = z + bias.double()
        err = err + U * z.abs()
    want = ref.act(z, act)
    if act:  # |act'| < 1.13; the activation itself is good to 2^-20 of its argument's size
        err = 1.13 * err + 2.0**-20 * z.abs()
    close(y, want, rounded(want, dtype, err), f"{tuple(y.shape)} k {x.q.shape[1]}")


LINEAR = [(1, 128, 128), (1, 5120, 640), (1, 1, 1), (2, 129, 130), (7, 1000, 333), (16, 13824, 256), (17, 4096, 1024),
          (32, 640, 5120), (33, 2056, 3080), (64, 512, 512), (65, 511, 257), (77, 2056, 3080), (128, 1024, 1024),
          (129, 128, 128), (130, 100, 100), (200, 3000, 1000), (256, 256, 256), (257, 384, 520), (300, 16, 2000),
          (513, 2176, 640), (1000, 1111, 777), (2048, 512, 4096), (4097, 640, 1283)]


@pytest.mark.parametrize("m,k,n", LINEAR)
def test_linear(m, k, n):
    g = gen(m * 7 + k * 3 + n)
    X = randn(g, m, k, dtype=BF16)
    X[:, k // 3] *= 50
    w = bl.convrot_fp8_quantize_weights(randn(g, n, k, std=0.05))
    bias = randn(g, n, std=0.1)
    x = bl.convrot_fp8_pack_activations(X)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for dtype, act, b, pad in ((F32, 0, None, 3), (BF16, 2, bias, 0), (F16, 0, bias, 8), (F32, 1, bias, 4)):
        out, intact = framed(m, n, dtype, pad)
        bl.convrot_fp8_linear(x, w, b, act, out=out, dev_status=st)
        intact()
        check_linear(out, x, w, b, act, dtype)
        # the pack inside the call: the same outputs, bit for bit
        both, intact = framed(m, n, dtype, pad)
        bl.convrot_fp8_pack_linear(X, w, b, act, out=both, dev_status=st)
        intact()
        check_linear(both, x, w, b, act, dtype)
    assert int(st) == cr.OK


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=["f32", "bf16", "f16"])
@pytest.mark.parametrize("m", [3, 70, 300])
def test_pack_linear_input_types_and_strides(m, dtype):
    g = gen(m)
    k, n = 520, 384
    w = bl.convrot_fp8_quantize_weights(randn(g, n, k, std=0.05))
    big = randn(g, m, k + 9, dtype=dtype)
    for X in (big[:, :k], big[:, 1:k + 1], big[:, 8:k + 8].contiguous()):
        y = bl.convrot_fp8_pack_linear(X, w, out_dtype=F32)
        check_linear(y, bl.convrot_fp8_pack_activations(X), w, None, 0, F32)


def test_linear_with_checkpoint_strides_and_one_row_of_weights():
    g = gen(5)
    big = randn(g, 300, 1040, std=0.05)
    w = bl.convrot_fp8_quantize_weights(big[:, :1000])
    wide = bl.fp8_codes(300, 2000)
    wide[:, :1000].view(torch.uint8).copy_(w.q.view(torch.uint8))
    wide.view(torch.uint8)[:, 1000:] = 0x7F  # NaN codes past k: not read
    scales = torch.full((3, 20), float("nan"), device="cuda")
    scales[:, :8] = w.scale
    odd = bl.Fp8Weights(wide[:, :1000], scales[:, :8])
    X = randn(g, 200, 1000, dtype=BF16)
    for m in (200, 9):
        assert torch.equal(bl.convrot_fp8_pack_linear(X[:m], odd), bl.convrot_fp8_pack_linear(X[:m], w))
    one = bl.convrot_fp8_quantize_weights(big[:1, :1000])
    for m in (200, 9):
        check_linear(bl.convrot_fp8_pack_linear(X[:m], one, out_dtype=F32), bl.convrot_fp8_pack_activations(X[:m]), one,
                     None, 0, F32)


def test_input_gradient_through_transposed_weights():
    """dX = dY W: the transposed blocks give the same products."""
    g = gen(11)
    W = randn(g, 300, 500, std=0.05)
    w = bl.convrot_fp8_quantize_weights(W)
    t = w.transposed()
    assert torch.equal(t.dequantize(), w.dequantize().t())
    dY = randn(g, 140, 300)
    dx = bl.convrot_fp8_pack_linear(dY, t, out_dtype=F32)
    check_linear(dx, bl.convrot_fp8_pack_activations(dY), t, None, 0, F32)


@pytest.mark.parametrize("m", [4, 500])
def test_linear_is_deterministic_and_captures(m):
    g = gen(m)
    X = randn(g, m, 1024, dtype=BF16)
    w = bl.convrot_fp8_quantize_weights(randn(g, 1536, 1024, std=0.05))
    work = torch.empty(max(1, bl.fp8_pack_linear_work_bytes(m, 1536, 1024)), dtype=torch.uint8, device="cuda")
    out = torch.empty(m, 1536, dtype=F32, device="cuda")
    bl.convrot_fp8_pack_linear(X, w, out=out, work=work)
    first = out.clone()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        bl.convrot_fp8_pack_linear(X, w, out=out, work=work)
    for _ in range(3):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)


# ---------------------------------------------------------------- the gated norm


def norm_case(m, d, rows, dtype, pdtype, post, pre, affine, branch=True, gate=True, modulate=True, res_scale=1.0, seed=0):
    g = gen(seed + m * 31 + d)
    batches = -(-m // rows)
    ada = randn(g, batches, 3 * d + 5, dtype=pdtype, std=0.4)
    v = {"x": randn(g, m, d + 2, dtype=dtype)[:, :d] + (0.5 * randn(g, 1, d)).to(dtype)}
    if branch:
        v["y"] = randn(g, m, d + 8, dtype=dtype, std=0.7)[:, :d]
    if branch and gate:
        v["gate"] = ada[:, :d]
    if modulate:
        v["scale"], v["shift"] = ada[:, d:2 * d], ada[:, 2 * d + 1:3 * d + 1]
    if affine:
        if branch:
            v["post_weight"], v["post_bias"] = randn(g, d, dtype=pdtype), randn(g, d, dtype=pdtype, std=0.1)
        v["pre_weight"], v["pre_bias"] = randn(g, d, dtype=pdtype), randn(g, d, dtype=pdtype, std=0.1)
    how = {"rows": rows, "res_scale": res_scale, "post": post, "pre": pre}
    return v, how


def own_args(how):
    return {"rows_per_batch": how["rows"], "res_scale": how["res_scale"], "post": how["post"], "pre": how["pre"]}


def params(v):
    return {n: t for n, t in v.items() if n not in ("x", "y")}


def norm_bounds(v, how):
    """(h, n, error of h's and of n's 32-bit value): a norm's output is off by a multiple of its row's largest value
    (the statistics' error moves every element by its own size; a mean's error by the size of the row's mean)."""
    wide = {n: t.double() for n, t in v.items()}
    h, n = ref.gated_norm(**wide, **how)
    size = h.abs() + (wide["x"] * how["res_scale"]).abs()
    if "y" in wide:
        u = ref.norm(wide["y"], how["post"], wide.get("post_weight"), wide.get("post_bias"))
        top = u.abs().amax(1, keepdim=True)
        if "gate" in wide:
            top = top * (1 + wide["gate"].abs().amax())
        size = size + top
    e_h = C32 * size
    # pre divides by its own deviation, so h's error is carried along as a multiple of 1 / deviation
    inv = 1.0 if how["pre"] == 0 else 1 / torch.sqrt(((h - (h.mean(1, keepdim=True) if how["pre"] == 2 else 0)) ** 2).mean(1, keepdim=True) + ref.EPS)
    grow = wide["pre_weight"].abs() if "pre_weight" in wide else 1.0
    mod = 1.0
    if "scale" in wide:
        sample = torch.arange(h.shape[0], device="cuda") // how["rows"]
        mod = (1 + wide["scale"][sample]).abs()
    bias = wide["pre_bias"].abs() if "pre_bias" in wide else 0.0
    shift = wide["shift"][sample].abs() if "shift" in wide else 0.0
    e_n = C32 * (n.abs() + shift + mod * bias) + 2 * e_h.amax(1, keepdim=True) * inv * grow * mod
    return h, n, e_h, e_n


NORMS = [
    (1, 1, 1), (3, 2, 1), (2, 7, 2), (5, 64, 2), (4, 127, 4), (9, 128, 3), (7, 130, 5), (33, 1024, 10), (6, 1155, 6),
    (5, 2048, 5), (3, 4096, 1), (4, 5120, 3), (3, 8191, 2), (2, 8192, 2), (2, 12296, 1), (3, 16384, 2), (2, 16383, 2),
    (1030, 256, 500), (700, 1536, 233), (19500, 256, 7000), (6200, 1536, 6200), (2500, 4104, 999)]


@pytest.mark.parametrize("dtype,pdtype", [(F32, F32), (BF16, F32), (BF16, BF16), (F16, F32), (F16, F16)],
                         ids=["f32", "bf16-f32", "bf16", "f16-f32", "f16"])
@pytest.mark.parametrize("m,d,rows", NORMS)
def test_gated_norm(m, d, rows, dtype, pdtype):
    for i, (post, pre, affine, branch, gate, modulate, a) in enumerate([
            (0, 2, False, True, True, True, 1.0), (1, 1, True, True, True, True, 1.0), (2, 2, True, True, False, True, 0.5),
            (0, 1, True, False, False, False, 1.0), (2, 0, False, True, True, False, -2.0), (0, 0, True, True, True, True, 1.0)]):
        v, how = norm_case(m, d, rows, dtype, pdtype, post, pre, affine, branch, gate, modulate, a, seed=i)
        h, n, e_h, e_n = norm_bounds(v, how)
        oh, h_intact = framed(m, d, dtype, 5)
        on, n_intact = framed(m, d, dtype, 8)
        bl.convrot_gated_norm(v["x"], v.get("y"), **params(v), **own_args(how), out_h=oh, out_n=on)
        h_intact(), n_intact()
        close(oh, h, rounded(h, dtype, e_h), f"h, form {i}")
        close(on, n, rounded(n, dtype, e_n), f"n, form {i}")
        # contiguous tensors (the wide loads) and the update in place agree with it
        x = v["x"].contiguous()
        h2, n2 = bl.convrot_gated_norm(x, v["y"].contiguous() if branch else None, **{k: t.contiguous() for k, t in params(v).items()},
                                       **own_args(how), out_h=x)
        assert h2 is x
        close(h2, h, rounded(h, dtype, e_h), f"h in place, form {i}")
        close(n2, n, rounded(n, dtype, e_n), f"n contiguous, form {i}")


@pytest.mark.parametrize("m,d", [(1, 1), (3, 127), (5, 128), (300, 640), (9, 1155), (4, 5120), (2, 16384), (130, 2056)])
def test_gated_norm_pack(m, d):
    """The packed n has the scales and codes of n, up to the codes at a tie of the last bits of n."""
    v, how = norm_case(m, d, max(1, m // 2), BF16, F32, 1, 2, True)
    h, n, e_h, e_n = norm_bounds(v, how)
    oh, packed = bl.convrot_gated_norm_pack(v["x"], v["y"], **params(v), **own_args(how))
    close(oh, h, rounded(h, BF16, e_h), "h")
    scale, _ = ref.block_scales(n)
    kb = scale.shape[1]
    e_block = torch.nn.functional.pad(e_n.expand_as(n), (0, kb * 128 - d)).view(m, kb, 128).amax(2)
    close(packed.scale.t()[:m], scale.double(), e_block / 448 + 4 * U * scale.double(), "scales")
    # a code is off by at most half a step (2^-4 of the value, or half the smallest step 2^-9 of the scale)
    s = ref.spread(scale.double(), m, d)
    close(packed.dequantize(), n, 2.0**-4 * n.abs() * 1.01 + 2.0**-10 * s + 2 * e_n, "codes")
    # and as convrot_fp8_linear's input it is what packing n would be
    w = bl.convrot_fp8_quantize_weights(randn(gen(1), 64, d, std=0.05))
    check_linear(bl.convrot_fp8_linear(packed, w, out_dtype=F32), packed, w, None, 0, F32)


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=["f32", "bf16", "f16"])
@pytest.mark.parametrize("m,d", [(3, 8), (5, 128), (9, 200), (300, 640), (4, 5120), (2, 8200), (3, 16384), (19500, 256), (6200, 1536), (2500, 4104)])
def test_gated_norm_pack_of_aligned_tensors(m, d, dtype):
    """The same where every tensor allows 16-byte accesses: few rows, and runs of many."""
    v, how = norm_case(m, d, max(1, m // 2), dtype, F32, 2, 1, True)
    v = {n: t.contiguous() for n, t in v.items()}
    h, n, e_h, e_n = norm_bounds(v, how)
    q, q_intact = framed(m, -(-d // 16) * 16, torch.uint8, 16, fill=7)
    out = bl.Fp8Rows(q[:, :d].view(torch.float8_e4m3fn), torch.full((-(-d // 128), m), float("nan"), device="cuda"))
    oh, packed = bl.convrot_gated_norm_pack(v["x"], v["y"], **params(v), **own_args(how), out=out)
    assert packed is out
    q_intact()
    assert torch.all(q[:, d:] == 7)
    close(oh, h, rounded(h, dtype, e_h), "h")
    scale, _ = ref.block_scales(n)
    kb = scale.shape[1]
    e_block = torch.nn.functional.pad(e_n.expand_as(n), (0, kb * 128 - d)).view(m, kb, 128).amax(2)
    close(packed.scale.t()[:m], scale.double(), e_block / 448 + 4 * U * scale.double(), "scales")
    s = ref.spread(scale.double(), m, d)
    close(packed.dequantize(), n, 2.0**-4 * n.abs() * 1.01 + 2.0**-10 * s + 2 * e_n, "codes")


def test_gated_norm_special_rows():
    """A row of zeros gives 0 (eps holds the division), and NaN or infinity stays in its row."""
    x = randn(gen(2), 6, 1000, dtype=BF16)
    x[1] = 0
    x[3, 9] = float("nan")
    x[4, 999] = float("inf")
    for kind in (bl.NORM_RMS, bl.NORM_LAYER):
        _, n = bl.convrot_gated_norm(x, pre=kind)
        assert torch.all(n[1] == 0) and torch.isnan(n[3]).any() and torch.isnan(n[4]).any()
        clean = torch.nan_to_num(x, 0, 0, 0)
        _, want = bl.convrot_gated_norm(clean, pre=kind)
        for r in (0, 1, 2, 5):
            assert torch.equal(n[r], want[r])
    big = torch.full((2, 512), 3.0e4, dtype=F16, device="cuda")  # squares past the type's range
    _, n = bl.convrot_gated_norm(big)
    close(n, torch.ones_like(n, dtype=torch.float64), torch.full((2, 512), 2.0**-11, device="cuda"), "large f16 rows")


def test_gated_norm_large_mean():
    """A layer norm whose mean is a thousand deviations away loses no more than the inputs' own bits."""
    x = 1000.0 + randn(gen(8), 5, 3000)
    _, n = bl.convrot_gated_norm(x, pre=bl.NORM_LAYER)
    want = ref.norm(x.double(), 2)
    close(n, want, 16 * U * 1000 + 16 * U * want.abs(), "large mean")


GRADS = [(1, 1, 1), (3, 7, 2), (2, 64, 1), (9, 128, 4), (6, 130, 5), (33, 1024, 10), (77, 1155, 77), (5, 4096, 5),
         (4, 5120, 3), (3, 8191, 2), (2, 12296, 2), (3, 16384, 2), (1030, 256, 500), (700, 1536, 233), (2100, 320, 2100)]


def grad_reference(v, how, dh, dn):
    """Every input's gradient by reverse-mode differentiation in 64 bits, with h as the forward pass stored it."""
    wide = {n: t.double().clone().requires_grad_() for n, t in v.items()}
    x = wide.pop("x")  # plays h
    first = {n: wide[n] for n in ("scale", "shift", "pre_weight", "pre_bias") if n in wide}
    _, n = ref.gated_norm(x, **first, rows=how["rows"], pre=how["pre"])
    got = torch.autograd.grad(n, [x, *first.values()], dn.double())
    d_h = got[0] + dh.double()
    out = {"d" + k: t for k, t in zip(first, got[1:])}
    out["dx"] = how["res_scale"] * d_h
    second = {n: wide[n] for n in ("y", "gate", "post_weight", "post_bias") if n in wide}
    if "y" in second:
        u, _ = ref.gated_norm(torch.zeros_like(x), **second, rows=how["rows"], post=how["post"])
        out |= {"d" + k: t for k, t in zip(second, torch.autograd.grad(u, list(second.values()), d_h))}
    return out, d_h


def grad_bounds(v, how, dh, dn, d_h):
    """The sizes of the terms that each gradient adds up, as 64-bit tensors."""
    w = {n: t.double() for n, t in v.items()}
    sample = torch.arange(w["x"].shape[0], device="cuda") // how["rows"]
    batches = int(sample[-1]) + 1

    def by_sample(t):
        return torch.zeros(batches, t.shape[1], device="cuda", dtype=torch.float64).index_add_(0, sample, t)

    def hat(t, kind):
        mean = t.mean(1, keepdim=True) if kind == 2 else 0.0
        inv = 1.0 if kind == 0 else 1 / torch.sqrt(((t - mean) ** 2).mean(1, keepdim=True) + ref.EPS)
        return ((t - mean) * inv).abs() + 1.0, inv

    one = torch.ones_like(w["x"])
    up = (1 + w["scale"][sample]).abs() if "scale" in w else one
    g = dn.double().abs() * up
    gw = g * w["pre_weight"].abs() if "pre_weight" in w else g
    hh, inv = hat(w["x"], how["pre"])
    e_dh = dh.double().abs() + d_h.abs() + inv * (gw + hh * (gw * hh).mean(1, keepdim=True) + gw.mean(1, keepdim=True))
    out = {"dx": abs(how["res_scale"]) * e_dh}
    affine = hh * w["pre_weight"].abs() + w["pre_bias"].abs() if "pre_weight" in w else hh
    if "scale" in w:
        out["dscale"], out["dshift"] = by_sample(dn.double().abs() * affine), by_sample(dn.double().abs())
    if "pre_weight" in w:
        out["dpre_weight"], out["dpre_bias"] = (g * hh).sum(0), g.sum(0)
    if "y" in w:
        yh, inv = hat(w["y"], how["post"])
        gate = w["gate"][sample].abs() if "gate" in w else one
        affine = yh * w["post_weight"].abs() + w["post_bias"].abs() if "post_weight" in w else yh
        if "gate" in w:
            out["dgate"] = by_sample(e_dh * affine)
        if "post_weight" in w:
            out["dpost_weight"], out["dpost_bias"] = (e_dh * gate * yh).sum(0), (e_dh * gate).sum(0)
        gw = e_dh * gate * (w["post_weight"].abs() if "post_weight" in w else 1.0)
        out["dy"] = inv * (gw + yh * (gw * yh).mean(1, keepdim=True) + gw.mean(1, keepdim=True))
    return out


@pytest.mark.parametrize("dtype,pdtype", [(F32, F32), (BF16, F32), (BF16, BF16), (F16, F16)], ids=["f32", "bf16-f32", "bf16", "f16"])
@pytest.mark.parametrize("m,d,rows", GRADS)
def test_gated_norm_backward(m, d, rows, dtype, pdtype):
    for i, (post, pre, affine, branch, gate, modulate, a) in enumerate([
            (0, 2, False, True, True, True, 1.0), (1, 1, True, True, True, True, 1.0), (2, 2, True, True, False, True, 0.5),
            (0, 1, True, False, False, False, 1.0), (2, 0, False, True, True, False, -2.0), (0, 0, True, True, True, True, 1.0)]):
        v, how = norm_case(m, d, rows, dtype, pdtype, post, pre, affine, branch, gate, modulate, a, seed=i)
        g = gen(i)
        dh, dn = randn(g, m, d + 1, dtype=dtype, std=0.1)[:, 1:], randn(g, m, d, dtype=dtype, std=0.1)
        want, d_h = grad_reference(v, how, dh, dn)
        sizes = grad_bounds(v, how, dh, dn, d_h)
        for contiguous in (False, True):
            w = {n: t.contiguous() if contiguous else t for n, t in v.items()}
            got = bl.convrot_gated_norm_backward(w["x"], w.get("y"), dh.contiguous() if contiguous else dh, dn, **params(w), **own_args(how))
            assert {n for n, t in got.items() if t is not None} == set(want)
            for name, t in want.items():
                bound = C32 * sizes[name]
                if name in ("dx", "dy"):
                    bound = rounded(t, dtype, bound)
                close(got[name], t, bound, f"{name}, form {i}, contiguous {contiguous}")


def test_gated_norm_backward_against_differences():
    """Each gradient against the change of <h, dh> + <n, dn> along a random direction, in 64 bits."""
    m, d, rows = 12, 96, 5
    for post, pre in ((1, 2), (2, 1), (0, 2), (1, 0)):
        v, how = norm_case(m, d, rows, F32, F32, post, pre, True, res_scale=0.7)
        wide = {n: t.double() for n, t in v.items()}
        h, n = ref.gated_norm(**wide, **how)
        g = gen(4)
        dh, dn = randn(g, m, d), randn(g, m, d)
        got = bl.convrot_gated_norm_backward(h.float(), v["y"], dh, dn, **params(v), **own_args(how))
        for name, t in wide.items():
            way = randn(g, *t.shape).double()
            step = 1e-5

            def loss(sign):
                moved = wide | {name: t + sign * step * way}
                hh, nn = ref.gated_norm(**moved, **how)
                return (hh * dh.double()).sum() + (nn * dn.double()).sum()

            change = (loss(1) - loss(-1)) / (2 * step)
            slope = (got["d" + name].double() * way).sum()
            size = (got["d" + name].double() * way).abs().sum()
            # differences: step^2 of the third derivative, about 1e-8 here; gradient: h rounded to 32 bits
            assert abs(float(change - slope)) < 1e-5 * float(size), name


def test_first_call_of_a_process():
    """Sizes whose shared memory is just under or over a launch's default limit, each as the first call of a process
    (a limit that an earlier call raised stays raised)."""
    import os
    import subprocess
    import sys

    code = ("import torch; from int8_hadamard_rotated_convrot_gb300 import block as bl; x = torch.ones(%d, %d, device='cuda').bfloat16(); "
            "bl.convrot_gated_norm_backward(x, x, x, x); bl.convrot_gated_norm(x, x); "
            "bl.convrot_fp8_pack_linear(x, bl.convrot_fp8_quantize_weights(x)); torch.cuda.synchronize()")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    for m, d in ((8, 1536), (8, 1024), (7000, 768)):
        subprocess.run([sys.executable, "-c", code % (m, d)], cwd=root, check=True, timeout=120)


def test_gated_norm_backward_without_dh_or_dn_and_empty():
    v, how = norm_case(40, 200, 13, F32, F32, 1, 2, True)
    dh, dn = randn(gen(1), 40, 200), randn(gen(2), 40, 200)
    zero = torch.zeros_like(dh)
    for a, b in ((None, dn), (dh, None), (None, None)):
        got = bl.convrot_gated_norm_backward(v["x"], v["y"], a, b, **params(v), **own_args(how))
        want = bl.convrot_gated_norm_backward(v["x"], v["y"], zero if a is None else a, zero if b is None else b, **params(v), **own_args(how))
        for name in want:
            assert torch.equal(got[name], want[name]), name
    e = torch.empty(0, 64, device="cuda")
    got = bl.convrot_gated_norm_backward(e, None, e, e, pre_weight=torch.ones(64, device="cuda"))
    assert got["dx"].shape == (0, 64) and torch.all(got["dpre_weight"] == 0)
    h, n = bl.convrot_gated_norm(e, e)
    assert h.shape == n.shape == (0, 64)


def test_gated_norm_is_deterministic_on_another_stream():
    v, how = norm_case(513, 1536, 200, BF16, F32, 1, 1, True)
    dh, dn = randn(gen(1), 513, 1536, dtype=BF16), randn(gen(2), 513, 1536, dtype=BF16)
    first = bl.convrot_gated_norm_backward(v["x"], v["y"], dh, dn, **params(v), **own_args(how))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = bl.convrot_gated_norm_backward(v["x"], v["y"], dh, dn, **params(v), **own_args(how), stream=side)
    side.synchronize()
    for name in first:
        assert torch.equal(first[name], again[name]), name


# ---------------------------------------------------------------- rotary positions


def check_rotary(got, v, cos, sin, at, layout, inverse, dtype):
    want = ref.rotary(v.double(), cos, sin, at, layout, inverse)
    size = ref.rotary(v.double().abs(), cos.abs(), -sin.abs(), at, layout).abs() + v.double().abs()
    close(got, want, rounded(want, dtype, 4 * U * size), "rotary")


ROTARY = [(1, 1, 1, 0, 2, 2), (2, 3, 4, 2, 8, 8), (8, 1, 40, 8, 128, 128), (1, 130, 3, 3, 64, 32), (3, 33, 24, 24, 96, 48),
          (2, 17, 5, 1, 72, 72), (1, 9, 7, 7, 80, 30), (2, 5, 2, 2, 130, 66), (1, 300, 16, 4, 256, 128), (1, 2, 1, 1, 4096, 4096),
          (4, 50, 12, 2, 128, 64)]


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=["f32", "bf16", "f16"])
@pytest.mark.parametrize("layout", [0, 1], ids=["half", "interleaved"])
@pytest.mark.parametrize("b,t,hq,hk,d,r", ROTARY)
def test_rotary(b, t, hq, hk, d, r, layout, dtype):
    g = gen(b + t + d)
    rows = t + 50
    cos, sin = bl.convrot_rotary_table(rows, bl.rotary_frequencies(r // 2)[0])
    qkv = randn(g, b, t, hq + 2 * hk, d, dtype=dtype)
    q, k = qkv[:, :, :hq], qkv[:, :, hq:hq + hk] if hk else None
    pos64 = torch.randint(0, rows, (b, t), generator=g, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    straight = torch.arange(t, device="cuda").expand(b, t)
    for positions, at in ((None, straight), (pos64, pos64), (pos64.int(), pos64), (pos64[0].contiguous(), pos64[0].expand(b, t))):
        for inverse in (False, True):
            oq, ok = bl.convrot_rotary(q, k, cos, sin, positions, layout=layout, inverse=inverse, dev_status=st)
            check_rotary(oq, q, cos, sin, at, layout, inverse, dtype)
            if k is not None:
                check_rotary(ok, k, cos, sin, at, layout, inverse, dtype)
    # heads before tokens, odd strides, and in place, each with the last result's values
    oq, ok = bl.convrot_rotary(q, k, cos, sin, pos64, layout=layout)
    odd = torch.full((b, hq, t, d + 1), -3.0, dtype=dtype, device="cuda")
    odd[..., :d] = q.transpose(1, 2)
    view = odd[..., :d].transpose(1, 2)
    got, _ = bl.convrot_rotary(view, None, cos, sin, pos64, layout=layout, out_q=view)
    assert got is view and torch.equal(got, oq) and torch.all(odd[..., d] == -3.0)
    kept = qkv[:, :, hq + hk:].clone()
    bl.convrot_rotary(q, k, cos, sin, pos64, layout=layout, out_q=q, out_k=k, dev_status=st)
    assert torch.equal(q, oq) and (k is None or torch.equal(k, ok)) and torch.equal(qkv[:, :, hq + hk:], kept)
    assert int(st) == cr.OK


def test_rotary_gradient_is_the_adjoint():
    """<R x, g> = <x, R' g> in 64 bits over the kernel's outputs, for the forward and the inverse call."""
    g = gen(6)
    cos, sin = bl.convrot_rotary_table(64, *bl.rotary_frequencies(16)[:1], factor=1.2)
    x, up = randn(g, 2, 64, 3, 40), randn(g, 2, 64, 3, 40)
    for layout in (0, 1):
        y, _ = bl.convrot_rotary(x, None, cos, sin, layout=layout)
        back, _ = bl.convrot_rotary(up, None, cos, sin, layout=layout, inverse=True)
        left, right = (y.double() * up.double()).sum(), (x.double() * back.double()).sum()
        assert abs(float(left - right)) < 8 * U * float((y.double() * up.double()).abs().sum())


def test_rotary_positions_outside_the_table():
    g = gen(9)
    cos, sin = bl.convrot_rotary_table(10, bl.rotary_frequencies(16)[0])
    q = randn(g, 1, 4, 2, 48)
    for bad in (10, -1, 1 << 40):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        at = torch.tensor([[0, bad, 9, 3]], device="cuda")
        got, _ = bl.convrot_rotary(q, None, cos, sin, at, dev_status=st)
        assert int(st) == cr.ERR_INVALID_ARG
        assert torch.isnan(got[0, 1, :, :32]).all() and torch.equal(got[0, 1, :, 32:], q[0, 1, :, 32:])
        ok = torch.tensor([0, 2, 3], device="cuda")
        check_rotary(got[:, ok], q[:, ok], cos, sin, at[:, ok], 0, False, F32)
        bl.convrot_rotary(q, None, cos, sin, at)  # no status word: the same, silently


def test_rotary_table():
    """Late positions keep their angles, several axes take each its own, and an axis that is not there gives NaN."""
    freq, factor = bl.rotary_frequencies(32, 10000.0, scaling="yarn", factor=8.0, original_length=4096)
    at = torch.tensor([0, 1, 4095, 32767, 131071, 10_000_019], device="cuda")
    cos, sin = bl.convrot_rotary_table(at, freq, factor=factor)
    angle = at.double()[:, None] * torch.tensor(freq, dtype=torch.float64, device="cuda")
    close(cos, factor * angle.cos(), torch.full_like(angle, 1e-7 + 2e-9), "cos")
    close(sin, factor * angle.sin(), torch.full_like(angle, 1e-7 + 2e-9), "sin")
    grid = torch.stack(torch.meshgrid(torch.arange(3), torch.arange(5), torch.arange(7), indexing="ij"), -1).reshape(-1, 3).cuda()
    axis = [0] * 8 + [1] * 12 + [2] * 12
    cos, sin = bl.convrot_rotary_table(grid, freq, axis)
    angle = grid.double()[:, axis] * torch.tensor(freq, dtype=torch.float64, device="cuda")
    close(cos, angle.cos(), torch.full_like(angle, 1e-7), "cos of three axes")
    close(sin, angle.sin(), torch.full_like(angle, 1e-7), "sin of three axes")
    cos, _ = bl.convrot_rotary_table(grid, freq, [0] * 31 + [3])
    assert torch.isnan(cos[:, 31]).all() and torch.isfinite(cos[:, :31]).all()
    cos, sin = bl.convrot_rotary_table(0, freq, device="cuda")
    assert cos.shape == (0, 32)


@pytest.mark.parametrize("d", [5121, 8200, 10248, 16384])
def test_wide_gradient_of_a_row_a_cluster(d):
    """One row for each cluster, so that every sum is the first that its blocks exchange: many clusters, back to back."""
    m = 304
    g = gen(d)
    h, y, dh, dn = (randn(g, m, d, dtype=BF16) for _ in range(4))
    got = [bl.convrot_gated_norm_backward(h, y, dh, dn, rows_per_batch=1, post=bl.NORM_RMS, pre=bl.NORM_RMS) for _ in range(20)]
    v = {"x": h, "y": y}
    how = {"rows": 1, "res_scale": 1.0, "post": 1, "pre": 1}
    want, d_h = grad_reference(v, how, dh, dn)
    sizes = grad_bounds(v, how, dh, dn, d_h)
    for name in ("dx", "dy"):
        close(got[0][name], want[name], rounded(want[name], BF16, C32 * sizes[name]), name)
        for other in got[1:]:
            assert torch.equal(other[name], got[0][name]), name


@pytest.mark.parametrize("m,k,n", [(20, 1024, 2048), (64, 5120, 640), (300, 1024, 2048)])
def test_linears_read_what_the_call_before_wrote(m, k, n):
    """Packs and linears back to back over the same buffers, each starting while the one before drains."""
    g = gen(m)
    X = [randn(g, m, k, dtype=BF16) * 2.0**i for i in range(8)]
    w = bl.convrot_fp8_quantize_weights(randn(g, n, k, std=0.05))
    biases = torch.empty(8, n, device="cuda")
    want = []
    for i, x in enumerate(X):
        packed = bl.convrot_fp8_pack_activations(x)
        torch.cuda.synchronize()
        want.append(bl.convrot_fp8_linear(packed, w, out_dtype=F32))
        torch.cuda.synchronize()
        # a linear's outputs as the next one's bias, too
        biases[i] = want[-1][0]
        want[-1] = (want[-1], bl.convrot_fp8_linear(packed, w, biases[i], out_dtype=F32))
    packed = bl.empty_fp8_rows(m, k)
    y, z = (torch.empty(8, m, n, device="cuda") for _ in range(2))
    for _ in range(5):
        y.zero_(), z.zero_()
        for i, x in enumerate(X):
            bl.convrot_fp8_pack_activations(x, out=packed)
            bl.convrot_fp8_linear(packed, w, out=y[i])
            bl.convrot_fp8_linear(packed, w, y[i][0], out=z[i])
        for i in range(8):
            assert torch.equal(y[i], want[i][0]) and torch.equal(z[i], want[i][1])


# ---------------------------------------------------------------- streams


def stream_calls():
    """name -> call(stream) for every call that allocates, its inputs made and finished beforehand"""
    g = gen(21)
    X, W = randn(g, 300, 1024, dtype=BF16), randn(g, 640, 1024, std=0.05)
    w = bl.convrot_fp8_quantize_weights(W)
    packed = bl.convrot_fp8_pack_activations(X)
    forms = {}
    for name, (m, d) in {"small": (40, 1024), "large": (900, 3000)}.items():  # workspaces under and over 2 MB
        v, how = norm_case(m, d, 50, BF16, F32, 1, 2, True)
        dh, dn = randn(g, m, d, dtype=BF16), randn(g, m, d, dtype=BF16)
        forms["gradient, " + name] = lambda s, v=v, how=how, dh=dh, dn=dn: list(bl.convrot_gated_norm_backward(
            v["x"], v["y"], dh, dn, **params(v), **own_args(how), stream=s).values())
        forms["norm, " + name] = lambda s, v=v, how=how: list(bl.convrot_gated_norm(
            v["x"], v["y"], **params(v), **own_args(how), stream=s))

    def rows(p):
        return [p.q.view(torch.uint8), p.scale]

    cos, sin = bl.convrot_rotary_table(500, bl.rotary_frequencies(32)[0])
    q, k = randn(g, 2, 500, 6, 64), randn(g, 2, 500, 2, 64)
    return forms | {
        "norm pack": lambda s: rows(bl.convrot_gated_norm_pack(X, stream=s)[1]),
        "pack": lambda s: rows(bl.convrot_fp8_pack_activations(X, stream=s)),
        "quantize": lambda s: rows(bl.convrot_fp8_quantize_weights(W, stream=s)),
        "linear": lambda s: [bl.convrot_fp8_linear(packed, w, stream=s)],
        "pack and linear": lambda s: [bl.convrot_fp8_pack_linear(X, w, stream=s)],
        "rotary": lambda s: list(bl.convrot_rotary(q, k, cos, sin, stream=s)),
    }


STREAM_CALLS = ["gradient, small", "norm, small", "gradient, large", "norm, large", "norm pack", "pack", "quantize", "linear",
                "pack and linear", "rotary"]


@pytest.mark.parametrize("name", STREAM_CALLS)
def test_memory_of_a_call_on_another_stream(name):
    """The call's stream is late: what the caller allocates and fills meanwhile is not the call's workspace. Then the
    caller's stream is late: what it still writes into freed memory does not reach the call's outputs."""
    call = stream_calls()[name]
    want = [t.clone() for t in call(None) if t is not None]
    sizes = [max(256, t.numel() * t.element_size()) for t in want] + [1 << 20, 3 << 20, 300 * 1024 + (300 * 8 * 4), 12 << 20]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()

    def fill():
        return [torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]

    for late in (side, torch.cuda.current_stream()):
        for _ in range(3):
            torch.cuda.empty_cache()
            with torch.cuda.stream(late):
                torch.cuda._sleep(20_000_000)  # 10 ms
            if late is side:
                got = [t for t in call(side) if t is not None]
                kept = fill()
            else:
                kept = fill()
                del kept  # their memory is free for the current stream's next tensors, behind the fills
                got = [t for t in call(side) if t is not None]
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want, strict=True))


def test_outputs_of_another_stream_outlive_their_last_use():
    """An output freed while the caller's stream still has to read it: the call's stream does not write over it."""
    g = gen(22)
    X, w = randn(g, 300, 1024, dtype=BF16), bl.convrot_fp8_quantize_weights(randn(g, 640, 1024, std=0.05))
    want = bl.convrot_fp8_pack_linear(X, w)
    side, zero = torch.cuda.Stream(), torch.zeros_like(X)
    torch.cuda.synchronize()
    for _ in range(3):
        y = bl.convrot_fp8_pack_linear(X, w, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(20_000_000)
        copy = y.clone()
        del y
        others = [bl.convrot_fp8_pack_linear(zero, w, stream=side) for _ in range(4)]
        torch.cuda.synchronize()
        assert torch.equal(copy, want) and not any(o.any() for o in others)


def test_tables_on_another_stream():
    """Positions that the call's stream makes, converted where it reads them, and not overwritten while it does."""
    freq, _ = bl.rotary_frequencies(64)
    axis = [i % 3 for i in range(64)]
    side = torch.cuda.Stream()
    want = bl.convrot_rotary_table(torch.arange(30000, device="cuda").view(-1, 3), freq, axis)
    torch.cuda.synchronize()
    for _ in range(3):
        torch.cuda.empty_cache()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
            at = torch.arange(30000, device="cuda").view(-1, 3)
        got = bl.convrot_rotary_table(at, freq, axis, stream=side)
        kept = [torch.full((n,), 3.0, dtype=torch.float64, device="cuda") for n in (30000, 64, 32, 10000 * 32) for _ in range(2)]
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        del kept


def test_kept_gradients_hold_their_own_memory_alone():
    import io

    v, how = norm_case(60, 1024, 20, BF16, F32, 2, 2, True)
    dh, dn = randn(gen(1), 60, 1024, dtype=BF16), randn(gen(2), 60, 1024, dtype=BF16)
    got = bl.convrot_gated_norm_backward(v["x"], v["y"], dh, dn, **params(v), **own_args(how))
    assert len({t.untyped_storage().data_ptr() for t in got.values()}) == len(got)
    for name, t in got.items():
        assert t.is_contiguous() and t.untyped_storage().nbytes() == t.numel() * t.element_size(), name
        assert not t.requires_grad and t.device == v["x"].device
    saved = io.BytesIO()
    torch.save(got["dpre_weight"], saved)
    assert saved.tell() < 2 * 4 * 1024


# ---------------------------------------------------------------- infinite values


@pytest.mark.parametrize("pre", [0, 1, 2])
@pytest.mark.parametrize("m,d,pad", [(5, 256, 0), (19500, 256, 0), (19500, 258, 0), (19500, 257, 0), (6200, 1536, 8)])
def test_gated_norm_of_an_infinite_scale(m, d, pad, pre):
    """(1 + scale) times a finite value, then a finite shift: infinite with the value's sign, in every form of the kernel."""
    g = gen(m + d)
    x = randn(g, m, d + pad, dtype=BF16)[:, :d]
    scale, shift = randn(g, 1, d), randn(g, 1, d)
    scale[0, 3], scale[0, d - 1] = float("inf"), float("-inf")
    for kw in (dict(shift=shift), dict(), dict(shift=shift, pre_weight=randn(g, d))):
        _, n = bl.convrot_gated_norm(x, scale=scale, pre=pre, **kw)
        _, want = ref.gated_norm(x.double(), scale=scale.double(), pre=pre, **{k: t.double() for k, t in kw.items()})
        for c in (3, d - 1):
            keep = torch.isinf(want[:, c])  # (a value of exactly zero times infinity is NaN)
            assert keep.sum() >= m - m // 50 - 1 and torch.equal(n[keep, c].double(), want[keep, c])
        rest = torch.ones(d, dtype=torch.bool, device="cuda")
        rest[[3, d - 1]] = False
        assert torch.isfinite(n[:, rest]).all()


@pytest.mark.parametrize("pre,post", [(0, 1), (1, 0), (2, 2)])
@pytest.mark.parametrize("m,d", [(40, 256), (7, 257), (5, 6000)])
def test_infinite_values_stay_in_their_rows_of_dx_and_dy(m, d, pre, post):
    g = gen(m + d + post)
    h, y, dh, dn = (randn(g, m, d, dtype=F16) for _ in range(4))
    kw = dict(scale=randn(g, 1, d, std=0.3), gate=randn(g, 1, d), pre=pre, post=post, post_weight=randn(g, d))
    want = bl.convrot_gated_norm_backward(h, y, dh, dn, **kw)
    h[1, 5], h[2, d - 1], y[4, 0] = float("inf"), float("-inf"), float("inf")
    got = bl.convrot_gated_norm_backward(h, y, dh, dn, **kw)
    for r in range(m):
        if r not in (1, 2, 4):
            assert torch.equal(got["dx"][r], want["dx"][r]) and torch.equal(got["dy"][r], want["dy"][r])


# ---------------------------------------------------------------- sizes past a grid's limit, none, and one


def test_quantize_weights_of_very_many_rows():
    n = 65535 * 128 + 130
    W = torch.zeros(n, 1, device="cuda", dtype=BF16)
    W[::1000] = 3.0
    W[-1] = -5.0
    w = bl.convrot_fp8_quantize_weights(W)
    scale, up = ref.block_scales(W, weights=True)
    assert torch.equal(w.scale, scale)
    assert torch.equal(w.q.view(torch.uint8), ref.e4m3_codes(W.float() * ref.spread(up, n, 1, weights=True)))


def test_rotary_table_of_no_positions():
    freq, _ = bl.rotary_frequencies(8)
    for at in (torch.empty(0, device="cuda"), torch.empty(0, 1, device="cuda", dtype=torch.int64)):
        cos, sin = bl.convrot_rotary_table(at, freq)
        assert cos.shape == sin.shape == (0, 8)
    cos, _ = bl.convrot_rotary_table(torch.empty(0, 3, device="cuda"), freq, [0, 1, 2, 0, 1, 2, 0, 1])
    assert cos.shape == (0, 8)


def test_rotary_with_a_table_of_one_row():
    """One row has no leading dimension: cosines and sines of different strides are the same table."""
    g = gen(31)
    q = randn(g, 3, 1, 4, 32)
    cos, sin = bl.convrot_rotary_table(torch.tensor([7.0], device="cuda"), bl.rotary_frequencies(16)[0])
    wide = torch.zeros(1, 40, device="cuda")
    wide[:, 8:24] = cos
    want, _ = bl.convrot_rotary(q, None, cos, sin)
    for c, s in ((wide[:, 8:24], sin), (cos, sin.as_strided((1, 16), (3, 1)))):
        got, _ = bl.convrot_rotary(q, None, c, s)
        assert torch.equal(got, want)


def test_rotary_of_single_batches_tokens_and_heads_at_any_strides():
    """What there is one of has no stride to speak of, in place as well."""
    g = gen(33)
    cos, sin = bl.convrot_rotary_table(4, bl.rotary_frequencies(16)[0])
    for b, t, h in ((1, 4, 3), (2, 1, 3), (2, 4, 1), (1, 1, 1)):
        q = randn(g, b, t, h, 32)
        want, _ = bl.convrot_rotary(q, None, cos, sin)
        strides = [0 if n == 1 else s for n, s in zip(q.shape[:3], q.stride()[:3])] + [1]
        out = torch.empty_like(q)
        bl.convrot_rotary(q, None, cos, sin, out_q=out.as_strided(q.shape, strides))
        assert torch.equal(out, want)
        bl.convrot_rotary(q, None, cos, sin, out_q=q.as_strided(q.shape, strides))
        assert torch.equal(q, want)


def test_gradients_are_ordinary_tensors_and_capture():
    v, how = norm_case(60, 1024, 20, BF16, F32, 2, 2, True)
    dh, dn = randn(gen(1), 60, 1024, dtype=BF16), randn(gen(2), 60, 1024, dtype=BF16)
    call = lambda: bl.convrot_gated_norm_backward(v["x"], v["y"], dh, dn, **params(v), **own_args(how))
    want = call()
    got = call()
    leaf = got["dpre_weight"].clone().requires_grad_()
    (leaf * got["dpre_bias"]).sum().backward()  # as a constant of a graph
    assert torch.equal(leaf.grad, want["dpre_bias"])
    got["dscale"].add_(1).mul_(2)
    assert torch.equal(got["dscale"], (want["dscale"] + 1) * 2)
    weight = torch.nn.Parameter(torch.zeros(1024, device="cuda"))
    weight.grad = got["dpre_weight"]
    torch.optim.SGD([weight], lr=1.0).step()
    assert torch.equal(weight.detach(), -want["dpre_weight"])
    with torch.inference_mode():
        assert torch.equal(call()["dgate"], want["dgate"])
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    X, w = randn(gen(3), 300, 512), bl.convrot_fp8_quantize_weights(randn(gen(4), 256, 512))
    y = bl.convrot_fp8_pack_linear(X, w)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):  # with the workspaces that the calls allocate
        kept, z = call(), bl.convrot_fp8_pack_linear(X, w)
    for _ in range(3):
        for t in (*kept.values(), z):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(kept[n], want[n]) for n in want) and torch.equal(z, y)
