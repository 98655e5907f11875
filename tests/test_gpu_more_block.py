"""GPU tests of the gated feed-forward's projections and of attention to other
states against plain 64-bit forms (more_reference.py, where the bounds are derived)."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from int8_hadamard_rotated_convrot_gb300 import block as bl  # noqa: E402
from int8_hadamard_rotated_convrot_gb300 import convrot as cr  # noqa: E402

from . import more_reference as ref  # noqa: E402

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
TYPES = pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
ACTS = (bl.ACT_SILU, bl.ACT_GELU_ERF, bl.ACT_GELU_TANH, bl.ACT_NONE)


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


def close(got, want, bound, what=""):
    """|got - want| <= bound elementwise, both finite."""
    assert got.shape == want.shape, (what, got.shape, want.shape)
    off = (got.double() - want).abs()
    assert torch.isfinite(off).all(), f"{what}: not finite"
    bad = off > bound
    if bad.any():
        at = tuple(torch.nonzero(bad)[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; first at {at}: got {float(got[at])}, "
                             f"want {float(want[at])}, off by {float(off[at]):.3g}, bound {float(bound[at]):.3g}")


# ---------------------------------------------------------------- the gated linear

GATED = [(1, 64, 64), (1, 1, 1), (2, 17, 3), (7, 256, 128), (16, 640, 200), (17, 128, 1000), (33, 72, 264), (64, 1024, 384), (77, 2056, 328),
         (128, 192, 128), (129, 256, 130), (200, 515, 77), (256, 128, 256), (257, 1000, 129), (300, 64, 640), (513, 320, 520), (1023, 200, 136)]


def gated_inputs(m, k, n, dtype, bias=True, pad=0):
    g = gen(m * 10007 + k * 101 + n)
    x = randn(g, m, k + pad, dtype=dtype)[:, :k]
    wg, wu = (randn(g, n, k + pad, dtype=dtype, std=k**-0.5)[:, :k] for _ in range(2))
    biases = [randn(g, n, std=0.3) for _ in range(2)] if bias else [None, None]
    return g, x, wg, wu, *biases


@TYPES
@pytest.mark.parametrize("m,k,n", GATED)
def test_gated_linear(m, k, n, dtype):
    for i, act in enumerate(ACTS):
        _, x, wg, wu, bg, bu = gated_inputs(m, k, n, dtype, bias=i % 2 == 0, pad=(0, 8, 3, 1)[i])
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = bl.convrot_gated_linear(x, wg, wu, bg, bu, act, keep=True, dev_status=status)
        want, bound = ref.gated(x, wg, wu, bg, bu, act)
        for name, a, b, c in zip(("y", "gate", "up"), got, want, bound):
            close(a, b, c, f"{name}, act {act}")
        assert torch.equal(bl.convrot_gated_linear(x, wg, wu, bg, bu, act), got[0])  # without keeping, and twice the same
        assert int(status) == 0


@TYPES
def test_gated_linear_writes_its_rows_alone(dtype):
    """Outputs with a leading dimension of their own, at any alignment; the two halves of one weight; one bias alone."""
    for m, k, n, pad, first in ((5, 64, 40, 8, 0), (5, 64, 40, 3, 1), (300, 128, 200, 8, 8), (300, 128, 201, 5, 1)):
        g = gen(m + n)
        x, w, b = randn(g, m, k, dtype=dtype), randn(g, 2 * n, k, dtype=dtype, std=k**-0.5), randn(g, n)
        big = torch.full((m + 2, n + pad + first), -3.0, dtype=dtype, device="cuda")
        out = big[1:m + 1, first:first + n]
        bl.convrot_gated_linear(x, w[:n], w[n:], b, out=out)
        (want, _, _), (bound, _, _) = ref.gated(x, w[:n], w[n:], b)
        close(out, want, bound)
        rest = big.clone()
        rest[1:m + 1, first:first + n] = -3.0
        assert torch.all(rest == -3.0)


@TYPES
@pytest.mark.parametrize("m,k,n", GATED)
def test_gated_linear_gradient(m, k, n, dtype):
    for i, act in enumerate(ACTS):
        g, x, wg, wu, _, _ = gated_inputs(m, k, n, dtype, pad=(0, 8, 3, 1)[i])
        pad = (0, 8, 5, 1)[i]
        gate, up, dy = (randn(g, m, n + pad, dtype=dtype)[:, :n] for _ in range(3))
        got = bl.convrot_gated_linear_backward(x, wg, wu, gate, up, dy, act, biases=True)
        want, bound = ref.gated_gradient(x, wg, wu, gate, up, dy, act)
        assert set(got) == set(want)
        for name in want:
            close(got[name], want[name], bound[name], f"{name}, act {act}")
        again = bl.convrot_gated_linear_backward(x, wg, wu, gate, up, dy, act, weights=False)
        assert torch.equal(again["dx"], got["dx"]) and again["dw_gate"] is None and again["db_up"] is None
        again = bl.convrot_gated_linear_backward(x, wg, wu, gate, up, dy, act, input=False, biases=True)
        assert again["dx"] is None and all(torch.equal(again[name], got[name]) for name in ("dw_gate", "dw_up", "db_gate", "db_up"))


def test_gated_linear_gradient_against_differences():
    """The gradients of sum(y dy), as central differences of the forward formula in 64 bits say."""
    m, k, n, dtype = 9, 24, 40, BF16
    g, x, wg, wu, bg, bu = gated_inputs(m, k, n, dtype)
    dy = randn(g, m, n, dtype=dtype)
    for act in ACTS:
        _, gate, up = bl.convrot_gated_linear(x, wg, wu, bg, bu, act, keep=True)
        got = bl.convrot_gated_linear_backward(x, wg, wu, gate, up, dy, act, biases=True)
        wide = [t.double() for t in (x, wg, wu, bg, bu)]

        def loss(parts):
            x, wg, wu, bg, bu = parts
            return float(((ref.act(x @ wg.t() + bg, act) * (x @ wu.t() + bu)) * dy.double()).sum())

        for i, name in enumerate(("dx", "dw_gate", "dw_up", "db_gate", "db_up")):
            for at in torch.randint(0, wide[i].numel(), (6,), generator=g, device="cuda").tolist():
                step = torch.zeros(wide[i].numel(), dtype=torch.float64, device="cuda")
                step[at] = 1e-4
                step = step.view_as(wide[i])
                up_, down = ([t + s * step if j == i else t for j, t in enumerate(wide)] for s in (1, -1))
                want = (loss(up_) - loss(down)) / 2e-4
                # gate, up, dg, du and the result are rounded to 8 bits: five roundings of 2^-8 on terms of a sum of up to 80
                assert abs(float(got[name].reshape(-1)[at]) - want) <= 0.1 * max(1.0, abs(want)), (name, act, at)


def test_gated_linear_extremes():
    """Large values keep their limits: a gate far below 0 gives 0, far above 0 itself; NaN and infinity stay in their rows."""
    x = torch.zeros(300, 64, dtype=BF16, device="cuda")
    x[0, 0], x[1, 0], x[2, 0] = 1e4, -1e4, 1e20
    x[130, 0], x[299, 1] = float("nan"), float("inf")
    w = torch.eye(64, dtype=BF16, device="cuda")
    one = torch.ones(64, device="cuda")
    zero = torch.zeros(64, 64, dtype=BF16, device="cuda")
    for act in ACTS:
        for rows in (300, 4):
            y, gate, up = bl.convrot_gated_linear(x[:rows], w, zero, None, one, act, keep=True)
            assert float(y[0, 0]) == float(x[0, 0]) and float(y[2, 0]) == float(x[2, 0])
            assert float(y[1, 0]) == (float(x[1, 0]) if act == bl.ACT_NONE else 0.0)
            clean = [r for r in range(rows) if r not in (130, 299)]
            assert torch.isfinite(y[clean]).all()
            if rows == 300:
                assert torch.isnan(y[130, 0]) and not torch.isfinite(y[299]).all()
            dy = torch.ones(4, 64, dtype=BF16, device="cuda")
            grads = bl.convrot_gated_linear_backward(x[:4], w, w, gate[:4], up[:4], dy, act, biases=True)
            # (dw_up's first value is 1e20 times 1e20, past every 32-bit float)
            assert all(torch.isfinite(t).all() for name, t in grads.items() if name != "dw_up")
            assert torch.isfinite(grads["dw_up"].flatten()[1:]).all() and float(grads["dw_up"][0, 0]) == float("inf")


@TYPES
def test_gated_linear_without_rows(dtype):
    for m, n in ((0, 8), (3, 0), (0, 0)):
        x, w = torch.ones(m, 16, dtype=dtype, device="cuda"), torch.ones(n, 16, dtype=dtype, device="cuda")
        y, gate, up = bl.convrot_gated_linear(x, w, w, keep=True)
        assert y.shape == gate.shape == up.shape == (m, n)
        got = bl.convrot_gated_linear_backward(x, w, w, gate, up, y, biases=True)
        assert got["dx"].shape == (m, 16) and got["dw_up"].shape == (n, 16) and got["db_gate"].shape == (n,)
        assert all(not t.any() for t in got.values())


# ---------------------------------------------------------------- attention

# batch, queries, keys, heads, key heads, head_dim
SHAPES = [(1, 1, 1, 1, 1, 8), (2, 1, 5, 4, 2, 64), (1, 3, 128, 2, 1, 128), (2, 77, 77, 3, 3, 40), (1, 128, 129, 2, 2, 72), (3, 129, 127, 4, 1, 64),
          (1, 256, 300, 2, 2, 128), (2, 257, 1, 2, 1, 96), (1, 300, 512, 3, 3, 80), (2, 130, 640, 2, 2, 100), (1, 33, 260, 5, 5, 33), (1, 515, 200, 6, 2, 1),
          (5, 1, 1000, 8, 8, 128), (1, 1, 4096, 8, 1, 64), (2, 5, 257, 16, 2, 128), (70, 40, 30, 9, 3, 16),
          (1, 1, 70001, 2, 1, 128), (1, 4, 30000, 4, 1, 60), (3, 16, 777, 2, 2, 64), (2, 17, 777, 2, 2, 64)]
MASKS = ["none", "padded", "scattered"]


def attention_inputs(b, tq, tk, hq, hk, d, dtype, mask="none", seed=0):
    g = gen(seed + b + 3 * tq + 7 * tk + hq * 11 + d)
    q = randn(g, b, tq, hq, d, dtype=dtype, std=1.5)
    kv = randn(g, b, tk, 2, hk, d, dtype=dtype)
    there = None
    if mask == "padded":
        there = torch.arange(tk, device="cuda") < torch.randint(0, tk + 1, (b, 1), generator=g, device="cuda")
    elif mask == "scattered":
        there = torch.rand(b, tk, generator=g, device="cuda") < torch.rand(b, 1, generator=g, device="cuda")
    if there is not None:
        there[0] = False  # nothing is there
        kv[~there] = float("nan")
    return g, q, kv[:, :, 0], kv[:, :, 1], there


@TYPES
@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("b,tq,tk,hq,hk,d", SHAPES)
def test_attention(b, tq, tk, hq, hk, d, mask, dtype):
    _, q, k, v, there = attention_inputs(b, tq, tk, hq, hk, d, dtype, mask)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = bl.convrot_attention(q, k, v, there, dev_status=status)
    want = ref.Attention(q, k, v, there)
    assert int(status) == 0
    close(out, want.out, want.out_bound, "out")
    empty = want.lse == -float("inf")
    assert torch.equal(lse == -float("inf"), empty) and not out.transpose(1, 2)[empty].any()
    close(lse[~empty], want.lse[~empty], want.lse_bound[~empty], "lse")
    again, lse2 = bl.convrot_attention(q, k, v, there)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@TYPES
@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("b,tq,tk,hq,hk,d", SHAPES)
def test_attention_gradient(b, tq, tk, hq, hk, d, mask, dtype):
    g, q, k, v, there = attention_inputs(b, tq, tk, hq, hk, d, dtype, mask)
    dout = randn(g, b, tq, hq, d, dtype=dtype)
    out, lse = bl.convrot_attention(q, k, v, there)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = bl.convrot_attention_backward(q, k, v, out, lse, dout, there, dev_status=status)
    want, bound = ref.Attention(q, k, v, there).gradient(dout)
    assert int(status) == 0
    for name in ("dq", "dk", "dv"):
        close(got[name], want[name], bound[name], name)
    if there is not None:
        assert not got["dk"][~there].any() and not got["dv"][~there].any()
    again = bl.convrot_attention_backward(q, k, v, out, lse, dout, there)
    assert all(torch.equal(got[name], again[name]) for name in got)


@TYPES
@pytest.mark.parametrize("b,tq,tk,hq,hk,d,mask", [
    (2, 2600, 20, 24, 2, 72, "padded"), (40, 130, 128, 20, 20, 64, "scattered"), (40, 130, 100, 20, 20, 128, "scattered"), (3, 2100, 90, 20, 4, 64, "padded"),
    (60, 130, 300, 10, 10, 64, "padded"), (2, 2600, 300, 24, 2, 128, "none"), (2, 2600, 400, 24, 8, 64, "none"), (1, 9000, 700, 8, 1, 128, "scattered"),
    (30, 500, 100, 20, 20, 128, "scattered"), (2, 2600, 90, 24, 2, 80, "none"),
    (5, 4000, 130, 1, 1, 100, "none")])
def test_attention_many_items(b, tq, tk, hq, hk, d, mask, dtype):
    """So many items that each ring and each barrier of a CTA comes round several times."""
    g, q, k, v, there = attention_inputs(b, tq, tk, hq, hk, d, dtype, mask)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = bl.convrot_attention(q, k, v, there, dev_status=status)
    dout = randn(g, b, tq, hq, d, dtype=dtype)
    got = bl.convrot_attention_backward(q, k, v, out, lse, dout, there, dev_status=status)
    assert int(status) == 0
    for i in range(b):  # (sample by sample: the plain form's matrices are large)
        at = slice(i, i + 1)
        want = ref.Attention(q[at], k[at], v[at], None if there is None else there[at])
        close(out[at], want.out, want.out_bound, "out")
        grads, bound = want.gradient(dout[at])
        for name in grads:
            close(got[name][at], grads[name], bound[name], name)


@TYPES
@pytest.mark.parametrize("b,tq,tk,hq,hk,d,mask", [
    (1, 64, 4096, 16, 16, 64, "none"), (2, 200, 1500, 4, 2, 128, "scattered"), (3, 40, 900, 2, 1, 50, "padded"), (1, 300, 257, 1, 1, 33, "none"),
    (1, 17, 20000, 1, 1, 128, "padded"), (1, 257, 513, 30, 3, 72, "none"), (5, 100, 700, 3, 3, 1, "scattered")])
def test_attention_keys_shared_out(b, tq, tk, hq, hk, d, mask, dtype):
    """Few queries and long keys: the keys are shared out, samples with fewer of them than shares among them."""
    g, q, k, v, there = attention_inputs(b, tq, tk, hq, hk, d, dtype, mask)
    if there is not None:
        there[-1, 100:] = False
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = bl.convrot_attention(q, k, v, there, dev_status=status)
    dout = randn(g, b, tq, hq, d, dtype=dtype)
    got = bl.convrot_attention_backward(q, k, v, out, lse, dout, there, dev_status=status)
    assert int(status) == 0
    want = ref.Attention(q, k, v, there)
    close(out, want.out, want.out_bound, "out")
    empty = want.lse == -float("inf")
    assert torch.equal(lse == -float("inf"), empty)
    close(lse[~empty], want.lse[~empty], want.lse_bound[~empty], "lse")
    grads, bound = want.gradient(dout)
    for name in grads:
        close(got[name], grads[name], bound[name], name)


def test_attention_gradient_against_differences():
    b, tq, tk, hq, hk, d = 2, 5, 9, 4, 2, 16
    g, q, k, v, there = attention_inputs(b, tq, tk, hq, hk, d, BF16, "padded", seed=3)
    k, v = (t.nan_to_num(0.0) for t in (k, v))
    dout = randn(g, b, tq, hq, d, dtype=BF16)
    out, lse = bl.convrot_attention(q, k, v, there, scale=0.4)
    got = bl.convrot_attention_backward(q, k, v, out, lse, dout, there, scale=0.4)
    wide = [t.double() for t in (q, k, v)]

    def loss(parts):
        return float((ref.Attention(*parts, there, scale=0.4).out * dout.double()).sum())

    for i, name in enumerate(("dq", "dk", "dv")):
        for at in torch.randint(0, wide[i].numel(), (8,), generator=g, device="cuda").tolist():
            step = torch.zeros(wide[i].numel(), dtype=torch.float64, device="cuda")
            step[at] = 1e-4
            step = step.view_as(wide[i])
            up, down = ([t + s * step if j == i else t for j, t in enumerate(wide)] for s in (1, -1))
            want = (loss(up) - loss(down)) / 2e-4
            # out, P, dS and the result are rounded to 8 bits: four roundings of 2^-8 on terms that are a few units each
            assert abs(float(got[name].reshape(-1)[at]) - want) <= 0.1 * max(1.0, abs(want)), (name, at)


@TYPES
def test_attention_strides(dtype):
    """Heads before tokens, shared (expanded) keys, broadcast samples, heads that start anywhere; an output inside another tensor."""
    b, tq, tk, hq, hk, d = 2, 140, 150, 4, 2, 64
    g = gen(5)
    q = randn(g, b, hq, tq, d, dtype=dtype).transpose(1, 2)
    k, v = (randn(g, 1, tk, 1, d, dtype=dtype).expand(b, tk, hk, d) for _ in range(2))
    odd = randn(g, b, tk, hk, d + 1, dtype=dtype)
    dout = randn(g, b, hq, tq, d + 3, dtype=dtype).transpose(1, 2)[..., 3:]
    big = torch.full((b, tq + 1, hq + 1, d + 5), -3.0, dtype=dtype, device="cuda")
    for kk, vv in ((k, v), (odd[..., 1:], odd[..., :d])):
        for out in (None, big[:, :tq, 1:, 5:], big[:, :tq, 1:, 4:4 + d]):
            big.fill_(-3.0)
            got, lse = bl.convrot_attention(q, kk, vv, out=out)
            want = ref.Attention(q, kk, vv)
            close(got, want.out, want.out_bound)
            if out is not None:
                out.fill_(-3.0)
                assert torch.all(big == -3.0)
        got, lse = bl.convrot_attention(q, kk, vv)
        grads = bl.convrot_attention_backward(q, kk, vv, got, lse, dout)
        want, bound = want.gradient(dout)
        for name in want:
            close(grads[name], want[name], bound[name], name)


@TYPES
def test_attention_large_scores(dtype):
    """One key far above all others, scores far below 0, and maxima that grow along the keys by more than the reference may lag."""
    g = gen(11)
    q, k, v = randn(g, 1, 200, 2, 64, dtype=dtype), randn(g, 1, 700, 2, 64, dtype=dtype), randn(g, 1, 700, 2, 64, dtype=dtype)
    grow = torch.linspace(0.1, 12.0, 700, device="cuda")[None, :, None, None]
    one = torch.where(torch.arange(700, device="cuda") == 333, 20.0, 0.5)[None, :, None, None]
    for kk in ((k * grow).to(dtype), (k * grow.flip(1)).to(dtype), (k * one).to(dtype), (k * 0).to(dtype), (-q[:, :1].abs() * grow).to(dtype)):
        out, lse = bl.convrot_attention(q, kk, v)
        want = ref.Attention(q, kk, v)
        close(out, want.out, want.out_bound, "out")
        close(lse, want.lse, want.lse_bound, "lse")


def test_attention_gradient_of_small_float16():
    """dout a millionth of what float16 resolves well: the gradients that float16 can hold are there."""
    g, q, k, v, _ = attention_inputs(1, 200, 300, 4, 2, 64, F16)
    v = v * 100
    for size in (1e-5, 1e-3, 1.0, 1000.0):
        dout = randn(g, 1, 200, 4, 64, dtype=F16, std=size)
        out, lse = bl.convrot_attention(q, k, v)
        got = bl.convrot_attention_backward(q, k, v, out, lse, dout)
        want, bound = ref.Attention(q, k, v).gradient(dout)
        for name in got:
            fits = want[name].abs() < 60000
            close(got[name][fits], want[name][fits], bound[name][fits], f"{name} at {size}")


@TYPES
def test_attention_without_queries_or_keys(dtype):
    for b, tq, tk, hq, hk in ((2, 0, 5, 4, 2), (2, 5, 0, 4, 2), (0, 3, 3, 2, 1), (1, 3, 4, 0, 2)):
        q, k = torch.ones(b, tq, hq, 32, dtype=dtype, device="cuda"), torch.ones(b, tk, hk, 32, dtype=dtype, device="cuda")
        out, lse = bl.convrot_attention(q, k, k)
        assert out.shape == q.shape and not out.any() and torch.all(lse == -float("inf")) and lse.shape == (b, hq, tq)
        got = bl.convrot_attention_backward(q, k, k, out, lse, q)
        assert got["dq"].shape == q.shape and got["dk"].shape == got["dv"].shape == k.shape
        assert not any(t.any() for t in got.values())


def test_attention_of_no_elements_is_refused():
    q = torch.empty(1, 2, 1, 0, dtype=BF16, device="cuda")
    with pytest.raises(cr.ConvrotError):
        bl.convrot_attention(q, q, q)
    with pytest.raises(cr.ConvrotError):
        bl.convrot_attention_backward(q, q, q, q, torch.empty(1, 1, 2, device="cuda"), q)


def test_attention_mask_layouts():
    """uint8 masks with any value, one for all samples, and rows that start anywhere."""
    g, q, k, v, _ = attention_inputs(3, 20, 203, 2, 2, 32, BF16)
    whole = torch.rand(3, 206, generator=g, device="cuda") < 0.4
    for there in (whole[:, 1:204], whole[:1, :203].expand(3, 203), whole[:, 3:]):
        want = ref.Attention(q, k, v, there)
        byte = torch.where(there, 128, 0).to(torch.uint8) if there.stride(0) else there
        for mask in (there, byte):
            out, lse = bl.convrot_attention(q, k, v, mask)
            close(out, want.out, want.out_bound)
