"""GPU tests of calls at the edges of what include/convrot_block.h allows of attention to other states and of the gated
linear, through the C entry points where the Python binding has no such call. The arguments are test_more_block_abi.py's."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from int8_hadamard_rotated_convrot_gb300 import block as bl  # noqa: E402
from int8_hadamard_rotated_convrot_gb300 import convrot as cr  # noqa: E402

from . import more_reference as more  # noqa: E402
from . import test_more_block_abi as abi  # noqa: E402
from . import test_more_reference as plain  # noqa: E402

BF16, F16 = torch.bfloat16, torch.float16
TYPES = pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from int8_hadamard_rotated_convrot_gb300 import build

    build.build()
    return cr.load()


@TYPES
@pytest.mark.parametrize("tq,hq,hk,d", [(30, 4, 2, 64), (1, 4, 2, 64), (700, 2, 1, 128), (2000, 8, 1, 72)])
def test_a_mask_of_no_keys(lib, tq, hq, hk, d, dtype):
    """kv_tokens == 0 beside the address of a mask: nothing of it is read or waited for."""
    b = 3
    q = torch.randn(b, tq, hq, d, device="cuda").to(dtype)
    out, lse = torch.full_like(q, 7.0), torch.full((b, hq, tq), 7.0, device="cuda")
    mask, status = torch.ones(64, dtype=torch.uint8, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    strides = (tq * hq * d, hq * d, d)
    args = abi.attention_args(q=q.data_ptr(), k=0, v=0, mask=mask.data_ptr(), out=out.data_ptr(), lse=lse.data_ptr(), status=status.data_ptr(),
                              batch=b, tq=tq, tk=0, hq=hq, hk=hk, qs=strides, os=strides, d=d, dtype=bl.BF16 if dtype is BF16 else bl.F16)
    assert lib.convrot_attention_work_bytes(args) == 0
    assert lib.convrot_attention(args, None) == cr.OK
    torch.cuda.synchronize()
    assert int(status) == 0 and not out.any() and torch.all(lse == -float("inf"))


# queries, keys, heads, key heads, head_dim, mask: few rows, a cluster's and several; tiles that pass by, that stay, that are shared out; masks in place and gathered
FORMS = [(3, 300, 4, 2, 64, False), (3, 40000, 2, 1, 128, True), (90, 300, 2, 2, 64, False), (300, 100, 4, 4, 128, True), (1500, 100, 4, 1, 64, True),
         (60, 4096, 2, 2, 64, False), (60, 4096, 2, 2, 128, True), (300, 500, 2, 2, 72, True)]


def infinite_scores(tq, tk, hq, hk, d, masked, dtype, of_q, of_k):
    """Queries of -1, 0 and 1 in turn, times of_q, to keys that are all of_k."""
    g = torch.Generator(device="cuda").manual_seed(tq + tk)
    kind = (torch.arange(tq, device="cuda") % 3 - 1)[None, :, None, None]
    q = (kind * of_q).expand(2, tq, hq, d).to(dtype).contiguous()
    k = torch.full((2, tk, hk, d), of_k, device="cuda", dtype=dtype)
    v = torch.randn(2, tk, hk, d, generator=g, device="cuda").to(dtype)
    mask = torch.rand(2, tk, generator=g, device="cuda") < 0.7 if masked else None
    there = torch.ones(2, tk, dtype=torch.bool, device="cuda") if mask is None else mask
    mean = torch.stack([v[i, there[i]].double().mean(0) for i in range(2)]).repeat_interleave(hq // hk, 1)  # [2, hq, d]
    return q, k, v, mask, kind[0, :, 0, 0], there.sum(1).double(), mean


def check_infinite_scores(out, lse, kind, count, mean, dtype):
    assert torch.isnan(out[:, kind == 1]).all() and torch.isnan(lse[:, :, kind == 1]).all()
    assert not out[:, kind == -1].any() and torch.all(lse[:, :, kind == -1] == -float("inf"))
    # equal probabilities, exact but for the sums of up to 40000 terms in fp32 (each off by 2^-23 of the sum of their sizes at most,
    # and no more than 3000 after one another) and the rounding of results of up to 4
    assert (out[:, kind == 0].double() - mean[:, None]).abs().max() <= 4 * torch.finfo(dtype).eps / 2 + 3000 * 2.0**-23
    assert (lse[:, :, kind == 0].double() - count.log()[:, None, None]).abs().max() <= 2.0**-18


@TYPES
@pytest.mark.parametrize("tq,tk,hq,hk,d,masked", FORMS)
def test_scores_past_the_floats(lib, tq, tk, hq, hk, d, masked, dtype):
    """The largest scale takes scores of +-d past the floats: they are infinite, and those of 0 stay."""
    q, k, v, mask, *want = infinite_scores(tq, tk, hq, hk, d, masked, dtype, 1.0, 1.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = bl.convrot_attention(q, k, v, mask, scale=1.7e38, dev_status=status)
    assert int(status) == 0
    check_infinite_scores(out, lse, *want, dtype)


@pytest.mark.parametrize("tq,tk,hq,hk,d,masked", FORMS)
def test_infinite_scores_and_their_gradients(lib, tq, tk, hq, hk, d, masked):
    """Products of 2^126 a term are past the floats themselves. A query whose scores are all -infinity has no part in a gradient."""
    q, k, v, mask, kind, count, mean = infinite_scores(tq, tk, hq, hk, d, masked, BF16, 2.0**63, 2.0**63)
    out, lse = bl.convrot_attention(q, k, v, mask)
    check_infinite_scores(out, lse, kind, count, mean, BF16)
    q[:, kind == 1] = 0
    out, lse = bl.convrot_attention(q, k, v, mask)
    dout = torch.ones_like(out)
    got = bl.convrot_attention_backward(q, k, v, out, lse, dout, mask)
    assert not got["dq"][:, kind == -1].any() and not got["dk"].any()
    there = torch.ones(2, tk, dtype=torch.bool, device="cuda") if mask is None else mask
    want = torch.where(there, (hq // hk) * int((kind != -1).sum()) / count[:, None], 0.0)[:, :, None, None]
    # sums of equal terms, whose probability is one exponential of an lse that is off by up to 2^-18, rounded to 8 bits; fp32 sums as above
    assert ((got["dv"].double() - want).abs() <= want * (2 * 2.0**-8 + 2.0**-17 + 3000 * 2.0**-23)).all()


@TYPES
@pytest.mark.parametrize("tq,tk,hq,hk,d", [(5, 9, 4, 2, 16), (150, 77, 4, 2, 64), (20, 200, 4, 1, 128), (40, 130, 2, 2, 72)])
def test_attention_gradient_against_differences_where_it_is_large(lib, tq, tk, hq, hk, d, dtype):
    """The twelve largest elements of each gradient, keys in every sample, against central differences of the formula in 64 bits.
    A result may be off by the elementwise bound of its roundings, which is a few percent to a quarter of these elements, under half of them in any case."""
    g = torch.Generator(device="cuda").manual_seed(tq)
    q, k, v, dout = (torch.randn(2, t, h, d, generator=g, device="cuda") for t, h in ((tq, hq), (tk, hk), (tk, hk), (tq, hq)))
    q, k, v, dout = (t.to(dtype) for t in (1.5 * q, k, v, dout))
    mask = torch.rand(2, tk, generator=g, device="cuda") < 0.6
    mask[:, 0] = True
    out, lse = bl.convrot_attention(q, k, v, mask, scale=0.4)
    got = bl.convrot_attention_backward(q, k, v, out, lse, dout, mask, scale=0.4)
    grads, bound = more.Attention(q, k, v, mask, scale=0.4).gradient(dout)
    wide = [t.double() for t in (q, k, v)]
    for i, name in enumerate(("dq", "dk", "dv")):
        for at in grads[name].abs().flatten().topk(12).indices.tolist():
            step = torch.zeros_like(wide[i])
            step.view(-1)[at] = 1e-4
            up, down = (float((plain.attention(*(t + s * step if j == i else t for j, t in enumerate(wide)), mask, 0.4) * dout.double()).sum())
                        for s in (1, -1))
            want, off = (up - down) / 2e-4, float(bound[name].reshape(-1)[at])
            assert off < 0.5 * abs(want), (name, at)
            # (the differences' own error: 1e-8 of a third derivative, 1e-12 / 1e-4 of roundings)
            assert abs(float(got[name].reshape(-1)[at]) - want) <= off + 1e-5 * max(1.0, abs(want)), (name, at, want, off)


@TYPES
@pytest.mark.parametrize("m,k,n", [(129, 2560, 130), (200, 5120, 77), (256, 1500, 640), (255, 2056, 1), (130, 13824, 640), (192, 1289, 1920), (256, 5120, 3840)])
def test_gated_linear_of_long_narrow_layers(lib, m, k, n, dtype):
    """129 to 256 rows whose k is shared out over a cluster, each activation once."""
    for i, act in enumerate((bl.ACT_SILU, bl.ACT_GELU_ERF, bl.ACT_GELU_TANH, bl.ACT_NONE)):
        g = torch.Generator(device="cuda").manual_seed(m + i)
        pad = (0, 8, 3, 1)[i]
        x, wg, wu = (torch.randn(r, k + pad, generator=g, device="cuda") for r in (m, n, n))
        x, wg, wu = (t.to(dtype)[:, :k] for t in (x, wg * k**-0.5, wu * k**-0.5))
        bg, bu = (torch.randn(n, generator=g, device="cuda") if i % 2 else None for _ in range(2))
        big = torch.full((m + 1, n + 5), -3.0, dtype=dtype, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = bl.convrot_gated_linear(x, wg, wu, bg, bu, act, keep=True, out=big[:m, :n], dev_status=status)
        want, bound = more.gated(x, wg, wu, bg, bu, act)
        for name, a, b, c in zip(("y", "gate", "up"), got, want, bound):
            off = (a.double() - b).abs()
            assert (off <= c).all(), (name, act, float((off - c).max()))
        assert int(status) == 0 and torch.all(big[m] == -3.0) and torch.all(big[:, n:] == -3.0)
        assert torch.equal(bl.convrot_gated_linear(x, wg, wu, bg, bu, act), got[0])
