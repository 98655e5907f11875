"""The host side of the operators around the linears: refusals, empty problems
and the rotary frequencies. No call here reaches a kernel."""

import math
import os
import struct
import subprocess
import sys

import pytest
import torch

from int8_hadamard_rotated_convrot_gb300 import block as bl
from int8_hadamard_rotated_convrot_gb300 import build as cbuild
from int8_hadamard_rotated_convrot_gb300 import convrot as cr

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # aligned and never dereferenced on these paths

# the argument structs of include/convrot_block.h, field by field
LINEAR = struct.Struct("@8P3q5qq4i")
NORM = struct.Struct("@13P3q9q2f4i")
NORM_BACKWARD = struct.Struct("@20Pq3q8q2f4i")
ROTARY = struct.Struct("@8P4q12q3q6i")


@pytest.fixture(scope="module")
def lib():
    cbuild.build()
    return cr.load()


def linear_args(**kw):
    v = dict(x=FAKE, xs=FAKE, w=FAKE, ws=FAKE, bias=0, y=FAKE, work=FAKE, status=0, m=4, n=8, k=256, ldx=256, ldxs=4,
             ldw=256, ldws=2, ldy=8, work_bytes=1 << 30, x_dtype=bl.BF16, y_dtype=bl.BF16, act=0, reserved=0)
    assert set(kw) <= set(v)
    return LINEAR.pack(*(v | kw).values())


LINEAR_BAD = [
    (dict(m=-1), cr.ERR_INVALID_ARG), (dict(n=-1), cr.ERR_INVALID_ARG), (dict(m=1 << 31), cr.ERR_INVALID_ARG),
    (dict(k=0), cr.ERR_K_RANGE), (dict(k=cr.MAX_K + 1), cr.ERR_K_RANGE), (dict(w=0), cr.ERR_INVALID_ARG),
    (dict(w=FAKE + 8), cr.ERR_ALIGNMENT), (dict(ldw=255), cr.ERR_INVALID_ARG), (dict(ldw=264), cr.ERR_ALIGNMENT),
    (dict(ws=0), cr.ERR_INVALID_ARG), (dict(ldws=1), cr.ERR_INVALID_ARG), (dict(ws=FAKE + 2), cr.ERR_ALIGNMENT),
    (dict(y=0), cr.ERR_INVALID_ARG), (dict(ldy=7), cr.ERR_INVALID_ARG), (dict(y=FAKE + 1), cr.ERR_ALIGNMENT),
    (dict(y_dtype=3), cr.ERR_INVALID_ARG), (dict(act=3), cr.ERR_INVALID_ARG), (dict(act=-1), cr.ERR_INVALID_ARG),
    (dict(bias=FAKE + 2), cr.ERR_ALIGNMENT), (dict(status=FAKE + 2), cr.ERR_ALIGNMENT),
    (dict(reserved=1), cr.ERR_INVALID_ARG), (dict(x=0), cr.ERR_INVALID_ARG), (dict(ldx=255), cr.ERR_INVALID_ARG),
]


@pytest.mark.parametrize("kw,status", LINEAR_BAD, ids=[str(k) for k, _ in LINEAR_BAD])
def test_linears_refuse(lib, kw, status):
    assert lib.convrot_fp8_linear(linear_args(**kw), None) == status
    assert lib.convrot_fp8_pack_linear(linear_args(**kw), None) == status


def test_linear_refuses_its_own_operands(lib):
    assert lib.convrot_fp8_linear(None, None) == cr.ERR_INVALID_ARG
    assert lib.convrot_fp8_pack_linear(None, None) == cr.ERR_INVALID_ARG
    assert lib.convrot_fp8_linear(linear_args(x=FAKE + 8), None) == cr.ERR_ALIGNMENT
    assert lib.convrot_fp8_linear(linear_args(ldx=264), None) == cr.ERR_ALIGNMENT
    assert lib.convrot_fp8_linear(linear_args(xs=0), None) == cr.ERR_INVALID_ARG
    assert lib.convrot_fp8_linear(linear_args(ldxs=3), None) == cr.ERR_INVALID_ARG
    assert lib.convrot_fp8_pack_linear(linear_args(x_dtype=-1), None) == cr.ERR_INVALID_ARG
    assert lib.convrot_fp8_pack_linear(linear_args(x=FAKE + 1), None) == cr.ERR_ALIGNMENT


def test_pack_linear_refuses_a_short_workspace(lib):
    m, n, k = 4096, 512, 256
    need = bl.fp8_pack_linear_work_bytes(m, n, k)
    assert need > m * k
    big = dict(m=m, n=n, k=k, ldy=n, ldws=2)
    assert lib.convrot_fp8_pack_linear(linear_args(**big, work_bytes=need - 1), None) == cr.ERR_INVALID_ARG
    assert lib.convrot_fp8_pack_linear(linear_args(**big, work=0), None) == cr.ERR_INVALID_ARG
    assert lib.convrot_fp8_pack_linear(linear_args(**big, work=FAKE + 64), None) == cr.ERR_ALIGNMENT
    for bad in ((0, 1, 1), (1, 0, 1), (1, 1, 0), (1, 1, cr.MAX_K + 1)):
        assert bl.fp8_pack_linear_work_bytes(*bad) == 0


def test_empty_linears_launch_nothing(lib):
    for kw in (dict(m=0, x=0, xs=0, y=0), dict(n=0, w=0, ws=0, y=0)):
        assert lib.convrot_fp8_linear(linear_args(**kw), None) == cr.OK
        assert lib.convrot_fp8_pack_linear(linear_args(**kw), None) == cr.OK


@pytest.mark.parametrize("kw,status", [
    (dict(k=0), cr.ERR_K_RANGE), (dict(m=-1), cr.ERR_INVALID_ARG), (dict(dtype=3), cr.ERR_INVALID_ARG),
    (dict(x=None), cr.ERR_INVALID_ARG), (dict(x=FAKE + 1), cr.ERR_ALIGNMENT), (dict(ldx=255), cr.ERR_INVALID_ARG),
    (dict(q=None), cr.ERR_INVALID_ARG), (dict(q=FAKE + 8), cr.ERR_ALIGNMENT), (dict(ldq=250), cr.ERR_INVALID_ARG),
    (dict(ldq=264), cr.ERR_ALIGNMENT), (dict(s=None), cr.ERR_INVALID_ARG), (dict(lds=1), cr.ERR_INVALID_ARG)], ids=str)
def test_quantizers_refuse(lib, kw, status):
    v = dict(x=FAKE, dtype=bl.BF16, m=4, k=256, ldx=256, q=FAKE, ldq=256, s=FAKE, lds=4) | kw
    assert lib.convrot_fp8_pack_activations(*v.values(), None) == status
    assert lib.convrot_fp8_quantize_weights(*v.values(), None) == status


def test_empty_packs_launch_nothing(lib):
    assert lib.convrot_fp8_pack_activations(None, bl.F32, 0, 256, 256, None, 256, None, 0, None) == cr.OK
    assert lib.convrot_fp8_quantize_weights(None, bl.F32, 0, 256, 256, None, 256, None, 2, None) == cr.OK


def norm_args(**kw):
    v = dict(x=FAKE, y=FAKE, gate=0, scale=0, shift=0, post_w=0, post_b=0, pre_w=0, pre_b=0, h=FAKE, n=FAKE, q=0, qs=0,
             m=4, d=64, rows=4, ldx=64, ldy=64, ldgate=64, ldscale=64, ldshift=64, ldh=64, ldn=64, ldq=64, ldqs=4,
             res_scale=1.0, eps=1e-6, post=0, pre=1, dtype=bl.BF16, p=bl.F32)
    assert set(kw) <= set(v)
    return NORM.pack(*(v | kw).values())


NORM_BAD = [
    (dict(m=-1), cr.ERR_INVALID_ARG), (dict(d=0), cr.ERR_INVALID_ARG), (dict(d=bl.NORM_MAX_D + 1), cr.ERR_UNSUPPORTED),
    (dict(rows=0), cr.ERR_INVALID_ARG), (dict(dtype=3), cr.ERR_INVALID_ARG), (dict(p=bl.F16), cr.ERR_INVALID_ARG),
    (dict(post=3), cr.ERR_INVALID_ARG), (dict(pre=-1), cr.ERR_INVALID_ARG), (dict(x=0), cr.ERR_INVALID_ARG),
    (dict(x=FAKE + 1), cr.ERR_ALIGNMENT), (dict(ldx=63), cr.ERR_INVALID_ARG), (dict(ldy=63), cr.ERR_INVALID_ARG),
    (dict(gate=FAKE + 2), cr.ERR_ALIGNMENT), (dict(gate=FAKE, ldgate=8), cr.ERR_INVALID_ARG),
    (dict(scale=FAKE, ldscale=8), cr.ERR_INVALID_ARG), (dict(shift=FAKE, ldshift=8), cr.ERR_INVALID_ARG),
    (dict(pre_w=FAKE + 2), cr.ERR_ALIGNMENT), (dict(ldh=63), cr.ERR_INVALID_ARG), (dict(ldn=63), cr.ERR_INVALID_ARG),
    (dict(h=FAKE, x=FAKE, ldh=128), cr.ERR_INVALID_ARG), (dict(q=FAKE), cr.ERR_INVALID_ARG),
    (dict(eps=-1e-6), cr.ERR_INVALID_ARG), (dict(eps=float("nan")), cr.ERR_INVALID_ARG),
    (dict(q=FAKE + 8, qs=FAKE), cr.ERR_ALIGNMENT), (dict(q=FAKE, qs=FAKE, ldqs=3), cr.ERR_INVALID_ARG),
]


@pytest.mark.parametrize("kw,status", NORM_BAD, ids=[str(k) for k, _ in NORM_BAD])
def test_gated_norm_refuses(lib, kw, status):
    assert lib.convrot_gated_norm(norm_args(**kw), None) == status


def test_empty_norms_launch_nothing(lib):
    assert lib.convrot_gated_norm(None, None) == cr.ERR_INVALID_ARG
    assert lib.convrot_gated_norm(norm_args(m=0, x=0, y=0, h=0, n=0), None) == cr.OK
    assert lib.convrot_gated_norm(norm_args(h=0, n=0), None) == cr.OK  # nothing wanted


def grad_args(**kw):
    v = dict(h=FAKE, y=FAKE, dh=FAKE, dn=FAKE, gate=0, scale=0, post_w=0, post_b=0, pre_w=0, pre_b=0, dx=FAKE, dy=FAKE,
             dgate=0, dscale=0, dshift=0, dpost_w=0, dpost_b=0, dpre_w=0, dpre_b=0, work=FAKE, work_bytes=1 << 30,
             m=4, d=64, rows=4, ldh=64, ldy=64, lddh=64, lddn=64, ldgate=64, ldscale=64, lddx=64, lddy=64,
             res_scale=1.0, eps=1e-6, post=0, pre=1, dtype=bl.BF16, p=bl.F32)
    assert set(kw) <= set(v)
    return NORM_BACKWARD.pack(*(v | kw).values())


GRAD_BAD = [
    (dict(m=-1), cr.ERR_INVALID_ARG), (dict(d=bl.NORM_MAX_D + 1), cr.ERR_UNSUPPORTED), (dict(h=0), cr.ERR_INVALID_ARG),
    (dict(lddn=63), cr.ERR_INVALID_ARG), (dict(dh=FAKE + 1), cr.ERR_ALIGNMENT), (dict(lddx=1), cr.ERR_INVALID_ARG),
    (dict(y=0), cr.ERR_INVALID_ARG), (dict(y=0, dy=0, dgate=FAKE), cr.ERR_INVALID_ARG),
    (dict(dgate=FAKE + 2), cr.ERR_ALIGNMENT), (dict(work=0), cr.ERR_INVALID_ARG), (dict(work_bytes=0), cr.ERR_INVALID_ARG),
    (dict(work=FAKE + 16), cr.ERR_ALIGNMENT), (dict(post=-1), cr.ERR_INVALID_ARG),
]


@pytest.mark.parametrize("kw,status", GRAD_BAD, ids=[str(k) for k, _ in GRAD_BAD])
def test_gated_norm_backward_refuses(lib, kw, status):
    assert lib.convrot_gated_norm_backward(grad_args(**kw), None) == status


def test_empty_norm_gradient_launches_nothing(lib):
    assert lib.convrot_gated_norm_backward(None, None) == cr.ERR_INVALID_ARG
    assert lib.convrot_gated_norm_backward(grad_args(m=0, h=0, y=0, dh=0, dn=0, dx=0, dy=0, work=0), None) == cr.OK
    assert lib.convrot_gated_norm_backward_work_bytes(0, 64, 1) == 0
    assert lib.convrot_gated_norm_backward_work_bytes(4, 64, 0) == 0


def rotary_args(**kw):
    v = dict(q=FAKE, k=FAKE, oq=FAKE, ok=FAKE, cos=FAKE, sin=FAKE, positions=0, status=0, batch=2, tokens=3, qh=4, kh=2,
             qs=(1536, 512, 128), ks=(768, 256, 128), oqs=(1536, 512, 128), oks=(768, 256, 128), rows=3, ldt=64,
             pos_stride=3, d=128, r=128, layout=0, inverse=0, dtype=bl.BF16, bits=64)
    assert set(kw) <= set(v)
    flat = []
    for x in (v | kw).values():
        flat += x if isinstance(x, tuple) else [x]
    return ROTARY.pack(*flat)


ROTARY_BAD = [
    (dict(batch=-1), cr.ERR_INVALID_ARG), (dict(qh=-1), cr.ERR_INVALID_ARG), (dict(r=0), cr.ERR_INVALID_ARG),
    (dict(r=7), cr.ERR_INVALID_ARG), (dict(r=130), cr.ERR_INVALID_ARG), (dict(layout=2), cr.ERR_INVALID_ARG),
    (dict(dtype=9), cr.ERR_INVALID_ARG), (dict(d=bl.ROTARY_MAX_D + 2), cr.ERR_UNSUPPORTED), (dict(ldt=63), cr.ERR_INVALID_ARG),
    (dict(cos=0), cr.ERR_INVALID_ARG), (dict(sin=FAKE + 2), cr.ERR_ALIGNMENT), (dict(q=FAKE + 1), cr.ERR_ALIGNMENT),
    (dict(oq=0), cr.ERR_INVALID_ARG), (dict(ok=0), cr.ERR_INVALID_ARG), (dict(qs=(1536, -512, 128)), cr.ERR_INVALID_ARG),
    (dict(rows=2), cr.ERR_INVALID_ARG), (dict(positions=FAKE, bits=16), cr.ERR_INVALID_ARG),
    (dict(positions=FAKE + 4), cr.ERR_ALIGNMENT), (dict(positions=FAKE, rows=0), cr.ERR_INVALID_ARG),
    (dict(positions=FAKE, pos_stride=-1), cr.ERR_INVALID_ARG), (dict(status=FAKE + 1), cr.ERR_ALIGNMENT),
    (dict(batch=1 << 20, tokens=1 << 20), cr.ERR_INVALID_ARG),
]


@pytest.mark.parametrize("kw,status", ROTARY_BAD, ids=[str(k) for k, _ in ROTARY_BAD])
def test_rotary_refuses(lib, kw, status):
    assert lib.convrot_rotary(rotary_args(**kw), None) == status


def test_empty_rotary_launches_nothing(lib):
    assert lib.convrot_rotary(None, None) == cr.ERR_INVALID_ARG
    for kw in (dict(batch=0), dict(tokens=0), dict(q=0, k=0), dict(qh=0, kh=0)):
        assert lib.convrot_rotary(rotary_args(**kw), None) == cr.OK


def test_rotary_table_refuses(lib):
    call = lambda pos=None, rows=4, axes=1, f=FAKE, ax=None, pairs=8, c=FAKE, s=FAKE, ldt=8: lib.convrot_rotary_table(
        pos, rows, axes, f, ax, pairs, 1.0, c, s, ldt, None)
    assert call(rows=-1) == cr.ERR_INVALID_ARG
    assert call(axes=2) == cr.ERR_INVALID_ARG  # several axes need positions
    assert call(f=None) == cr.ERR_INVALID_ARG
    assert call(f=FAKE + 4) == cr.ERR_ALIGNMENT
    assert call(ldt=7) == cr.ERR_INVALID_ARG
    assert call(c=None) == cr.ERR_INVALID_ARG
    assert call(pairs=0) == cr.ERR_INVALID_ARG
    assert call(rows=0, c=None, s=None) == cr.OK


def test_binding_refuses_tensors_the_c_side_cannot_check(lib):
    x = torch.zeros(4, 64)
    with pytest.raises(TypeError):
        bl.convrot_gated_norm(x)  # not on the GPU
    with pytest.raises(TypeError):
        bl.convrot_fp8_pack_activations(x.double())
    with pytest.raises(TypeError):
        bl.convrot_rotary(torch.zeros(2, 3, 8), None, x, x)
    with pytest.raises(TypeError):
        bl.convrot_rotary_table(torch.zeros(4), [1.0])


# calls with tensors that have no memory of their own, each in a process: "plain" ones, and the slices that vmap hands out
WITHOUT_MEMORY = """
import sys, torch
from torch._subclasses import FakeTensorMode
from int8_hadamard_rotated_convrot_gb300 import block as bl
name, batched = sys.argv[1], sys.argv[2] == "vmap"
with FakeTensorMode():
    like = dict(device="cuda", dtype=torch.bfloat16)
    x, vec, table = torch.empty(4, 64, **like), torch.empty(64, **like), torch.empty(4, 8, device="cuda")
    w = bl.Fp8Weights(bl.fp8_codes(16, 64), torch.empty(1, 1, device="cuda"))
    call = {
        "norm": lambda t: bl.convrot_gated_norm(t, pre_weight=vec)[1],
        "vector": lambda t: bl.convrot_gated_norm(x, pre_weight=t[0], out_n=x)[1],
        "norm pack": lambda t: bl.convrot_gated_norm_pack(t)[1].scale,
        "gradient": lambda t: bl.convrot_gated_norm_backward(t, None, t, t)["dx"],
        "pack": lambda t: bl.convrot_fp8_pack_activations(t).scale,
        "linear": lambda t: bl.convrot_fp8_pack_linear(t, w),
        "rotary": lambda t: bl.convrot_rotary(t.view(1, 4, 2, 32), None, table, table)[0],
    }[name]
    try:
        torch.vmap(call)(torch.empty(3, 4, 64, **like)) if batched else call(x)
    except Exception as e:
        print("raised", type(e).__name__)
"""


@pytest.mark.parametrize("how", ["plain", "vmap"])
@pytest.mark.parametrize("name", ["norm", "vector", "norm pack", "gradient", "pack", "linear", "rotary"])
def test_tensors_without_memory_raise(lib, name, how):
    r = subprocess.run([sys.executable, "-c", WITHOUT_MEMORY, name, how], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("raised"), r.stdout + r.stderr[-2000:]


def test_tensors_of_two_devices_are_refused(lib):
    from torch._subclasses import FakeTensorMode

    with FakeTensorMode():
        a, b = (dict(device=f"cuda:{i}") for i in (0, 1))
        x, y = torch.empty(4, 64, **a), torch.empty(4, 64, **b)
        vec, one, work = torch.empty(64, **b), torch.empty(1, dtype=torch.int32, **b), torch.empty(64, dtype=torch.uint8, **b)
        w = bl.Fp8Weights(bl.fp8_codes(16, 64, "cuda:0"), torch.empty(1, 1, **a))
        other = bl.Fp8Weights(w.q, torch.empty(1, 1, **b))
        packed = bl.empty_fp8_rows(4, 64, "cuda:1")
        q, table = torch.empty(1, 4, 2, 16, **a), torch.empty(4, 8, **a)
        calls = [lambda: bl.convrot_fp8_pack_activations(x, out=packed), lambda: bl.convrot_fp8_pack_linear(x, other),
                 lambda: bl.convrot_fp8_linear(packed, w), lambda: bl.convrot_fp8_pack_linear(x, w, out=torch.empty(4, 16, **b)),
                 lambda: bl.convrot_fp8_pack_linear(x, w, dev_status=one), lambda: bl.convrot_fp8_pack_linear(x, w, work=work),
                 lambda: bl.convrot_gated_norm(x, y), lambda: bl.convrot_gated_norm(x, pre_weight=vec),
                 lambda: bl.convrot_gated_norm(x, out_n=y), lambda: bl.convrot_gated_norm_pack(x, out=packed),
                 lambda: bl.convrot_gated_norm_backward(x, None, x, y), lambda: bl.convrot_gated_norm_backward(x, None, x, x, work=work),
                 lambda: bl.convrot_rotary(q, None, table, torch.empty(4, 8, **b)),
                 lambda: bl.convrot_rotary(q, None, table, table, torch.empty(4, dtype=torch.int64, **b))]
        for call in calls:
            with pytest.raises(ValueError, match="one device"):
                call()


def test_gate_and_post_norm_belong_to_a_branch(lib):
    from torch._subclasses import FakeTensorMode

    with FakeTensorMode():
        x, gate, vec = (torch.empty(*shape, device="cuda") for shape in ((4, 64), (1, 64), (64,)))
        for kw in (dict(gate=gate), dict(post_weight=vec), dict(post_bias=vec)):
            for call in (lambda: bl.convrot_gated_norm(x, **kw), lambda: bl.convrot_gated_norm_pack(x, **kw),
                         lambda: bl.convrot_gated_norm_backward(x, None, x, x, **kw)):
                with pytest.raises(ValueError, match="belong to a branch"):
                    call()


def test_rotary_frequencies():
    plain, one = bl.rotary_frequencies(8, 10000.0)
    assert one == 1.0 and plain == [10000.0 ** (-i / 8) for i in range(8)]
    linear, _ = bl.rotary_frequencies(8, 10000.0, scaling="linear", factor=4.0)
    assert linear == [f / 4 for f in plain]
    ntk, _ = bl.rotary_frequencies(8, 10000.0, scaling="ntk", factor=4.0)
    assert ntk[0] == 1.0 and math.isclose(ntk[-1], plain[-1] / 4, rel_tol=1e-12)
    yarn, m = bl.rotary_frequencies(64, 10000.0, scaling="yarn", factor=16.0, original_length=4096)
    plain, _ = bl.rotary_frequencies(64, 10000.0)
    assert m == pytest.approx(0.1 * math.log(16.0) + 1.0)
    turns = [4096 * f / (2 * math.pi) for f in plain]
    for f, g, n in zip(plain, yarn, turns):
        assert f / 16 * (1 - 1e-12) <= g <= f * (1 + 1e-12)
        if n > 40:
            assert g == f
        if n < 0.8:
            assert math.isclose(g, f / 16, rel_tol=1e-12)
    for bad in (dict(pairs=0), dict(pairs=4, factor=0.5), dict(pairs=4, scaling="yarn"), dict(pairs=4, scaling="other")):
        with pytest.raises(ValueError):
            bl.rotary_frequencies(**bad)


@pytest.mark.parametrize("pairs,base,length,factor", [
    (64, 10000.0, 4096, 16.0), (64, 10000.0, 131072, 8.0), (32, 10000.0, 1 << 20, 4.0), (48, 500000.0, 8192, 8.0), (8, 100.0, 100000, 2.0)])
def test_yarn_ramp_of_long_trained_lengths(pairs, base, length, factor):
    """Each pair's frequency from the definition: also where even the slowest pair turns more than beta_slow times."""
    got, _ = bl.rotary_frequencies(pairs, base, scaling="yarn", factor=factor, original_length=length)
    at = lambda turns: pairs * math.log(length / (2 * math.pi * turns), base)
    start, end = max(math.floor(at(32.0)), 0), math.ceil(at(1.0))
    for i, f in enumerate(got):
        plain = base ** (-i / pairs)
        t = (i - start) / (end - start)
        t = 0.0 if t < 0 else 1.0 if t > 1 else t
        assert math.isclose(f, plain * ((1 - t) + t / factor), rel_tol=1e-9), i
        turns = length * plain / (2 * math.pi)
        if turns > 1.0 and i < end:
            assert f > plain / factor * (1 + 1e-9), f"pair {i} turns {turns:.2f} times and is divided by the whole factor"


@pytest.mark.parametrize("rows", [41, 1 << 31, (1 << 63) - 40, (1 << 63) - 1])
def test_samples_longer_than_the_call(lib, rows):
    """Any number of rows a sample: what is past the last row does not count."""
    assert lib.convrot_gated_norm_backward_work_bytes(40, 64, rows) == lib.convrot_gated_norm_backward_work_bytes(40, 64, 40) > 0
    for bad in (dict(gate=FAKE, ldgate=8), dict(scale=FAKE, ldscale=8)):
        assert lib.convrot_gated_norm_backward(grad_args(**bad, rows=rows), None) == cr.ERR_INVALID_ARG
        assert lib.convrot_gated_norm(norm_args(**bad, rows=rows), None) == cr.ERR_INVALID_ARG
    assert lib.convrot_gated_norm_backward(grad_args(rows=rows, work_bytes=0), None) == cr.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    dict(oq=FAKE + 4096, oqs=(1536, 512, 0)), dict(oq=FAKE + 4096, oqs=(1536, 0, 128)), dict(oq=FAKE + 4096, oqs=(0, 512, 128)),
    dict(oq=FAKE + 4096, oqs=(1536, 512, 127)), dict(oq=FAKE + 4096, oqs=(512, 512, 128)), dict(oq=FAKE + 4096, oqs=(600, 512, 128)),
    dict(ok=FAKE + 4096, oks=(768, 256, 64)), dict(oqs=(4096, 512, 128)), dict(oks=(768, 512, 128))], ids=str)
def test_rotary_refuses_outputs_over_one_another_or_their_input(lib, kw):
    assert lib.convrot_rotary(rotary_args(**kw), None) == cr.ERR_INVALID_ARG


@pytest.mark.parametrize("k", [48, 50])
def test_checkpoint_codes_of_another_type_are_refused(k):
    """Whether or not the rows have to be copied: 8-bit integers or e5m2 values are not e4m3 codes."""
    scale = torch.ones(1, 1)
    for dtype in (torch.float8_e5m2, torch.int8, torch.uint8, torch.float32):
        with pytest.raises(TypeError):
            bl.fp8_weights_from_codes(torch.zeros(16, k, dtype=dtype), scale)
    with pytest.raises(TypeError):
        bl.fp8_weights_from_codes(torch.zeros(16, dtype=torch.float8_e4m3fn), scale)
    codes = torch.arange(16 * k, dtype=torch.int64).remainder(120).to(torch.uint8).view(16, k).view(torch.float8_e4m3fn)
    w = bl.fp8_weights_from_codes(codes, scale.bfloat16())
    assert torch.equal(w.q.view(torch.uint8), codes.view(torch.uint8)) and w.q.stride(0) % 16 == 0 and w.scale.dtype == torch.float32
