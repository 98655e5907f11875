"""The host side of the gated linear and of attention: refusals, empty problems, workspaces and tensor memory.
No call here reaches a kernel."""

import itertools
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
GATED = struct.Struct("@10P3q6qq2i")
GATED_BACKWARD = struct.Struct("@13P3q9qq2i")
ATTENTION = struct.Struct("@8P5q12q2qf3i")
ATTENTION_BACKWARD = struct.Struct("@12P5q15q2qf3i")


@pytest.fixture(scope="module")
def lib():
    cbuild.build()
    return cr.load()


def pack(form, values):
    flat = []
    for x in values:
        flat += x if isinstance(x, tuple) else [x]
    return form.pack(*flat)


def gated_args(**kw):
    v = dict(x=FAKE, wg=FAKE, wu=FAKE, bg=0, bu=0, y=FAKE, gate=0, up=0, work=0, status=0, m=4, n=8, k=16, ldx=16, ldwg=16, ldwu=16, ldy=8,
             ldgate=8, ldup=8, work_bytes=0, dtype=bl.BF16, act=3)
    assert set(kw) <= set(v)
    return pack(GATED, (v | kw).values())


GATED_BAD = [
    (dict(m=-1), cr.ERR_INVALID_ARG), (dict(n=-1), cr.ERR_INVALID_ARG), (dict(k=0), cr.ERR_INVALID_ARG), (dict(m=(1 << 30) + 1), cr.ERR_INVALID_ARG),
    (dict(dtype=bl.F32), cr.ERR_UNSUPPORTED), (dict(dtype=3), cr.ERR_INVALID_ARG), (dict(act=4), cr.ERR_INVALID_ARG), (dict(act=-1), cr.ERR_INVALID_ARG),
    (dict(x=0), cr.ERR_INVALID_ARG), (dict(wg=0), cr.ERR_INVALID_ARG), (dict(wu=0), cr.ERR_INVALID_ARG), (dict(y=0), cr.ERR_INVALID_ARG),
    (dict(x=FAKE + 1), cr.ERR_ALIGNMENT), (dict(y=FAKE + 1), cr.ERR_ALIGNMENT), (dict(bg=FAKE + 2), cr.ERR_ALIGNMENT), (dict(ldx=15), cr.ERR_INVALID_ARG),
    (dict(ldwg=15), cr.ERR_INVALID_ARG), (dict(ldwu=15), cr.ERR_INVALID_ARG), (dict(ldy=7), cr.ERR_INVALID_ARG), (dict(gate=FAKE), cr.ERR_INVALID_ARG),
    (dict(up=FAKE), cr.ERR_INVALID_ARG), (dict(gate=FAKE, up=FAKE, ldup=7), cr.ERR_INVALID_ARG), (dict(status=FAKE + 2), cr.ERR_ALIGNMENT),
    (dict(x=FAKE + 2), cr.ERR_INVALID_ARG), (dict(ldwg=17), cr.ERR_INVALID_ARG),  # need a workspace
    (dict(x=FAKE + 2, work=FAKE + 16, work_bytes=1 << 20), cr.ERR_ALIGNMENT),
]


@pytest.mark.parametrize("kw,status", GATED_BAD, ids=[str(k) for k, _ in GATED_BAD])
def test_gated_linear_refuses(lib, kw, status):
    assert lib.convrot_gated_linear(gated_args(**kw), None) == status


def test_empty_gated_linear_launches_nothing(lib):
    assert lib.convrot_gated_linear(None, None) == cr.ERR_INVALID_ARG
    assert lib.convrot_gated_linear(gated_args(m=0, x=0, y=0), None) == cr.OK
    assert lib.convrot_gated_linear(gated_args(n=0, wg=0, wu=0, y=0), None) == cr.OK


def test_gated_workspaces(lib):
    assert lib.convrot_gated_linear_work_bytes(gated_args()) == 0
    assert lib.convrot_gated_linear_work_bytes(gated_args(x=FAKE + 2)) == 256
    assert lib.convrot_gated_linear_work_bytes(gated_args(x=FAKE + 2, ldwu=17)) == 512
    assert lib.convrot_gated_linear_work_bytes(gated_args(x=FAKE + 2, m=0)) == 0
    need = lib.convrot_gated_linear_work_bytes(gated_args(ldx=17, ldwg=17, ldwu=18))
    assert need == 3 * 256
    assert lib.convrot_gated_linear(gated_args(ldx=17, ldwg=17, ldwu=18, work=FAKE, work_bytes=need - 1), None) == cr.ERR_INVALID_ARG
    need = lib.convrot_gated_linear_backward_work_bytes(gated_grad_args())
    assert need >= 2 * 4 * 8 * 2
    assert lib.convrot_gated_linear_backward(gated_grad_args(work_bytes=need - 1), None) == cr.ERR_INVALID_ARG
    assert lib.convrot_gated_linear_backward(gated_grad_args(work=FAKE + 16), None) == cr.ERR_ALIGNMENT


def gated_grad_args(**kw):
    v = dict(x=FAKE, wg=FAKE, wu=FAKE, gate=FAKE, up=FAKE, dy=FAKE, dx=FAKE, dwg=FAKE, dwu=FAKE, dbg=0, dbu=0, work=FAKE, status=0, m=4, n=8, k=16,
             ldx=16, ldwg=16, ldwu=16, ldgate=8, ldup=8, lddy=8, lddx=16, lddwg=16, lddwu=16, work_bytes=1 << 30, dtype=bl.BF16, act=3)
    assert set(kw) <= set(v)
    return pack(GATED_BACKWARD, (v | kw).values())


GATED_GRAD_BAD = [
    (dict(m=-1), cr.ERR_INVALID_ARG), (dict(k=0), cr.ERR_INVALID_ARG), (dict(dtype=bl.F32), cr.ERR_UNSUPPORTED), (dict(act=4), cr.ERR_INVALID_ARG),
    (dict(dwg=0), cr.ERR_INVALID_ARG), (dict(dbg=FAKE), cr.ERR_INVALID_ARG), (dict(gate=0), cr.ERR_INVALID_ARG), (dict(up=0), cr.ERR_INVALID_ARG),
    (dict(dy=0), cr.ERR_INVALID_ARG), (dict(x=0), cr.ERR_INVALID_ARG), (dict(wg=0), cr.ERR_INVALID_ARG), (dict(ldgate=7), cr.ERR_INVALID_ARG),
    (dict(lddx=15), cr.ERR_INVALID_ARG), (dict(lddwu=15), cr.ERR_INVALID_ARG), (dict(dx=FAKE + 1), cr.ERR_ALIGNMENT), (dict(dbg=FAKE, dbu=FAKE + 2), cr.ERR_ALIGNMENT),
    (dict(work=0), cr.ERR_INVALID_ARG),
]


@pytest.mark.parametrize("kw,status", GATED_GRAD_BAD, ids=[str(k) for k, _ in GATED_GRAD_BAD])
def test_gated_linear_backward_refuses(lib, kw, status):
    assert lib.convrot_gated_linear_backward(gated_grad_args(**kw), None) == status


def test_gated_linear_backward_of_nothing(lib):
    assert lib.convrot_gated_linear_backward(None, None) == cr.ERR_INVALID_ARG
    assert lib.convrot_gated_linear_backward(gated_grad_args(dx=0, dwg=0, dwu=0, wg=0, wu=0, x=0), None) == cr.OK  # nothing wanted
    assert lib.convrot_gated_linear_backward_work_bytes(gated_grad_args(m=0)) == 0


SHAPE = dict(batch=2, tq=3, tk=5, hq=4, hk=2)
Q, K = (3 * 4 * 64, 4 * 64, 64), (5 * 2 * 64, 2 * 64, 64)


def attention_args(**kw):
    v = dict(q=FAKE, k=FAKE, v=FAKE, mask=0, out=FAKE, lse=FAKE, work=0, status=0) | SHAPE | dict(
        qs=Q, ks=K, vs=K, os=Q, mask_stride=5, work_bytes=0, scale=0.125, d=64, dtype=bl.BF16, reserved=0)
    assert set(kw) <= set(v)
    return pack(ATTENTION, (v | kw).values())


def attention_grad_args(**kw):
    v = dict(q=FAKE, k=FAKE, v=FAKE, out=FAKE, dout=FAKE, mask=0, lse=FAKE, dq=FAKE, dk=FAKE, dv=FAKE, work=FAKE, status=0) | SHAPE | dict(
        qs=Q, ks=K, vs=K, os=Q, dos=Q, mask_stride=5, work_bytes=1 << 30, scale=0.125, d=64, dtype=bl.BF16, reserved=0)
    assert set(kw) <= set(v)
    return pack(ATTENTION_BACKWARD, (v | kw).values())


BOTH_BAD = [
    (dict(batch=-1), cr.ERR_INVALID_ARG), (dict(tq=-1), cr.ERR_INVALID_ARG), (dict(tk=-1), cr.ERR_INVALID_ARG), (dict(hq=5), cr.ERR_INVALID_ARG),
    (dict(hk=0), cr.ERR_INVALID_ARG), (dict(d=0), cr.ERR_INVALID_ARG), (dict(d=129), cr.ERR_UNSUPPORTED), (dict(dtype=bl.F32), cr.ERR_UNSUPPORTED),
    (dict(dtype=7), cr.ERR_INVALID_ARG), (dict(scale=float("nan")), cr.ERR_INVALID_ARG), (dict(scale=float("inf")), cr.ERR_INVALID_ARG),
    (dict(scale=0.0), cr.ERR_INVALID_ARG), (dict(scale=-1.0), cr.ERR_INVALID_ARG), (dict(reserved=1), cr.ERR_INVALID_ARG), (dict(q=0), cr.ERR_INVALID_ARG),
    (dict(k=0), cr.ERR_INVALID_ARG), (dict(v=FAKE + 1), cr.ERR_ALIGNMENT), (dict(out=0), cr.ERR_INVALID_ARG), (dict(lse=0), cr.ERR_INVALID_ARG),
    (dict(lse=FAKE + 2), cr.ERR_ALIGNMENT), (dict(qs=(-1, 256, 64)), cr.ERR_INVALID_ARG), (dict(ks=(640, -1, 64)), cr.ERR_INVALID_ARG),
    (dict(mask_stride=-1), cr.ERR_INVALID_ARG), (dict(status=FAKE + 1), cr.ERR_ALIGNMENT), (dict(batch=1 << 25, tq=1 << 20), cr.ERR_INVALID_ARG),
]


@pytest.mark.parametrize("kw,status", BOTH_BAD, ids=[str(k) for k, _ in BOTH_BAD])
def test_attention_refuses(lib, kw, status):
    assert lib.convrot_attention(attention_args(**kw), None) == status
    assert lib.convrot_attention_backward(attention_grad_args(**kw), None) == status


def test_attention_refuses_its_own_operands(lib):
    assert lib.convrot_attention(None, None) == cr.ERR_INVALID_ARG
    assert lib.convrot_attention_backward(None, None) == cr.ERR_INVALID_ARG
    for strides in ((768, 256, 0), (768, 32, 64), (0, 256, 64), (768, 256, 256), (64, 256, 64)):  # heads of out over one another
        assert lib.convrot_attention(attention_args(os=strides), None) == cr.ERR_INVALID_ARG
    assert lib.convrot_attention(attention_args(mask=FAKE, tq=30, tk=200), None) == cr.ERR_INVALID_ARG  # needs a workspace
    for kw in (dict(dq=0), dict(dk=0), dict(dv=0), dict(dout=0), dict(work=0), dict(work_bytes=64)):
        assert lib.convrot_attention_backward(attention_grad_args(**kw), None) == cr.ERR_INVALID_ARG
    assert lib.convrot_attention_backward(attention_grad_args(work=FAKE + 8), None) == cr.ERR_ALIGNMENT


def test_empty_attention_launches_nothing(lib):
    for kw in (dict(batch=0), dict(tq=0), dict(hq=0)):
        assert lib.convrot_attention(attention_args(q=0, out=0, lse=0, **kw), None) == cr.OK
        assert lib.convrot_attention_work_bytes(attention_args(mask=FAKE, **kw)) == 0
    for kw in (dict(batch=0), dict(hq=0, hk=0)):
        assert lib.convrot_attention_backward(attention_grad_args(q=0, dq=0, dk=0, dv=0, **kw), None) == cr.OK


def test_attention_workspaces(lib):
    assert lib.convrot_attention_work_bytes(attention_args()) == 0
    many, rows = dict(tq=30), 2 * 256 * 2 * 64 * 2
    assert lib.convrot_attention_work_bytes(attention_args(mask=FAKE, **many, tk=200)) == 256 + 2 * rows
    assert lib.convrot_attention_work_bytes(attention_args(mask=FAKE, **many)) == 0  # a tile's mask is applied in place
    assert lib.convrot_attention_work_bytes(attention_args(q=FAKE + 2, **many)) == 2 * 30 * 4 * 64 * 2
    assert lib.convrot_attention_work_bytes(attention_args(tk=0, mask=FAKE, **many)) == 0
    # few queries: the mask is read as it is, unaligned keys are copied, and long states are shared out over clusters
    assert lib.convrot_attention_work_bytes(attention_args(mask=FAKE, q=FAKE + 2)) == 0
    assert lib.convrot_attention_work_bytes(attention_args(k=FAKE + 2)) == 2 * 5 * 2 * 64 * 2
    assert lib.convrot_attention_work_bytes(attention_args(tk=1 << 20)) > 0


def test_binding_refuses(lib):
    from torch._subclasses import FakeTensorMode

    with pytest.raises(TypeError):
        bl.convrot_gated_linear(torch.zeros(2, 8), torch.zeros(4, 8), torch.zeros(4, 8))  # not on the GPU
    with pytest.raises(TypeError):
        bl.convrot_attention(*(torch.zeros(1, 2, 2, 8) for _ in range(3)))
    with FakeTensorMode():
        on = dict(device="cuda", dtype=torch.bfloat16)
        x, w, y = torch.empty(3, 16, **on), torch.empty(8, 16, **on), torch.empty(3, 8, **on)
        for error, call in [
                (TypeError, lambda: bl.convrot_gated_linear(x, w, w.half())), (ValueError, lambda: bl.convrot_gated_linear(x, w, w[:4])),
                (ValueError, lambda: bl.convrot_gated_linear(x, w[:, :8], w)), (TypeError, lambda: bl.convrot_gated_linear(x[0], w, w)),
                (TypeError, lambda: bl.convrot_gated_linear(x, w, w, torch.empty(8, **on))), (ValueError, lambda: bl.convrot_gated_linear(x, w, w, out=x)),
                (TypeError, lambda: bl.convrot_gated_linear(x, w, w, out=y.half())),
                (ValueError, lambda: bl.convrot_gated_linear(x.t().contiguous().t(), w, w)),
                (ValueError, lambda: bl.convrot_gated_linear_backward(x, w, w, y, y, x)),
                (ValueError, lambda: bl.convrot_gated_linear(x, w, torch.empty(8, 16, device="cuda:1", dtype=torch.bfloat16)))]:
            with pytest.raises(error):
                call()
        q, k, mask = torch.empty(2, 3, 4, 64, **on), torch.empty(2, 5, 2, 64, **on), torch.empty(2, 5, device="cuda", dtype=torch.bool)
        lse = torch.empty(2, 4, 3, device="cuda")
        for error, call in [
                (TypeError, lambda: bl.convrot_attention(q[0], k, k)), (TypeError, lambda: bl.convrot_attention(q, k.half(), k)),
                (ValueError, lambda: bl.convrot_attention(q, k, k[:, :4])), (ValueError, lambda: bl.convrot_attention(q, k[:1], k)),
                (ValueError, lambda: bl.convrot_attention(q, k[..., :32], k)), (TypeError, lambda: bl.convrot_attention(q, k, k, mask.float())),
                (ValueError, lambda: bl.convrot_attention(q, k, k, mask[:1])), (ValueError, lambda: bl.convrot_attention(q, k, k, mask[:, :4])),
                (ValueError, lambda: bl.convrot_attention(q, k, k, out=k)), (ValueError, lambda: bl.convrot_attention(q.transpose(2, 3), k, k)),
                (ValueError, lambda: bl.convrot_attention(q, k, torch.empty(2, 5, 2, 64, device="cuda:1", dtype=torch.bfloat16))),
                (ValueError, lambda: bl.convrot_attention_backward(q, k, k, q, lse[:1], q)), (ValueError, lambda: bl.convrot_attention_backward(q, k, k, k, lse, q)),
                (ValueError, lambda: bl.convrot_attention_backward(q, k, k, q, lse, k))]:
            with pytest.raises(error):
                call()


# calls with tensors that have no memory of their own, each in a process: plain ones, and the slices that vmap hands out
WITHOUT_MEMORY = """
import sys, torch
from torch._subclasses import FakeTensorMode
from int8_hadamard_rotated_convrot_gb300 import block as bl
name, batched = sys.argv[1], sys.argv[2] == "vmap"
with FakeTensorMode():
    like = dict(device="cuda", dtype=torch.bfloat16)
    x, w, q, lse = torch.empty(4, 64, **like), torch.empty(32, 64, **like), torch.empty(2, 4, 2, 16, **like), torch.empty(2, 2, 4, device="cuda")
    y = torch.empty(4, 32, **like)
    call = {
        "gated": lambda t: bl.convrot_gated_linear(t, w, w),
        "gated out": lambda t: bl.convrot_gated_linear(t, w, w, keep=True, out=y)[1],
        "gated gradient": lambda t: bl.convrot_gated_linear_backward(t, w, w, y, y, y)["dx"],
        "attention": lambda t: bl.convrot_attention(t.view(2, 2, 2, 32), t.view(2, 2, 2, 32), t.view(2, 2, 2, 32))[0],
        "attention out": lambda t: bl.convrot_attention(q, q, q, out=t.view(2, 4, 2, 16))[0],
        "attention gradient": lambda t: bl.convrot_attention_backward(q, q, q, q, lse, t.view(2, 4, 2, 16))["dq"],
    }[name]
    try:
        torch.vmap(call)(torch.empty(3, 4, 64, **like)) if batched else call(x)
    except Exception as e:
        print("raised", type(e).__name__)
"""


@pytest.mark.parametrize("how", ["plain", "vmap"])
@pytest.mark.parametrize("name", ["gated", "gated out", "gated gradient", "attention", "attention out", "attention gradient"])
def test_tensors_without_memory_raise(lib, name, how):
    r = subprocess.run([sys.executable, "-c", WITHOUT_MEMORY, name, how], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("raised"), r.stdout + r.stderr[-2000:]


# ---------------------------------------------------------------- tensor memory

SM_SHARED, BLOCK_RESERVE, COLUMNS = 228 * 1024, 1024, 512
SOURCE = r"""
#include <cstdint>
#include <cstdio>
#include <initializer_list>
namespace convrot {
int lora_down_shared(int r);
int fp8_few_shared(int64_t m, int64_t n, int64_t k, bool quantize, int *columns);
int gated_gemm_shared(int form, int *columns);
int gated_few_shared(int form, int *columns);
int attention_shared(int form, int *columns);
int attention_grad_q_shared(int form, int *columns);
int attention_grad_kv_shared(int form, int *columns);
}
int main()
{
    using namespace convrot;
    int columns = 0;
    for (auto f : {gated_gemm_shared, gated_few_shared, attention_shared, attention_grad_q_shared, attention_grad_kv_shared})
        for (int form = 0; const int bytes = f(form, &columns); ++form) printf("%d %d\n", columns, bytes);
    // the smallest of the others, by columns
    for (int64_t m : {1, 17, 64}) {
        const int bytes = fp8_few_shared(m, 128, 128, false, &columns);
        printf("%d %d\n", columns, bytes);
    }
    for (int r = 16; r <= 256; r += 16) printf("512 %d\n", lora_down_shared(r));
}
"""


def test_no_mix_of_blocks_needs_more_columns_than_an_sm_has(lib, tmp_path):
    """Blocks that fit an SM side by side by their shared memory have 512 columns of tensor memory together at most."""
    source, program = tmp_path / "shapes.cpp", tmp_path / "shapes"
    source.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-o", str(program), str(source), "-L", cbuild.BUILD, "-lconvrot", "-Wl,-rpath," + cbuild.BUILD], check=True)
    least = {}
    for line in subprocess.run([str(program)], check=True, capture_output=True, text=True).stdout.split("\n"):
        if line:
            columns, shared = map(int, line.split())
            assert columns % 32 == 0 and 0 < columns <= COLUMNS and shared <= 227 * 1024
            least[columns] = min(shared, least.get(columns, shared))
    fits = SM_SHARED // (min(least.values()) + BLOCK_RESERVE)
    for n in range(1, fits + 2):
        for mix in itertools.combinations_with_replacement(sorted(least), n):
            if sum(least[c] + BLOCK_RESERVE for c in mix) <= SM_SHARED:
                assert sum(mix) <= COLUMNS, mix


def test_every_allocation_is_under_the_rule():
    for name in os.listdir(cbuild.CSRC16):
        text = open(os.path.join(cbuild.CSRC16, name)).read()
        if "tmem_alloc<" in text and name != "mma16.cuh":
            assert "tmem_share(" in text or "> kTmemAlone" in text, name
