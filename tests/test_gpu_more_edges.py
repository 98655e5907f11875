"""GPU tests of calls at the edges of what include/convrot_block.h allows of attention to other states and of the gated
linear, through the C entry points where the Python binding has no such call. The arguments are test_more_block_abi.py's."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from int8_hadamard_rotated_convrot_gb300 import block as bl  # noqa: E402
from int8_hadamard_rotated_convrot_gb300 import convrot as cr  # noqa: E402

from . import test_more_block_abi as abi  # noqa: E402

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
