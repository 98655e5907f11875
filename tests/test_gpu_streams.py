"""Memory of the int8 linears' calls on another stream than the current one: what
a call allocates belongs to its own stream, whatever the caller's does meanwhile."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from int8_hadamard_rotated_convrot_gb300 import convrot as cr  # noqa: E402


@pytest.fixture(scope="module")
def calls():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from int8_hadamard_rotated_convrot_gb300 import build

    build.build()
    cr.load()
    g = torch.Generator(device="cuda").manual_seed(3)
    randn = lambda *shape: torch.randn(*shape, generator=g, device="cuda")
    m, n, k, r, G = 300, 1024, 512, 16, 256
    X, W, bias, A, B = randn(m, k), 0.02 * randn(n, k), randn(n), randn(r, k), 0.05 * randn(n, r)
    x, w = cr.convrot_pack_activations(X, G, cr.CODES_BF16), cr.convrot_quantize_weights(W, G, cr.CODES_BF16)
    a_ext, b_ext = cr.convrot_lora_prepare_down(A), cr.convrot_lora_prepare(B, 2.0)
    t_ext = cr.convrot_lora_down(X, a_ext)
    torch.cuda.synchronize()

    def rows(p):
        return [p.q, p.scale]

    return {
        "pack": lambda s: rows(cr.convrot_pack_activations(X, G, cr.CODES_BF16, stream=s)),
        "weights": lambda s: rows(cr.convrot_quantize_weights(W, G, stream=s)),
        "linear": lambda s: [cr.convrot_linear(x, w, bias, stream=s)],
        "linear and pack": lambda s: rows(cr.convrot_linear_act_pack(x, w, bias, cr.ACT_GELU_TANH, G, stream=s)),
        "rotated in two": lambda s: rows(cr.convrot_linear_act_pack(x, w, bias, cr.ACT_NONE, 1024, stream=s)),
        "adapter up": lambda s: [cr.convrot_lora_prepare(B, 2.0, stream=s)],
        "adapter down": lambda s: [cr.convrot_lora_prepare_down(A, stream=s)],
        "adapter rows": lambda s: [cr.convrot_lora_down(X, a_ext, stream=s)],
        "linear with adapter": lambda s: [cr.convrot_linear_lora(x, w, bias, 0, t_ext, b_ext, r, stream=s)],
        "integers": lambda s: [cr.convrot_gemm_i32(x, w, stream=s)],
    }


@pytest.mark.parametrize("name", ["pack", "weights", "linear", "linear and pack", "rotated in two", "adapter up", "adapter down",
                                  "adapter rows", "linear with adapter", "integers"])
def test_memory_of_a_call_on_another_stream(calls, name):
    want = [t.clone() for t in calls[name](None)]
    sizes = [t.numel() * t.element_size() for t in want] + [300 * 1024 * 4, 300 * 1024 * 4 + 300 * 4 + 4096, 2 << 20]
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
                got = calls[name](side)
                kept = fill()
            else:
                kept = fill()
                del kept
                got = calls[name](side)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want, strict=True))
