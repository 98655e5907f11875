"""The example that runs the operators around the linears together, against the
same stretch in plain 64-bit torch on the dequantized weights, forward and back.

The difference is the e4m3 rounding of the activations: at most 2^-4 of a value,
2^-4 / sqrt(12) to 2^-4 / sqrt(3) of it in the root mean square, so 4 % of a
linear's output; three linears in a row, and the bf16 results between them, stay
under 10 % of the norm of any output, and the six of a gradient under 15 %."""

import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from . import block_reference as ref  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from int8_hadamard_rotated_convrot_gb300 import build

    build.build()
    spec = importlib.util.spec_from_file_location("between_attentions", os.path.join(ROOT, "examples", "between_attentions.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def plain(net, x, attention, modulation, tables):
    b, t, d = x.shape

    def linear(v, layer):
        return v @ layer.w.dequantize().double().t() + layer.bias.double()

    (g1, c1, s1), (g2, c2, s2) = [[m.double() for m in ms] for ms in modulation]
    y1 = linear(attention.reshape(-1, d), net.proj)
    h1, n1 = ref.gated_norm(x.reshape(-1, d), y1, g1, c1, s1, rows=t, pre_weight=net.norms[0].double())
    y2 = linear(ref.act(linear(n1, net.up), 2), net.down)
    h2, n2 = ref.gated_norm(h1, y2, g2, c2, s2, rows=t, pre_weight=net.norms[1].double())
    q, k, v = linear(n2, net.qkv).view(b, t, 3 * net.heads, net.head_dim).split(net.heads, 2)
    at = torch.arange(t, device=x.device).expand(b, t)
    cos, sin = (m.double()[at][:, :, None] for m in tables)

    def rotate(z):
        a, c = z.chunk(2, -1)
        return torch.cat([a * cos - c * sin, c * cos + a * sin], -1)

    return h2.view(b, t, d), rotate(q), rotate(k), v


@pytest.mark.parametrize("batch,tokens,width,heads,hidden", [(2, 150, 512, 8, 1024), (1, 1, 256, 4, 640), (3, 7, 384, 4, 512)])
def test_stretch_between_attentions(example, batch, tokens, width, heads, hidden):
    net = example.Stretch(width, heads, hidden, seed=tokens)
    g = torch.Generator(device="cuda").manual_seed(5)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    x, attention = (normal(batch, tokens, width).bfloat16() for _ in range(2))
    modulation = [[0.3 * normal(batch, width) for _ in range(3)] for _ in range(2)]
    tables = net.tables(tokens)
    got, saved = net.forward(x, attention, modulation, tables)
    wide = [t.double().requires_grad_() for t in (x, attention)]
    want = plain(net, *wide, modulation, tables)
    for name, a, b in zip(("residual", "q", "k", "v"), got, want):
        off = float((a.double() - b.detach()).norm() / b.detach().norm())
        assert off < 0.10, f"{name}: {off:.3f}"
    up = [0.1 * normal(*t.shape).bfloat16() for t in got]
    dx = net.input_gradient(saved, modulation, tables, *up)
    for name, a, b in zip(("x", "attention"), dx, torch.autograd.grad(want, wide, [u.double() for u in up])):
        off = float((a.double() - b.detach()).norm() / b.detach().norm())
        assert off < 0.15, f"gradient of {name}: {off:.3f}"


def test_long_context_tables(example):
    net = example.Stretch(256, 4, 256)
    cos, sin = net.tables(4096, scale=4.0)
    assert cos.shape == sin.shape == (4096, 32)
    # YaRN's attention factor is on both
    assert abs(float((cos**2 + sin**2).sqrt().mean()) - (1 + 0.1 * 1.3862943611198906)) < 1e-5
