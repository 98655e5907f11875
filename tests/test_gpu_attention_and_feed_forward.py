"""The example that runs attention to a prompt and the gated feed-forward together, against the same run in plain 64-bit
torch on the dequantized weights, forward and back; and their calls on other streams, at once, in captured graphs and with
workspaces of the caller's.

The difference from 64 bits is the e4m3 rounding of the frozen projections' inputs: 4 % of a linear's output at most in the
root mean square (its largest is 2^-4 of a value). The residual stream has it from two projections in a row beside the
attention's probabilities, whose exponents are off by what q and k are: under 10 % of its norm. A gradient passes through up
to five such projections, and through the attention's probabilities twice: sqrt(5 + 4) times 4 % and what the forward's own
differences add, under 20 %."""

import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from int8_hadamard_rotated_convrot_gb300 import block as bl  # noqa: E402

from . import block_reference as ref  # noqa: E402
from . import more_reference as more  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from int8_hadamard_rotated_convrot_gb300 import build

    build.build()
    path = os.path.join(ROOT, "examples", "attention_and_feed_forward.py")
    spec = importlib.util.spec_from_file_location("attention_and_feed_forward", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def plain(net, x, prompt, mask, w, bias):
    b, t, d = x.shape
    n = net.hidden

    def linear(v, layer):
        return v @ layer.w.dequantize().double().t() + layer.bias.double()

    _, n1 = ref.gated_norm(x.reshape(-1, d), pre_weight=net.norms[0].double())
    q = linear(n1, net.q).view(b, t, net.heads, -1).transpose(1, 2)
    k, v = linear(prompt.reshape(-1, d), net.kv).view(b, -1, 2, net.heads, net.head_dim).permute(2, 0, 3, 1, 4)
    scores = (q @ k.transpose(2, 3) * net.head_dim**-0.5).masked_fill(~mask[:, None, None], -float("inf"))
    a = (torch.softmax(scores, -1) @ v).transpose(1, 2).reshape(-1, d)
    h1, n2 = ref.gated_norm(x.reshape(-1, d), linear(a, net.proj), pre_weight=net.norms[1].double())
    y = more.act(n2 @ w[:n].t() + bias[:n], more.SILU) * (n2 @ w[n:].t() + bias[n:])
    return (h1 + linear(y, net.down)).view(b, t, d)


@pytest.mark.parametrize("batch,tokens,prompt,width,heads,hidden", [(2, 300, 77, 512, 8, 1024), (2, 150, 200, 384, 3, 640), (1, 1, 5, 256, 4, 320)])
def test_attention_and_feed_forward(example, batch, tokens, prompt, width, heads, hidden):
    net = example.Half(width, heads, hidden, seed=tokens)
    g = torch.Generator(device="cuda").manual_seed(5)
    x, states = (torch.randn(batch, n, width, generator=g, device="cuda").bfloat16() for n in (tokens, prompt))
    mask = torch.arange(prompt, device="cuda") < torch.tensor([prompt * (i + 1) // batch for i in range(batch)], device="cuda")[:, None]
    got, saved = net.forward(x, states, mask)
    wide = {"x": x, "prompt": states, "w": net.w, "b": net.b}
    wide = {name: t.double().requires_grad_() for name, t in wide.items()}
    want = plain(net, wide["x"], wide["prompt"], mask, wide["w"], wide["b"])
    off = float((got.double() - want.detach()).norm() / want.detach().norm())
    assert off < 0.10, f"residual: {off:.3f}"
    dh = (0.1 * torch.randn(*got.shape, generator=g, device="cuda")).bfloat16()
    grads = net.gradient(x, saved, mask, dh)
    for (name, t), b in zip(wide.items(), torch.autograd.grad(want, list(wide.values()), dh.double())):
        off = float((grads[name].double() - b).norm() / b.norm())
        assert grads[name].shape == t.shape and off < 0.20, f"gradient of {name}: {off:.3f}"
    assert not grads["prompt"][~mask].any()


# ---------------------------------------------------------------- streams, graphs, workspaces


def make_calls():
    g = torch.Generator(device="cuda").manual_seed(3)

    def randn(*shape, dtype=BF16, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    calls = {}
    for name, m, k, n, pad in (("few", 5, 512, 384, 0), ("many", 700, 320, 520, 0), ("unaligned", 300, 200, 200, 1)):
        x, wg, wu = randn(m, k + pad)[:, :k], randn(n, k + pad, std=k**-0.5)[:, :k], randn(n, k, std=k**-0.5)
        bg, bu = randn(n, dtype=torch.float32), randn(n, dtype=torch.float32)
        gate, up, dy = randn(m, n), randn(m, n), randn(m, n)
        calls["gated " + name] = lambda s=None, x=x, wg=wg, wu=wu, bg=bg, bu=bu, **kw: list(
            bl.convrot_gated_linear(x, wg, wu, bg, bu, keep=True, stream=s, **kw))
        calls["gated gradient " + name] = lambda s=None, x=x, wg=wg, wu=wu, gate=gate, up=up, dy=dy, **kw: list(
            bl.convrot_gated_linear_backward(x, wg, wu, gate, up, dy, biases=True, stream=s, **kw).values())
    for name, b, tq, tk, hq, hk, d, masked in (("few", 2, 3, 900, 8, 2, 64, True), ("long", 1, 1, 70000, 2, 1, 64, False), ("one tile", 2, 600, 77, 4, 4, 64, True),
                                               ("wide heads", 2, 300, 100, 2, 1, 128, True), ("gathered", 2, 300, 333, 4, 2, 72, True),
                                               ("unaligned", 1, 140, 150, 2, 2, 33, False)):
        q, k, v, dout = randn(b, tq, hq, d), randn(b, tk, hk, d), randn(b, tk, hk, d), randn(b, tq, hq, d)
        mask = torch.rand(b, tk, generator=g, device="cuda") < 0.6 if masked else None
        out, lse = bl.convrot_attention(q, k, v, mask)
        calls["attention " + name] = lambda s=None, q=q, k=k, v=v, mask=mask, **kw: list(bl.convrot_attention(q, k, v, mask, stream=s, **kw))
        calls["attention gradient " + name] = lambda s=None, q=q, k=k, v=v, mask=mask, out=out, lse=lse, dout=dout, **kw: list(
            bl.convrot_attention_backward(q, k, v, out, lse, dout, mask, stream=s, **kw).values())
    torch.cuda.synchronize()
    return calls


NAMES = [f"{op} {kind}" for op, kinds in (("gated", ("few", "many", "unaligned")), ("attention", ("few", "long", "one tile", "wide heads", "gathered", "unaligned")))
         for kind in kinds] + [f"{op} gradient {kind}" for op, kinds in (("gated", ("few", "many", "unaligned")),
                                                                         ("attention", ("few", "long", "one tile", "wide heads", "gathered", "unaligned")))
                               for kind in kinds]


@pytest.fixture(scope="module")
def calls(example):
    return make_calls()


def same(got, want):
    return all(torch.equal(a.view(torch.uint8) if a.dtype != torch.uint8 else a, b.view(torch.uint8)) for a, b in zip(got, want, strict=True))


@pytest.mark.parametrize("name", NAMES)
def test_memory_of_a_call_on_another_stream(calls, name):
    """What a call allocates belongs to its own stream, whatever the caller's does meanwhile."""
    want = [t.clone() for t in calls[name]()]
    sizes = [t.numel() * t.element_size() for t in want] + [300 * 200 * 2, 700 * 520 * 2, 2 << 20]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()

    def fill():
        return [torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]

    for late in (side, torch.cuda.current_stream()):
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
        assert same(got, want)


def test_calls_at_once(calls):
    """Every call on one of four streams, all in flight together, twice over."""
    want = {name: [t.clone() for t in call()] for name, call in calls.items()}
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    got = []
    for turn in range(2):
        for i, name in enumerate(calls):
            got.append((name, calls[name](streams[(i + turn) % 4])))
    torch.cuda.synchronize()
    for name, result in got:
        assert same(result, want[name]), name


def test_calls_in_a_graph(calls):
    """All calls captured together, with the workspaces that they allocate, and replayed."""
    want = {name: [t.clone() for t in call()] for name, call in calls.items()}
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        kept = {name: call() for name, call in calls.items()}
    for _ in range(3):
        for result in kept.values():
            for t in result:
                t.view(torch.uint8).fill_(0x7F)
        graph.replay()
        torch.cuda.synchronize()
        for name in want:
            assert same(kept[name], want[name]), name


@pytest.mark.parametrize("name", NAMES)
def test_workspace_of_the_caller(calls, name):
    """A workspace with anything in it, used twice, gives what the call's own does; what is behind its end stays."""
    want = calls[name]()
    big = torch.full((96 << 20,), 0x7F, dtype=torch.uint8, device="cuda")
    work = big[: 64 << 20]
    for _ in range(2):
        assert same(calls[name](work=work), want)
    assert torch.all(big[64 << 20:] == 0x7F)


def test_inference_mode_and_ordinary_tensors(calls):
    with torch.inference_mode():
        want = calls["attention one tile"]()
    out, lse = calls["attention one tile"]()
    assert same([out, lse], want)
    leaf = torch.ones_like(out).requires_grad_()
    (leaf * out).sum().backward()  # as a constant of a graph
    assert torch.equal(leaf.grad, out)
