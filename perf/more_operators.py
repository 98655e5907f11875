"""Attention to other states and the gated feed-forward input, as cases to measure.

Two operators that a transformer block has beside its 8-bit linears, each with
its gradient:

  attention  out = softmax(scale q k^T) v with queries [batch, tokens, heads,
             head_dim] and keys and values of another length (an encoder's
             states, a prompt), with as many heads or fewer, and a mask that says
             which keys there are; beside it the logarithm of each row's sum
  gated      y = act(x w_gate^T + b_gate) * (x w_up^T + b_up) with 16-bit
             weights: both projections of a gated feed-forward, the activation
             and the product

Where ``own`` is false, ``run`` computes them with elementary torch operations
in 32 bits, rounded once at the end; where it is true, with the framework's
kernels.
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------- the cases

def _attention(name, b, tq, tk, hq, hk, d, t="bf16", mask="none", backward=False):
    return {"name": name, "op": "attention", "b": b, "tq": tq, "tk": tk, "hq": hq, "hk": hk, "d": d, "t": t, "mask": mask,
            "backward": backward}


def _gated(name, m, k, n, t="bf16", act="silu", bias=False, keep=False, backward=False, weights=False):
    return {"name": name, "op": "gated", "m": m, "k": k, "n": n, "t": t, "act": act, "bias": bias, "keep": keep,
            "backward": backward, "weights": weights}


def listed():
    return [
        # one new token for each of eight sequences against a long encoder's states, shared key heads: latency and bytes
        _attention("attention_token", 8, 1, 4096, 40, 8, 128),
        # an image's tokens against two prompts of a guided step, the shorter one padded
        _attention("attention_prompt", 2, 4096, 77, 10, 10, 64, t="f16", mask="padded"),
        # lengths and heads that are no multiple of a tile, keys dropped anywhere
        _attention("attention_ragged", 3, 1363, 333, 24, 8, 72, mask="scattered"),
        # a video's tokens against a text encoder's 512 states
        _attention("attention_video", 1, 32760, 512, 40, 40, 128),
        # training: the gradient for an image's tokens and two prompts
        _attention("attention_gradient_prompt", 2, 4096, 77, 10, 10, 64, t="f16", mask="padded", backward=True),
        # training: the gradient at a quarter of a video
        _attention("attention_gradient_video", 1, 8190, 512, 40, 40, 128, backward=True),
        # one token: all latency and weight bytes
        _gated("gated_token", 1, 5120, 13824),
        # a prompt through widths that are no multiple of a tile
        _gated("gated_prompt_ragged", 77, 2056, 3080, t="f16", act="gelu_erf", bias=True),
        # an image's tokens in training: both projections are kept for the gradient
        _gated("gated_image_kept", 4096, 1280, 5120, t="f16", act="gelu_erf", bias=True, keep=True),
        # a video's tokens
        _gated("gated_video", 32760, 5120, 13824, act="gelu_tanh"),
        # training an adapter: the input's gradient through frozen weights, an odd number of tokens
        _gated("gated_input_gradient", 1023, 1280, 5120, t="f16", act="gelu_erf", backward=True),
        # training all of it: the gradients of input, weights and biases
        _gated("gated_gradient", 8190, 5120, 13824, act="silu", bias=True, backward=True, weights=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _maybe_round(rng, v, to):
    """Half of the widths are multiples of `to`, as most models' are."""
    return max(to, v // to * to) if rng.random() < 0.5 else v


def draw(rng):
    t = rng.choice(["bf16", "bf16", "f16"])
    backward = rng.random() < 0.45
    if rng.random() < 0.5:
        d = rng.choice([32, 40, 64, 64, 72, 80, 96, 100, 128, 128])
        b, hq = _log(rng, 1, 16), _log(rng, 1, 48)
        hk = rng.choice([h for h in range(1, hq + 1) if hq % h == 0])
        tk = _log(rng, 1, min(4096, 16 * 4096 * 8 * 128 // (b * hk * d)))
        scores = 40 * (8190 if backward else 32760) * 512
        tq = _log(rng, 1, max(2, min(32760, scores // (b * hq * tk), (4 if backward else 16) * 8190 * 40 * 128 // (b * hq * d) // 4)))
        c = _attention("", b, tq, tk, hq, hk, d, t=t, mask=rng.choice(["none", "none", "padded", "scattered", "empty"]), backward=backward)
    else:
        k, n = (_maybe_round(rng, _log(rng, 256, 13824), 64) for _ in range(2))
        m = _log(rng, 1, max(2, min(32760, (8190 if backward else 32760) * 5120 * 13824 // (k * n))))
        c = _gated("", m, k, n, t=t, act=rng.choice(["silu", "silu", "gelu_tanh", "gelu_erf", "none"]), bias=rng.random() < 0.5,
                   keep=not backward and rng.random() < 0.3, backward=backward, weights=backward and rng.random() < 0.6)
    del c["name"]
    return c


# ---------------------------------------------------------------- what a program has in hand

def _lengths(c):
    """The number of keys of each sample."""
    if c["mask"] == "none":
        return [c["tk"]] * c["b"]
    some = [max(1, c["tk"] * (i + 1) // c["b"]) for i in range(c["b"])]
    return [0] + some[1:] if c["mask"] == "empty" else some


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    t = TYPES[case["t"]]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=DEV) * std

    if case["op"] == "attention":
        b, tq, tk, hq, hk, d = (case[v] for v in ("b", "tq", "tk", "hq", "hk", "d"))
        q = normal(b, tq, hq, d).to(t)
        kv = normal(b, tk, 2, hk, d).to(t)  # one projection's output
        s = {"case": case, "q": q, "k": kv[:, :, 0], "v": kv[:, :, 1], "mask": None, "scale": d**-0.5}
        if case["mask"] != "none":
            count = torch.tensor(_lengths(case), device=DEV)[:, None]
            at = torch.arange(tk, device=DEV).expand(b, tk)
            if case["mask"] == "scattered":  # which keys are there is the seed's
                at = torch.rand(b, tk, generator=g, device=DEV).argsort(1).argsort(1)
            s["mask"] = at < count
        if case["backward"]:
            s["out"], s["lse"] = _plain_attention(s)  # kept from the forward pass
            s["dout"] = normal(b, tq, hq, d, std=0.1).to(t)
        return s
    m, k, n = case["m"], case["k"], case["n"]
    s = {"case": case, "x": normal(m, k).to(t), "w_gate": normal(n, k, std=k**-0.5).to(t), "w_up": normal(n, k, std=k**-0.5).to(t),
         "b_gate": None, "b_up": None}
    if case["bias"]:
        s["b_gate"], s["b_up"] = normal(n, std=0.1), normal(n, std=0.1)
    if case["backward"]:
        s["gate"], s["up"] = (v.to(t) for v in _plain_projections(s))  # kept from the forward pass
        s["dy"] = normal(m, n, std=0.1).to(t)
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    from int8_hadamard_rotated_convrot_gb300 import block

    c = s["case"]
    if c["op"] == "attention":
        if not c["backward"]:
            return block.convrot_attention(s["q"], s["k"], s["v"], s["mask"], scale=s["scale"])
        return block.convrot_attention_backward(s["q"], s["k"], s["v"], s["out"], s["lse"], s["dout"], s["mask"], scale=s["scale"])
    act = {"none": block.ACT_NONE, "silu": block.ACT_SILU, "gelu_erf": block.ACT_GELU_ERF, "gelu_tanh": block.ACT_GELU_TANH}[c["act"]]
    if not c["backward"]:
        return block.convrot_gated_linear(s["x"], s["w_gate"], s["w_up"], s["b_gate"], s["b_up"], act, keep=c["keep"])
    grads = block.convrot_gated_linear_backward(s["x"], s["w_gate"], s["w_up"], s["gate"], s["up"], s["dy"], act, weights=c["weights"],
                                                biases=c["weights"] and c["bias"])
    return {name: v for name, v in grads.items() if v is not None}


def _run_plain(s):
    c = s["case"]
    if c["op"] == "attention":
        return _plain_attention_gradient(s) if c["backward"] else _plain_attention(s)
    return _plain_gated_gradient(s) if c["backward"] else _plain_gated(s)


def _by_heads(v, heads):
    """[batch, heads, tokens, head_dim] in 32 bits; a shared head is there for each query head that reads it."""
    return v.float().transpose(1, 2).repeat_interleave(heads // v.shape[2], 1)


def _plain_scores(s):
    q = s["q"].float().transpose(1, 2)
    scores = (q @ _by_heads(s["k"], q.shape[1]).transpose(2, 3)) * s["scale"]
    if s["mask"] is not None:
        scores = scores.masked_fill(~s["mask"][:, None, None], -math.inf)
    return scores


def _plain_softmax(s):
    """(probabilities, logarithm of the sums); a row without keys has zeros and -infinity."""
    scores = _plain_scores(s)
    top = scores.amax(3, keepdim=True)
    e = torch.exp(scores - top.clamp_min(torch.finfo(torch.float32).min))
    total = e.sum(3, keepdim=True)
    return e / total.clamp_min(torch.finfo(torch.float32).tiny), (top + total.log())[..., 0]


def _plain_attention(s):
    p, lse = _plain_softmax(s)
    out = p @ _by_heads(s["v"], p.shape[1])
    return out.transpose(1, 2).contiguous().to(s["q"].dtype), lse


def _shared(grad, like):
    """[batch, tokens, heads, head_dim] of a gradient by query heads, added up over those that share a head."""
    b, h, t, d = grad.shape
    return grad.view(b, like.shape[2], -1, t, d).sum(2).transpose(1, 2).contiguous().to(like.dtype)


def _plain_attention_gradient(s):
    p, _ = _plain_softmax(s)
    heads, dout = p.shape[1], s["dout"].float().transpose(1, 2)
    dp = dout @ _by_heads(s["v"], heads).transpose(2, 3)
    ds = p * (dp - (p * dp).sum(3, keepdim=True)) * s["scale"]
    dq = (ds @ _by_heads(s["k"], heads)).transpose(1, 2).contiguous().to(s["q"].dtype)
    dk = ds.transpose(2, 3) @ s["q"].float().transpose(1, 2)
    return {"dq": dq, "dk": _shared(dk, s["k"]), "dv": _shared(p.transpose(2, 3) @ dout, s["v"])}


def _plain_projections(s):
    x = s["x"].float()
    gate, up = x @ s["w_gate"].float().t(), x @ s["w_up"].float().t()
    if s["b_gate"] is not None:
        gate, up = gate + s["b_gate"], up + s["b_up"]
    return gate, up


def _plain_act(v, kind):
    """(act(v), its derivative)"""
    if kind == "silu":
        p = torch.sigmoid(v)
        return v * p, p * (1 + v * (1 - p))
    if kind == "gelu_erf":
        p = 0.5 * (1 + torch.erf(v * math.sqrt(0.5)))
        return v * p, p + v * torch.exp(-0.5 * v * v) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        th = torch.tanh(c * (v + 0.044715 * v * v * v))
        return 0.5 * v * (1 + th), 0.5 * (1 + th) + 0.5 * v * (1 - th * th) * c * (1 + 3 * 0.044715 * v * v)
    return v, torch.ones_like(v)


def _plain_gated(s):
    c, t = s["case"], s["x"].dtype
    gate, up = _plain_projections(s)
    y = (_plain_act(gate, c["act"])[0] * up).to(t)
    return (y, gate.to(t), up.to(t)) if c["keep"] else y


def _plain_gated_gradient(s):
    c, t = s["case"], s["x"].dtype
    a, slope = _plain_act(s["gate"].float(), c["act"])
    dy = s["dy"].float()
    dgate, dup = dy * s["up"].float() * slope, dy * a
    out = {"dx": (dgate @ s["w_gate"].float() + dup @ s["w_up"].float()).to(t)}
    if c["weights"]:
        x = s["x"].float()
        out |= {"dw_gate": (dgate.t() @ x).to(t), "dw_up": (dup.t() @ x).to(t)}
        if c["bias"]:
            out |= {"db_gate": dgate.sum(0), "db_up": dup.sum(0)}
    return out


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"] == "attention":
        b, tq, hq, hk, d = (case[v] for v in ("b", "tq", "hq", "hk", "d"))
        keys = sum(_lengths(case))
        q, kv, rows = b * tq * hq * d * 2, 2 * keys * hk * d * 2, b * tq * hq * 4
        mask = b * case["tk"] * (case["mask"] != "none")
        if case["backward"]:  # q, out, dout and the sums in, dq out; k and v in, their gradients (of every key) out
            return {"bytes": 4 * q + kv + 2 * b * case["tk"] * hk * d * 2 + rows + mask, "flops": 10 * tq * keys * hq * d}
        return {"bytes": 2 * q + kv + rows + mask, "flops": 4 * tq * keys * hq * d}
    m, k, n = case["m"], case["k"], case["n"]
    x, w, y = m * k * 2, 2 * n * k * 2, m * n * 2
    if not case["backward"]:
        return {"bytes": x + w + y * (3 if case["keep"] else 1) + 8 * n * case["bias"], "flops": 4 * m * n * k}
    grads = x + (x + w + 8 * n * case["bias"] if case["weights"] else 0)  # dx out; with the weights' x in and theirs out
    return {"bytes": w + 3 * y + grads, "flops": (8 if case["weights"] else 4) * m * n * k}


# ---------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_attention(case, s) if case["op"] == "attention" else _exact_gated(case, s)


def _exact_attention(c, s):
    # sample by sample, over the keys that are there; gradients by the rules of products, quotients and exponentials
    b, tq, tk, hq, hk, d = (c[v] for v in ("b", "tq", "tk", "hq", "hk", "d"))
    zeros = lambda *shape: torch.zeros(*shape, device=DEV, dtype=torch.float64)  # noqa: E731
    out, lse, dq = zeros(b, tq, hq, d), torch.full((b, hq, tq), -math.inf, device=DEV, dtype=torch.float64), zeros(b, tq, hq, d)
    dk, dv = zeros(b, tk, hk, d), zeros(b, tk, hk, d)
    group = hq // hk
    for i in range(b):
        there = torch.arange(tk, device=DEV) if s["mask"] is None else torch.nonzero(s["mask"][i])[:, 0]
        if len(there) == 0:
            continue
        q = s["q"][i].double().view(tq, hk, group, d)
        k, v = s["k"][i][there].double(), s["v"][i][there].double()
        logits = torch.einsum("thgd,khd->hgtk", q, k).mul_(s["scale"])
        total = torch.logsumexp(logits, -1)
        p = logits.sub_(total[..., None]).exp_()
        if not c["backward"]:
            lse[i] = total.reshape(hq, tq)
            out[i] = torch.einsum("hgtk,khd->thgd", p, v).reshape(tq, hq, d)
            continue
        g = s["dout"][i].double().view(tq, hk, group, d)
        dv[i, there] = torch.einsum("hgtk,thgd->khd", p, g)
        e = torch.einsum("thgd,khd->hgtk", g, v)
        e = p * (e - torch.einsum("hgtk,hgtk->hgt", p, e)[..., None])
        dq[i] = s["scale"] * torch.einsum("hgtk,khd->thgd", e, k).reshape(tq, hq, d)
        dk[i, there] = s["scale"] * torch.einsum("hgtk,thgd->khd", e, q)
    return {"dq": dq, "dk": dk, "dv": dv} if c["backward"] else (out, lse)


def _exact_act(v, kind):
    if kind == "silu":
        return v / (1 + torch.exp(-v))
    if kind == "gelu_erf":
        return v * torch.special.ndtr(v)
    if kind == "gelu_tanh":
        return v * torch.sigmoid(math.sqrt(8 / math.pi) * (v + 0.044715 * v**3))
    return v


def _exact_gated(c, s):
    if c["backward"]:
        gate, up = (s[v].double().requires_grad_() for v in ("gate", "up"))
        dgate, dup = torch.autograd.grad(_exact_act(gate, c["act"]) * up, (gate, up), s["dy"].double())
        out = {"dx": torch.mm(dgate, s["w_gate"].double()) + torch.mm(dup, s["w_up"].double())}
        if c["weights"]:
            x = s["x"].double()
            out |= {"dw_gate": torch.mm(dgate.T, x), "dw_up": torch.mm(dup.T, x)}
            if c["bias"]:
                out |= {"db_gate": torch.einsum("mn->n", dgate), "db_up": torch.einsum("mn->n", dup)}
        return out
    x = s["x"].double()
    gate, up = torch.mm(x, s["w_gate"].double().T), torch.mm(x, s["w_up"].double().T)
    if c["bias"]:
        gate, up = gate + s["b_gate"].double(), up + s["b_up"].double()
    y = _exact_act(gate, c["act"]) * up
    return (y, gate, up) if c["keep"] else y
