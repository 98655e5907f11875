"""The operators of a transformer block around its 8-bit linears, as cases to measure.

Three operators carry a block from one attention's output to the inputs of the
next one:

  linear   y = act(x w^T + b) with x and w in 8-bit floating point (e4m3): x is
           quantized here, one scale for each 128 consecutive features of a row,
           w is held as codes with one scale for each 128 x 128 block
  norm     h = res_scale x + gate * post(y), n = pre(h) (1 + scale) + shift, and
           its gradient
  rotary   positions rotated into queries and keys, and its gradient (the
           rotation by the opposite angles)

Where ``own`` is false, ``run`` computes them with elementary torch operations
in 32 bits, rounded once at the end; where it is true, with the framework's
kernels.
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
BLOCK = 128            # features, and weight rows, that share a scale
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0**-96  # an all-zero block gets the scale of this maximum
EPS = 1e-6


# ---------------------------------------------------------------- the cases

def _linear(name, m, k, n, x="bf16", y="bf16", bias=True, act="none"):
    return {"name": name, "op": "linear", "m": m, "k": k, "n": n, "x": x, "y": y, "bias": bias, "act": act}


def _norm(name, m, d, rows, t="bf16", p="f32", backward=False, post="none", post_affine=False, pre="layer",
          pre_affine=False, branch=True, gate=True, modulate=True, res_scale=1.0):
    return {"name": name, "op": "norm", "m": m, "d": d, "rows": rows, "t": t, "p": p, "backward": backward,
            "post": post, "post_affine": post_affine, "pre": pre, "pre_affine": pre_affine, "branch": branch,
            "gate": gate, "modulate": modulate, "res_scale": res_scale}


def _rotary(name, b, t, hq, hk, d, r, dtype="bf16", layout="half", inverse=False, table=0):
    return {"name": name, "op": "rotary", "b": b, "t": t, "hq": hq, "hk": hk, "d": d, "r": r, "dtype": dtype,
            "layout": layout, "inverse": inverse, "table": table}


def listed():
    return [
        # one token (or one conditioning vector) through a square projection: all latency and weight bytes
        _linear("linear_token", 1, 5120, 5120),
        # a text prompt through an adapter whose widths are no multiple of a tile or of a block
        _linear("linear_prompt_ragged", 77, 2056, 3080, x="f16", y="f16"),
        # a video's tokens through the up projection of the MLP, GELU in the epilogue
        _linear("linear_video_up", 32760, 5120, 13824, act="gelu_tanh"),
        # training an adapter over frozen weights: dX = dY W, from 32-bit gradients
        _linear("linear_input_gradient", 8190, 13824, 5120, x="f32", y="f32", bias=False),
        # one row each for the two halves of a guided step, as a single-token step has them
        _norm("norm_token", 2, 5120, 1),
        # an odd width, weights and bias of a trained norm, no branch: the first norm of a model
        _norm("norm_odd_width", 4097, 1155, 4097, t="f16", p="f16", pre="layer", pre_affine=True, branch=False,
              gate=False, modulate=False),
        # norms on both sides of the block, at video length
        _norm("norm_video_sandwich", 32760, 5120, 32760, p="bf16", post="rms", post_affine=True, pre="rms",
              pre_affine=True),
        # the gradient for three samples of ragged length
        _norm("norm_gradient", 8190, 5120, 2730, backward=True, post="rms", post_affine=True, pre="rms",
              pre_affine=True),
        # the gradient at a prompt's length, in 32 bits, layer norm with residual scale
        _norm("norm_gradient_prompt", 77, 1024, 77, t="f32", backward=True, pre_affine=True, res_scale=0.5),
        # one new token for each of eight sequences, deep in a long context, shared key heads
        _rotary("rotary_token", 8, 1, 40, 8, 128, 128, table=131072),
        # gradient through a rotation of part of the head, 32 bits, odd length
        _rotary("rotary_partial_gradient", 3, 1363, 24, 24, 96, 48, dtype="f32", inverse=True),
        # a video's queries and keys, interleaved pairs
        _rotary("rotary_video", 1, 32760, 40, 40, 128, 128, layout="interleaved"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _maybe_round(rng, v, to):
    """Half of the widths are multiples of `to`, as most models' are."""
    return max(to, v // to * to) if rng.random() < 0.5 else v


def draw(rng):
    op = rng.choice(["linear", "linear", "norm", "norm gradient", "rotary"])
    if op == "linear":
        m = _log(rng, 1, 32760)
        k, n = (_maybe_round(rng, _log(rng, 256, 13824), 64) for _ in range(2))
        c = _linear("", m, k, n, x=rng.choice(["bf16", "bf16", "f16", "f32"]), y=rng.choice(["bf16", "bf16", "f16", "f32"]),
                    bias=rng.random() < 0.7, act=rng.choice(["none", "none", "gelu_tanh", "gelu_erf"]))
    elif op == "rotary":
        d = rng.choice([32, 64, 72, 80, 96, 128, 128, 256])
        r = d if rng.random() < 0.6 else d // 2
        hq = _log(rng, 1, 48)
        hk = rng.choice([h for h in range(1, hq + 1) if hq % h == 0])
        b = _log(rng, 1, 16)
        t = _log(rng, 1, min(32760, max(2, 32760 * 80 * 128 // (b * (hq + hk) * d))))
        c = _rotary("", b, t, hq, hk, d, r, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]),
                    layout=rng.choice(["half", "interleaved"]), inverse=rng.random() < 0.4,
                    table=rng.choice([0, 0, t + rng.randrange(1, 60000)]))
    else:
        d = _maybe_round(rng, _log(rng, 64, 16384), 64)
        m = _log(rng, 1, min(32760, 32760 * 5120 // d))
        rows = m if rng.random() < 0.4 else max(1, m // rng.randrange(1, 9))
        t = rng.choice(["bf16", "bf16", "f16", "f32"])
        branch = rng.random() < 0.8
        c = _norm("", m, d, rows, t=t, p=rng.choice(["f32", t]), backward=op != "norm",
                  post=rng.choice(["none", "rms", "layer"]) if branch else "none", post_affine=branch and rng.random() < 0.5,
                  pre=rng.choice(["rms", "layer"]), pre_affine=rng.random() < 0.6, branch=branch,
                  gate=branch and rng.random() < 0.8, modulate=rng.random() < 0.8,
                  res_scale=rng.choice([1.0, 1.0, 0.5]))
    del c["name"]
    return c


# ---------------------------------------------------------------- what a program has in hand

def _groups(v, size):
    return -(-v // size)


def _blocks(v):
    return _groups(v, BLOCK)


def _over_blocks(scale, rows, cols):
    """[rows, cols] of the scale that each element's 128 x 128 block has."""
    return scale.repeat_interleave(BLOCK, 0)[:rows].repeat_interleave(BLOCK, 1)[:, :cols]


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=DEV) * std

    op = case["op"]
    if op == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        x = normal(m, k)
        x[:, torch.randint(0, k, (max(1, k // 1000),), generator=g, device=DEV)] *= 50.0  # outlier channels
        w = normal(n, k, std=0.02)
        nb, kb = _blocks(n), _blocks(k)
        w_pad = torch.nn.functional.pad(w, (0, kb * BLOCK - k, 0, nb * BLOCK - n))
        amax = w_pad.view(nb, BLOCK, kb, BLOCK).abs().amax((1, 3))
        scale = amax.clamp_min(AMAX_FLOOR) / E4M3_MAX
        # codes with rows that start on 16 bytes, as a loader lays them out
        codes = torch.zeros(n, -(-k // 16) * 16, device=DEV, dtype=torch.float8_e4m3fn)
        codes[:, :k] = (w / _over_blocks(scale, n, k)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        return {"case": case, "x": x.to(TYPES[case["x"]]), "w": codes[:, :k], "w_scale": scale,
                "bias": normal(n, std=0.01) if case["bias"] else None,
                "out": torch.empty(m, n, device=DEV, dtype=TYPES[case["y"]])}
    if op == "norm":
        m, d, t, p = case["m"], case["d"], TYPES[case["t"]], TYPES[case["p"]]
        batches = _groups(m, case["rows"])
        s = {"case": case, "x": (normal(m, d) + 0.2 * normal(1, d)).to(t)}
        if case["branch"]:
            s["y"] = normal(m, d, std=0.7).to(t)
        # gate, shift and scale are columns of one modulation output, as the conditioning layer writes them
        ada = normal(batches, 3 * d, std=0.3).to(p)
        if case["gate"]:
            s["gate"] = ada[:, :d]
        if case["modulate"]:
            s["shift"], s["scale"] = ada[:, d:2 * d], ada[:, 2 * d:]
        for side in ("post", "pre"):
            if case[side + "_affine"]:
                s[side + "_weight"] = (1.0 + normal(d, std=0.1)).to(p)
                if case[side] == "layer":
                    s[side + "_bias"] = normal(d, std=0.05).to(p)
        if case["backward"]:
            s["dh"], s["dn"] = normal(m, d, std=0.1).to(t), normal(m, d, std=0.1).to(t)
        else:
            s["out_h"], s["out_n"] = torch.empty(m, d, device=DEV, dtype=t), torch.empty(m, d, device=DEV, dtype=t)
        return s
    b, t, hq, hk, d, r = (case[v] for v in ("b", "t", "hq", "hk", "d", "r"))
    qkv = normal(b, t, hq + 2 * hk, d).to(TYPES[case["dtype"]])  # one projection's output
    rows = case["table"] or t
    freq = 10000.0 ** (-torch.arange(r // 2, device=DEV, dtype=torch.float64) * 2 / r)
    angle = torch.arange(rows, device=DEV, dtype=torch.float64)[:, None] * freq
    positions = None
    if case["table"]:  # each sequence's tokens follow each other, from somewhere in the context
        start = torch.randint(0, rows - t + 1, (b, 1), generator=g, device=DEV)
        positions = start + torch.arange(t, device=DEV)
    return {"case": case, "q": qkv[:, :, :hq], "k": qkv[:, :, hq:hq + hk], "cos": angle.cos().float(),
            "sin": angle.sin().float(), "positions": positions,
            "out_q": torch.empty(b, t, hq, d, device=DEV, dtype=qkv.dtype),
            "out_k": torch.empty(b, t, hk, d, device=DEV, dtype=qkv.dtype)}


# ---------------------------------------------------------------- one pass

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    from int8_hadamard_rotated_convrot_gb300 import block

    c = s["case"]
    if c["op"] == "linear":
        act = {"none": block.ACT_NONE, "gelu_erf": block.ACT_GELU_ERF, "gelu_tanh": block.ACT_GELU_TANH}[c["act"]]
        w = block.Fp8Weights(s["w"], s["w_scale"])
        return block.convrot_fp8_pack_linear(s["x"], w, s["bias"], act, out=s["out"])
    if c["op"] == "rotary":
        layout = block.ROTARY_HALF if c["layout"] == "half" else block.ROTARY_INTERLEAVED
        return block.convrot_rotary(s["q"], s["k"], s["cos"], s["sin"], s["positions"], layout=layout,
                                    inverse=c["inverse"], out_q=s["out_q"], out_k=s["out_k"])
    kinds = {"none": block.NORM_NONE, "rms": block.NORM_RMS, "layer": block.NORM_LAYER}
    get = s.get
    if not c["backward"]:
        return block.convrot_gated_norm(
            s["x"], get("y"), gate=get("gate"), scale=get("scale"), shift=get("shift"), rows_per_batch=c["rows"],
            res_scale=c["res_scale"], post=kinds[c["post"]], post_weight=get("post_weight"),
            post_bias=get("post_bias"), pre=kinds[c["pre"]], pre_weight=get("pre_weight"), pre_bias=get("pre_bias"),
            eps=EPS, out_h=s["out_h"], out_n=s["out_n"])
    grads = block.convrot_gated_norm_backward(
        s["x"], get("y"), s["dh"], s["dn"], gate=get("gate"), scale=get("scale"), shift=get("shift"),
        rows_per_batch=c["rows"], res_scale=c["res_scale"], post=kinds[c["post"]], post_weight=get("post_weight"),
        post_bias=get("post_bias"), pre=kinds[c["pre"]], pre_weight=get("pre_weight"), pre_bias=get("pre_bias"),
        eps=EPS)
    return {name: v for name, v in grads.items() if v is not None}


def _run_plain(s):
    c = s["case"]
    if c["op"] == "linear":
        return _plain_linear(s)
    if c["op"] == "rotary":
        return tuple(_plain_rotary(s, s[v]) for v in ("q", "k"))
    return _plain_norm_gradient(s) if c["backward"] else _plain_norm(s)


def _plain_linear(s):
    c = s["case"]
    m, k, n, kb = c["m"], c["k"], c["n"], _blocks(c["k"])
    x = torch.nn.functional.pad(s["x"].float(), (0, kb * BLOCK - k)).view(m, kb, BLOCK)
    amax = x.abs().amax(2, keepdim=True).clamp_min(AMAX_FLOOR)
    codes = (x * (E4M3_MAX / amax)).to(torch.float8_e4m3fn)
    x = (codes.float() * (amax / E4M3_MAX)).view(m, kb * BLOCK)[:, :k]
    y = x @ (s["w"].float() * _over_blocks(s["w_scale"], n, k)).t()
    if s["bias"] is not None:
        y = y + s["bias"]
    if c["act"] == "gelu_tanh":
        y = 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    elif c["act"] == "gelu_erf":
        y = 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    return y.to(TYPES[c["y"]])


def _rows_of(p, s):
    """Each sample's vector for each of its rows, in 32 bits."""
    c = s["case"]
    return p.float().repeat_interleave(c["rows"], 0)[:c["m"]]


def _plain_hat(v, kind):
    """(v normalized without weights, 1 / its standard deviation)"""
    if kind == "none":
        return v, None
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    inv = torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)
    return v * inv, inv


def _plain_affine(v, s, side):
    if side + "_weight" in s:
        v = v * s[side + "_weight"].float()
    if side + "_bias" in s:
        v = v + s[side + "_bias"].float()
    return v


def _plain_norm(s):
    c = s["case"]
    h = c["res_scale"] * s["x"].float()
    if "y" in s:
        u = _plain_affine(_plain_hat(s["y"].float(), c["post"])[0], s, "post")
        h = h + (_rows_of(s["gate"], s) * u if "gate" in s else u)
    n = _plain_affine(_plain_hat(h, c["pre"])[0], s, "pre")
    if "scale" in s:
        n = n * (1 + _rows_of(s["scale"], s)) + _rows_of(s["shift"], s)
    t = TYPES[c["t"]]
    return h.to(t), n.to(t)


def _plain_hat_gradient(g, hat, inv, kind):
    if kind == "none":
        return g
    d = g - hat * (g * hat).mean(1, keepdim=True)
    if kind == "layer":
        d = d - g.mean(1, keepdim=True)
    return d * inv


def _by_sample(v, s):
    """Sums over each sample's rows; the last sample may be shorter."""
    c = s["case"]
    batches = _groups(c["m"], c["rows"])
    v = torch.nn.functional.pad(v, (0, 0, 0, batches * c["rows"] - c["m"]))
    return v.view(batches, c["rows"], c["d"]).sum(1)


def _plain_norm_gradient(s):
    c, out = s["case"], {}
    t = TYPES[c["t"]]
    dn = s["dn"].float()
    hat, inv = _plain_hat(s["x"].float(), c["pre"])  # x is the forward pass's h here
    g = dn * (1 + _rows_of(s["scale"], s)) if "scale" in s else dn
    if "scale" in s:
        out["dscale"] = _by_sample(dn * _plain_affine(hat, s, "pre"), s)
        out["dshift"] = _by_sample(dn, s)
    if "pre_weight" in s:
        out["dpre_weight"] = (g * hat).sum(0)
    if "pre_bias" in s:
        out["dpre_bias"] = g.sum(0)
    if "pre_weight" in s:
        g = g * s["pre_weight"].float()
    dh = _plain_hat_gradient(g, hat, inv, c["pre"]) + s["dh"].float()
    out["dx"] = (c["res_scale"] * dh).to(t)
    if "y" in s:
        hat, inv = _plain_hat(s["y"].float(), c["post"])
        g = dh
        if "gate" in s:
            out["dgate"] = _by_sample(dh * _plain_affine(hat, s, "post"), s)
            g = dh * _rows_of(s["gate"], s)
        if "post_weight" in s:
            out["dpost_weight"] = (g * hat).sum(0)
        if "post_bias" in s:
            out["dpost_bias"] = g.sum(0)
        if "post_weight" in s:
            g = g * s["post_weight"].float()
        out["dy"] = _plain_hat_gradient(g, hat, inv, c["post"]).to(t)
    return out


def _plain_rotary(s, v):
    c = s["case"]
    r, x = c["r"], v.float()
    cos, sin = (s[a][s["positions"]] if s["positions"] is not None else s[a][None] for a in ("cos", "sin"))
    cos, sin = cos[:, :, None], (-sin if c["inverse"] else sin)[:, :, None]
    out = x.clone()
    a, b = (slice(0, r // 2), slice(r // 2, r)) if c["layout"] == "half" else (slice(0, r, 2), slice(1, r, 2))
    out[..., a] = x[..., a] * cos - x[..., b] * sin
    out[..., b] = x[..., b] * cos + x[..., a] * sin
    return out.to(v.dtype)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"] == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        return {"bytes": m * k * SIZE[case["x"]] + n * k + _blocks(n) * _blocks(k) * 4 + m * n * SIZE[case["y"]]
                + 4 * n * case["bias"], "flops": 2 * m * n * k}
    if case["op"] == "rotary":
        rows = case["b"] * case["t"]
        values = rows * (case["hq"] + case["hk"]) * case["d"]
        table = rows * (case["r"] * 4 + 8) if case["table"] else case["t"] * case["r"] * 4
        return {"bytes": 2 * values * SIZE[case["dtype"]] + table, "flops": 3 * values}
    values, batches = case["m"] * case["d"], _groups(case["m"], case["rows"])
    # forward: x (and y) in, h and n out; backward: h, dh, dn (and y) in, dx (and dy) out
    tensors = (4 + 2 * case["branch"]) if case["backward"] else (3 + case["branch"])
    weights = sum((2 if case[side] == "layer" else 1) * case[side + "_affine"] for side in ("post", "pre"))
    vectors = batches * (case["gate"] + 2 * case["modulate"]) + weights  # each read, and its gradient written in f32
    per_vector = SIZE[case["p"]] + 4 * case["backward"]
    return {"bytes": values * SIZE[case["t"]] * tensors + vectors * case["d"] * per_vector,
            "flops": values * (30 if case["backward"] else 12)}


# ---------------------------------------------------------------- the definitions, in 64 bits

def _e4m3(v):
    """The nearest e4m3 value, ties to the even code: three bits below the leading one, none below 2^-9."""
    exponent = torch.floor(torch.log2(v.abs().clamp_min(2.0**-6)))
    step = torch.exp2(exponent - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def exact(case, seed):
    s = prepare(case, seed)
    wide = {name: v.double() for name, v in s.items() if isinstance(v, torch.Tensor) and name != "positions"}
    if case["op"] == "linear":
        return _exact_linear(case, wide)
    if case["op"] == "rotary":
        return _exact_rotary(case, wide, s["positions"])
    return _exact_norm_gradient(case, wide) if case["backward"] else _exact_norm(case, wide)


def _exact_linear(c, s):
    # an x code is the e4m3 value nearest to x over (the block's largest magnitude / 448)
    k = c["k"]
    x, top = s["x"], torch.zeros(c["m"], _blocks(k), device=DEV, dtype=torch.float64)
    which = (torch.arange(k, device=DEV) // BLOCK)
    top.scatter_reduce_(1, which.expand(c["m"], k), x.abs(), "amax")
    unit = (top.clamp_min(AMAX_FLOOR) / E4M3_MAX)[:, which]
    x = _e4m3(x / unit) * unit
    del unit
    rows = torch.arange(c["n"], device=DEV) // BLOCK
    y = torch.mm(x, (s["w"] * s["w_scale"][rows][:, which]).T)
    if "bias" in s:
        y += s["bias"]
    if c["act"] == "gelu_erf":
        y *= torch.special.ndtr(y)
    elif c["act"] == "gelu_tanh":
        y *= torch.sigmoid(math.sqrt(8 / math.pi) * (y + 0.044715 * y**3))
    return y


def _exact_sample(c):
    return torch.arange(c["m"], device=DEV) // c["rows"]


def _exact_stats(v, kind):
    mean = v.mean(1, keepdim=True) if kind == "layer" else torch.zeros(v.shape[0], 1, device=DEV, dtype=v.dtype)
    spread = ((v - mean) ** 2).sum(1, keepdim=True) / v.shape[1] + EPS
    return mean, 1 / spread.sqrt()


def _exact_norm_of(c, s, v, side):
    if c[side] != "none":
        mean, inv = _exact_stats(v, c[side])
        v = (v - mean) * inv
    return v * s.get(side + "_weight", 1.0) + s.get(side + "_bias", 0.0)


def _exact_norm(c, s):
    which = _exact_sample(c)
    h = c["res_scale"] * s["x"]
    if c["branch"]:
        u = _exact_norm_of(c, s, s["y"], "post")
        h = h + (u * s["gate"][which] if c["gate"] else u)
    n = _exact_norm_of(c, s, h, "pre")
    if c["modulate"]:
        n = n + n * s["scale"][which] + s["shift"][which]
    return h, n


def _exact_norm_gradient(c, s):
    # reverse-mode differentiation of the definition, in 64 bits
    names = [n for n in ("y", "gate", "scale", "shift", "pre_weight", "pre_bias", "post_weight", "post_bias") if n in s]
    which = _exact_sample(c)
    v = {n: s[n].clone().requires_grad_() for n in names}
    h = s["x"].clone().requires_grad_()
    n = _exact_norm_of(c, v, h, "pre")
    if c["modulate"]:
        n = n + n * v["scale"][which] + v["shift"][which]
    first = ["scale", "shift", "pre_weight", "pre_bias"]
    wrt = [a for a in first if a in v]
    got = torch.autograd.grad(n, [h] + [v[a] for a in wrt], s["dn"])
    dh = got[0] + s["dh"]
    out = {"d" + a: q for a, q in zip(wrt, got[1:])}
    out["dx"] = c["res_scale"] * dh
    if c["branch"]:
        u = _exact_norm_of(c, v, v["y"], "post")
        if c["gate"]:
            u = u * v["gate"][which]
        wrt = [a for a in ("y", "gate", "post_weight", "post_bias") if a in v]
        out |= {"d" + a: q for a, q in zip(wrt, torch.autograd.grad(u, [v[a] for a in wrt], dh))}
    return out


def _exact_rotary(c, s, positions):
    t, r = c["t"], c["r"]
    at = positions if positions is not None else torch.arange(t, device=DEV).expand(c["b"], t)
    turn = torch.complex(s["cos"], -s["sin"] if c["inverse"] else s["sin"])[at][:, :, None]

    def rotated(x):
        head = x[..., :r]
        pairs = head.unflatten(-1, (2, r // 2)).transpose(-1, -2) if c["layout"] == "half" else head.unflatten(-1, (r // 2, 2))
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        z = z.transpose(-1, -2).flatten(-2) if c["layout"] == "half" else z.flatten(-2)
        return torch.cat([z, x[..., r:]], -1)

    return rotated(s["q"]), rotated(s["k"])
