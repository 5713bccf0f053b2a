"""Measured cases of the operators that stand around the int8 linear layers.

Three families, each in the forms a diffusion transformer or its image decoder
uses beside a W8A8 layer:

  rotary       rotary positions on the heads that a projection wrote: one or
               several position axes, interleaved or half layout, all or part
               of the head, frequencies scaled for long contexts, and the
               gradient (the transposed rotation);
  group_norm   group normalization with SiLU over channels-last tensors: the
               output, the output as int8 rows with their scales (the operand
               of the int8 layer that follows), and the gradient;
  input_grad   the gradient of the W8A8 layer with respect to its input, an
               8-bit product against the stored int8 weights: the gradient rows
               times the channels' scales, quantized per token, times Wq.

`run` computes a case either in plain 32-bit torch operations or, where `own`
is set, through the package's entry points.  `exact` gives the same outputs
from the definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one new token of a text encoder: 32 query heads and 8 key heads
        {"name": "rotary token", "op": "rotary", "batch": 1, "tokens": 1, "heads": 32, "kv_heads": 8, "dim": 128, "rot": 128,
         "layout": "half", "axes": 1, "scaled": False, "far": 4096, "storage": "tokens", "grad": False, "dtype": "bf16"},
        # a transformer block's q and k beside v, 4096 image and 256 text tokens,
        # positions along three axes
        {"name": "rotary image", "op": "rotary", "batch": 1, "tokens": 4352, "heads": 32, "kv_heads": 32, "dim": 128, "rot": 128,
         "layout": "interleaved", "axes": 3, "scaled": False, "far": 64, "storage": "qkv", "grad": False, "dtype": "bf16"},
        # a long prompt at far positions, frequencies scaled for a context 32
        # times the trained one
        {"name": "rotary long", "op": "rotary", "batch": 1, "tokens": 16384, "heads": 32, "kv_heads": 8, "dim": 128, "rot": 128,
         "layout": "half", "axes": 1, "scaled": True, "far": 1000000, "storage": "tokens", "grad": False, "dtype": "fp16"},
        # the gradient for a padded batch stored head by head, a quarter of
        # each head rotated
        {"name": "rotary grad", "op": "rotary", "batch": 3, "tokens": 1009, "heads": 12, "kv_heads": 4, "dim": 256, "rot": 64,
         "layout": "half", "axes": 1, "scaled": False, "far": 8192, "storage": "heads", "grad": True, "dtype": "fp32"},
        # the innermost level of a denoiser: 8 x 8 pixels, conditional and
        # unconditional branch together
        {"name": "norm 8x8", "op": "norm", "batch": 2, "pixels": 64, "channels": 1280, "groups": 32, "silu": True, "stats": False, "dtype": "bf16"},
        # a training step's forward pass on an image of odd sides, statistics kept
        {"name": "norm 63x65", "op": "norm", "batch": 2, "pixels": 63 * 65, "channels": 640, "groups": 32, "silu": True, "stats": True, "dtype": "fp16"},
        # the last level of an image decoder: 1024 x 1024 pixels
        {"name": "norm 1024x1024", "op": "norm", "batch": 1, "pixels": 1024 * 1024, "channels": 128, "groups": 32, "silu": True, "stats": False, "dtype": "bf16"},
        # the norm ahead of an int8 projection: int8 rows and their scales
        {"name": "norm quant", "op": "norm_quant", "batch": 2, "pixels": 4096, "channels": 1280, "groups": 32, "silu": False, "dtype": "bf16"},
        # the same block's gradients
        {"name": "norm grad", "op": "norm_grad", "batch": 4, "pixels": 4096, "channels": 512, "groups": 32, "silu": True, "dtype": "bf16"},
        # gradients of a conditioning layer at 16 rows
        {"name": "input grad 16", "op": "input_grad", "rows": 16, "n": 12288, "k": 4096},
        # ... of a short sequence's projection
        {"name": "input grad 512", "op": "input_grad", "rows": 512, "n": 4096, "k": 12288},
        # ... of an image's up projection, 4096 image and 256 text tokens
        {"name": "input grad 4352", "op": "input_grad", "rows": 4352, "n": 12288, "k": 4096},
    ]


def spread(rng, low, high):
    """A whole number between low and high, spread over the logarithm."""
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    op = rng.choice(["rotary", "norm", "norm_quant", "norm_grad", "input_grad"])
    if op == "rotary":
        dim = rng.choice([64, 80, 96, 128, 256])
        heads = rng.choice([1, 3, 8, 12, 24, 32])
        axes = rng.choice([1, 1, 3])
        rot = dim if axes == 3 else rng.choice([dim, dim // 2, 32])
        batch = rng.choice([1, 1, 2, 3])
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        storage = rng.choice(["tokens", "qkv", "heads"])
        kv = heads if storage == "qkv" else rng.choice([h for h in (1, 2, 3, 4, 8, 12, 24, 32) if h <= heads and heads % h == 0])
        most = 16384 * 40 * 128 // (batch * (heads + kv) * dim * (2 if dtype == "fp32" else 1))
        return {"op": op, "batch": batch, "tokens": spread(rng, 1, max(1, min(20000, most))), "heads": heads, "kv_heads": kv, "dim": dim,
                "rot": rot, "layout": rng.choice(["half", "interleaved"]), "axes": axes, "scaled": axes == 1 and rng.random() < 0.5,
                "far": spread(rng, 64, 1000000) if axes == 1 else 64, "storage": storage, "grad": rng.random() < 0.3, "dtype": dtype}
    if op == "input_grad":
        n, k = 16 * spread(rng, 32, 768), 16 * spread(rng, 32, 768)
        most = 4352 * 12288 * 4096 // (n * k)
        return {"op": op, "rows": spread(rng, 1, max(1, min(8704, most))), "n": n - 8 * rng.randrange(2), "k": k}
    groups = rng.choice([1, 8, 32, 32, 32])
    channels = groups * rng.choice([8, 16, 24, 40]) if groups > 8 else 8 * spread(rng, 8, 256)
    batch = rng.choice([1, 2, 2, 4, 7])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp16", "fp32"])
    most = 1024 * 1024 * 128 // (batch * channels * (2 if dtype == "fp32" else 1) * (2 if op == "norm_grad" else 1))
    case = {"op": op, "batch": batch, "pixels": spread(rng, 1, max(1, most)), "channels": channels, "groups": groups,
            "silu": rng.random() < 0.6, "dtype": dtype}
    if op == "norm":
        case["stats"] = rng.random() < 0.5
    if op == "norm_quant":  # the int8 layer takes bf16 activations and rows of a multiple of 16
        case["dtype"], case["channels"] = "bf16", channels if channels % 16 == 0 else 2 * channels
        case["pixels"] = max(1, case["pixels"] // 2)
    return case


# ---------------------------------------------------------------- inputs

def frequencies(case):
    """Radians a position of each pair, and the factor on the rotated values.
    Scaled: a context 32 times the trained 4096 positions, pairs that turn more
    than 32 times over it kept, those that turn less than once interpolated, a
    ramp between, and the values raised by 0.1 ln 32 + 1."""
    pairs, base = case["rot"] // 2, 10000.0 if case["axes"] == 3 else 1000000.0
    if case["axes"] == 3:  # an eighth of the pairs for the first axis, the rest shared by the two others
        first = pairs // 8
        sizes = [first, (pairs - first) // 2, pairs - first - (pairs - first) // 2]
        freq = [base ** (-i / size) for size in sizes for i in range(size)]
        axis = [a for a, size in enumerate(sizes) for _ in range(size)]
        return freq, axis, 1.0
    freq = [base ** (-i / pairs) for i in range(pairs)]
    if not case["scaled"]:
        return freq, [0] * pairs, 1.0
    factor, trained = 32.0, 4096
    at = [pairs * math.log(trained / (turns * 2 * math.pi)) / math.log(base) for turns in (32.0, 1.0)]
    low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), pairs - 1)
    ramp = [min(1.0, max(0.0, (i - low) / max(high - low, 0.001))) for i in range(pairs)]
    return [f * (1 - r) + f / factor * r for f, r in zip(freq, ramp)], [0] * pairs, 0.1 * math.log(factor) + 1.0


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    if case["op"] == "rotary":
        b, t, h, kv, d = case["batch"], case["tokens"], case["heads"], case["kv_heads"], case["dim"]
        dtype = DTYPES[case["dtype"]]
        if case["storage"] == "qkv":  # views of the projection's output, v beside them
            both = normal(b, t, h + 2 * kv, d).to(dtype)
            q, k = both[:, :, :h], both[:, :, h:h + kv]
        elif case["storage"] == "heads":
            q, k = normal(b, h, t, d).to(dtype).transpose(1, 2), normal(b, kv, t, d).to(dtype).transpose(1, 2)
        else:
            q, k = normal(b, t, h, d).to(dtype), normal(b, t, kv, d).to(dtype)
        if case["axes"] == 1:
            start = torch.randint(0, case["far"], (b, 1), generator=gen, device="cuda")
            positions = start + torch.arange(t, device="cuda")
        else:
            positions = torch.randint(-case["far"], case["far"], (b, t, case["axes"]), generator=gen, device="cuda")
        freq, axis, scale = frequencies(case)
        freq, axis = torch.tensor(freq, dtype=torch.float64), torch.tensor(axis, dtype=torch.int32)
        return {"case": case, "q": q, "k": k, "positions": positions, "scale": scale, "freq": freq, "axis": axis,
                "freq_there": freq.cuda(), "axis_there": axis.cuda().long()}

    if case["op"] == "input_grad":
        m, n, k = case["rows"], case["n"], case["k"]
        dy = normal(m, n) * 1e-3
        dy[:, torch.randperm(n, generator=gen, device="cuda")[: max(1, n // 100)]] *= 8.0  # a few channels carry more
        codes = (normal(n, k) * 32.0).round().clamp(-127, 127).to(torch.int8)
        scales = (0.5 + torch.rand(n, generator=gen, device="cuda")) * 1e-3
        return {"case": case, "dy": dy.bfloat16(), "codes": codes, "scales": scales}

    b, s, c, g = case["batch"], case["pixels"], case["channels"], case["groups"]
    dtype = DTYPES[case["dtype"]]
    x = (normal(b, s, c) * (0.5 + torch.rand(c, generator=gen, device="cuda")) + normal(c) + 0.5).to(dtype)
    state = {"case": case, "x": x, "weight": (1.0 + 0.2 * normal(c)).to(dtype), "bias": (0.2 * normal(c)).to(dtype), "eps": 1e-5}
    if case["op"] == "norm_grad":  # what the forward pass left
        state["dy"] = normal(b, s, c).to(dtype)
        xs = x.view(b, s, g, c // g).float()
        mean = xs.mean((1, 3), dtype=torch.float64)
        square = torch.zeros_like(mean)
        for i in range(b):
            square[i] = (xs[i] - mean[i].float()[:, None]).square_().mean((0, 2), dtype=torch.float64)
        state["mean"], state["rstd"] = mean.float(), (square + 1e-5).rsqrt().float()
    return state


# ---------------------------------------------------------------- plain forms

def turned(x, cos, sin, case):
    """The first `rot` values of each head rotated, the rest as they are."""
    rot, half = case["rot"], case["rot"] // 2
    x32 = x.float()
    if case["layout"] == "half":
        a, b = x32[..., :half], x32[..., half:rot]
    else:
        a, b = x32[..., 0:rot:2], x32[..., 1:rot:2]
    first, second = a * cos - b * sin, a * sin + b * cos
    both = torch.cat((first, second), -1) if case["layout"] == "half" else torch.stack((first, second), -1).flatten(-2)
    return torch.cat((both, x32[..., rot:]), -1).to(x.dtype)


def plain_rotary(s):
    case = s["case"]
    positions = s["positions"]
    at = positions[..., None] if case["axes"] == 1 else positions[..., s["axis_there"]]
    angle = at.double() * s["freq_there"]
    cos = (angle.cos() * s["scale"]).float()[:, :, None]
    sin = (angle.sin() * s["scale"]).float()[:, :, None]
    if case["grad"]:
        sin = -sin
    return {"q": turned(s["q"], cos, sin, case), "k": turned(s["k"], cos, sin, case)}


def plain_norm(s):
    case = s["case"]
    b, p, c, g = case["batch"], case["pixels"], case["channels"], case["groups"]
    x = s["x"].float().view(b, p, g, c // g)
    mean = x.mean((1, 3), keepdim=True)
    x = x - mean
    rstd = (x.square().mean((1, 3), keepdim=True) + s["eps"]).rsqrt()
    z = (x * rstd).view(b, p, c) * s["weight"].float() + s["bias"].float()
    return (z / (1 + (-z).exp()) if case["silu"] else z), mean.view(b, g), rstd.view(b, g)


def plain_norm_grad(s):
    case = s["case"]
    b, p, c, g = case["batch"], case["pixels"], case["channels"], case["groups"]
    xhat = (s["x"].float().view(b, p, g, c // g) - s["mean"].view(b, 1, g, 1)) * s["rstd"].view(b, 1, g, 1)
    xhat = xhat.view(b, p, c)
    dz = s["dy"].float()
    if case["silu"]:
        z = xhat * s["weight"].float() + s["bias"].float()
        sig = 1 / (1 + (-z).exp())
        dz = dz * (sig * (1 + z * (1 - sig)))
    dweight, dbias = (dz * xhat).sum((0, 1)), dz.sum((0, 1))
    dxhat = (dz * s["weight"].float()).view(b, p, g, c // g)
    xhat = xhat.view(b, p, g, c // g)
    dx = dxhat - dxhat.mean((1, 3), keepdim=True) - xhat * (dxhat * xhat).mean((1, 3), keepdim=True)
    dx = (dx * s["rstd"].view(b, 1, g, 1)).view(b, p, c)
    return {"dx": dx.to(s["x"].dtype), "dweight": dweight, "dbias": dbias}


def plain_rows(y):
    """Symmetric int8 rows: codes and the scales they stand on."""
    scale = y.abs().amax(-1) / 127
    return (y / scale.clamp_min(1e-38)[..., None]).round().clamp(-127, 127), scale


def plain_input_grad(s):
    codes, scale = plain_rows(s["dy"].float() * s["scales"])
    return {"dx": ((codes @ s["codes"].float()) * scale[:, None]).bfloat16()}


# ---------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import w8a8_int8_dynamic_token_b200 as w8a8

        if op == "rotary":
            q, k = w8a8.rotary(state["q"], state["positions"], state["freq"], k=state["k"], layout=case["layout"],
                               axis=state["axis"] if case["axes"] > 1 else None, scale=state["scale"], backward=case["grad"])
            return {"q": q, "k": k}
        if op == "norm":
            if case["stats"]:
                y, mean, rstd = w8a8.group_norm(state["x"], case["groups"], state["weight"], state["bias"], eps=state["eps"],
                                                activation="silu" if case["silu"] else None, return_stats=True)
                return {"y": y, "mean": mean, "rstd": rstd}
            return {"y": w8a8.group_norm(state["x"], case["groups"], state["weight"], state["bias"], eps=state["eps"],
                                         activation="silu" if case["silu"] else None)}
        if op == "norm_quant":
            codes, scales = w8a8.group_norm_quant(state["x"], case["groups"], state["weight"], state["bias"], eps=state["eps"],
                                                  activation="silu" if case["silu"] else None)
            values = torch.empty(codes.shape, dtype=torch.bfloat16, device=codes.device)
            return {"values": torch.mul(codes, scales[:, None], out=values), "scales": scales}
        if op == "norm_grad":
            dx, dweight, dbias = w8a8.group_norm_backward(state["dy"], state["x"], state["mean"], state["rstd"], state["weight"],
                                                          state["bias"], activation="silu" if case["silu"] else None)
            return {"dx": dx, "dweight": dweight, "dbias": dbias}
        return {"dx": w8a8.linear_input_grad(state["dy"], state["codes"], state["scales"])}

    if op == "rotary":
        return plain_rotary(state)
    if op == "norm":
        y, mean, rstd = plain_norm(state)
        y = y.to(state["x"].dtype)
        return {"y": y, "mean": mean, "rstd": rstd} if case["stats"] else {"y": y}
    if op == "norm_quant":
        y, _, _ = plain_norm(state)
        codes, scale = plain_rows(y.view(-1, case["channels"]))
        return {"values": (codes * scale[:, None]).bfloat16(), "scales": scale}
    if op == "norm_grad":
        return plain_norm_grad(state)
    return plain_input_grad(state)


# ---------------------------------------------------------------- cost and reference

def work(case):
    if case["op"] == "rotary":
        size = 4 if case["dtype"] == "fp32" else 2
        values = case["batch"] * case["tokens"] * (case["heads"] + case["kv_heads"]) * case["dim"]
        rotated = case["batch"] * case["tokens"] * (case["heads"] + case["kv_heads"]) * case["rot"]
        return {"bytes": 2 * size * values + 8 * case["batch"] * case["tokens"] * case["axes"], "flops": 3 * rotated}
    if case["op"] == "input_grad":
        m, n, k = case["rows"], case["n"], case["k"]
        return {"bytes": 2 * m * n + n * k + 4 * n + 2 * m * k, "flops": 2 * m * n * k}
    size = 4 if case["dtype"] == "fp32" else 2
    values = case["batch"] * case["pixels"] * case["channels"]
    if case["op"] == "norm":
        return {"bytes": 2 * size * values, "flops": (8 + 5 * case["silu"]) * values}
    if case["op"] == "norm_quant":  # codes of one byte and a scale a row
        return {"bytes": (size + 1) * values + 4 * case["batch"] * case["pixels"], "flops": (11 + 5 * case["silu"]) * values}
    return {"bytes": 3 * size * values + 8 * case["channels"], "flops": (14 + 10 * case["silu"]) * values}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        at = s["positions"].double()
        at = at[..., None] if case["axes"] == 1 else at.index_select(-1, s["axis_there"])
        turn = at * s["freq_there"]
        turn = torch.polar(torch.full_like(turn, s["scale"]), -turn if case["grad"] else turn).unsqueeze(2)

        def whole(x):
            wide = x.double().contiguous()
            head = wide[..., : case["rot"]]
            if case["layout"] == "half":
                pairs = head.unflatten(-1, (2, -1)).transpose(-1, -2)
            else:
                pairs = head.unflatten(-1, (-1, 2))
            out = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
            out = out.transpose(-1, -2) if case["layout"] == "half" else out
            wide[..., : case["rot"]] = out.flatten(-2)
            return wide

        return {"q": whole(s["q"]), "k": whole(s["k"])}

    if case["op"] == "input_grad":
        rows = s["dy"].double() * s["scales"].double()
        step = rows.abs().max(1, keepdim=True).values / 127
        codes = torch.where(step > 0, torch.round(rows / step.clamp_min(1e-300)), torch.zeros_like(rows))
        return {"dx": step * torch.mm(codes, s["codes"].double())}

    c, g = case["channels"], case["groups"]
    weight, bias = s["weight"].double(), s["bias"].double()
    outs = []
    dweight, dbias = torch.zeros_like(weight), torch.zeros_like(weight)
    for i in range(case["batch"]):  # one image at a time keeps the 64-bit copies small
        x = s["x"][i].double().view(-1, g, c // g)
        if case["op"] == "norm_grad":
            mean, rstd = s["mean"][i].double()[:, None], s["rstd"][i].double()[:, None]
        else:
            var, mean = torch.var_mean(x, (0, 2), unbiased=False)
            mean, rstd = mean[:, None], 1 / torch.sqrt(var + s["eps"])[:, None]
        unit = ((x - mean) * rstd).view(-1, c)
        z = torch.addcmul(bias, unit, weight)
        gate = torch.special.expit(z)
        if case["op"] != "norm_grad":
            outs.append((z * gate if case["silu"] else z, mean[:, 0], rstd[:, 0]))
            continue
        dz = s["dy"][i].double()
        if case["silu"]:
            dz = dz * gate * (1 + z - z * gate)
        dweight += torch.einsum("pc,pc->c", dz, unit)
        dbias += torch.einsum("pc->c", dz)
        unit, dunit = unit.view(-1, g, c // g), (dz * weight).view(-1, g, c // g)
        n = unit.shape[0] * unit.shape[2]
        inner = torch.einsum("pgc,pgc->g", dunit, unit)[:, None] / n
        outs.append(((dunit - dunit.sum((0, 2))[:, None] / n - unit * inner) * rstd).view(-1, c))
    if case["op"] == "norm_grad":
        return {"dx": torch.stack(outs), "dweight": dweight, "dbias": dbias}
    y, mean, rstd = (torch.stack(v) for v in zip(*outs))
    if case["op"] == "norm":
        return {"y": y, "mean": mean, "rstd": rstd} if case["stats"] else {"y": y}
    y = y.flatten(0, 1)
    step = y.abs().max(1, keepdim=True).values / 127
    return {"values": torch.round(y / step.clamp_min(1e-300)) * step, "scales": step[:, 0]}
