"""Layer norm and the microscaled 4-bit product: what is measured, and their plain forms.

A residual stream is added up and layer-normalised, and leaves in 16 bits, in e4m3 with one scale a row, or in
microscaled 4-bit floats: e2m1 values (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives, two a byte, the low four bits
first) with one power of two for each 32 neighbours of a row, held as its exponent plus 127 in a byte (e8m0). Such rows
meet weights in the same form. Weights and activations that are 16-bit floats are brought into that form and back, and
the norm has its gradient. `run` computes a case in plain torch operations where `own` is false, and with this
repository's kernels where it is true.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
AMAX_MIN = 2.0 ** -100  # below it a row counts as zeros: keeps the scale and its reciprocal normal numbers
EPS = 1e-5
BLOCK = 32

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}


def listed():
    return [
        # A batch of short prompts, an odd number of rows, a width that is no power of two; 16-bit output.
        {"name": "norm 1021x5000 fp16", "op": "norm", "M": 1021, "N": 5000, "type": "fp16", "out": "fp16", "residual": True},
        # Long prompts, in front of a product with 8-bit weights.
        {"name": "norm 8192x8192 e4m3", "op": "norm", "M": 8192, "N": 8192, "type": "bf16", "out": "e4m3", "residual": True},
        # The gradient at an ordinary and at a large training step; the residual stream brings a gradient of its own.
        {"name": "grad 1021x2048 fp16", "op": "grad", "M": 1021, "N": 2048, "type": "fp16", "residual": False},
        {"name": "grad 8192x8192 bf16", "op": "grad", "M": 8192, "N": 8192, "type": "bf16", "residual": True},
        # 16-bit values into 4 bits and back: a few activations, and a large layer's weights.
        {"name": "round trip 24x4128 fp16", "op": "trip", "M": 24, "K": 4128, "type": "fp16"},
        {"name": "round trip 28672x8192 bf16", "op": "trip", "M": 28672, "K": 8192, "type": "bf16"},
        # 4-bit rows and weights: one token, a batch of tokens, a ragged prompt, a long prompt.
        {"name": "mx 1x4096x4096", "op": "mx", "M": 1, "N": 4096, "K": 4096, "out": "bf16"},
        {"name": "mx 24x8192x8192", "op": "mx", "M": 24, "N": 8192, "K": 8192, "out": "fp16"},
        {"name": "mx 1000x5000x4128", "op": "mx", "M": 1000, "N": 5000, "K": 4128, "out": "bf16"},
        {"name": "mx 8192x8192x8192", "op": "mx", "M": 8192, "N": 8192, "K": 8192, "out": "bf16"},
        # Both together, as a layer runs them: the stream's sum, its norm in 4 bits, the product. One token; a prompt.
        {"name": "layer 1x4096x4096", "op": "layer", "M": 1, "N": 4096, "K": 4096, "type": "bf16"},
        {"name": "layer 500x6000x2048", "op": "layer", "M": 500, "N": 6000, "K": 2048, "type": "fp16"},
    ]


def _between(rng, low, high, step=1):
    """A multiple of `step` in [low, high], spread evenly over its logarithm."""
    v = math.exp(rng.uniform(math.log(low), math.log(high + 1)))
    return min(high // step * step, max(-(-low // step) * step, int(v) // step * step))


def draw(rng):
    op = rng.choice(["norm", "grad", "trip", "mx", "layer"])
    if op in ("norm", "grad"):
        N = _between(rng, 256, 16384, 8)
        M = _between(rng, 1, min(8192, (1 << 26) // N))
        case = {"op": op, "M": M, "N": N, "type": rng.choice(["bf16", "fp16"]), "residual": rng.random() < 0.7}
        if op == "norm":
            case["out"] = rng.choice([case["type"], "e4m3"])
        return case
    if op == "trip":
        K = _between(rng, 256, 28672, BLOCK)
        return {"op": op, "M": _between(rng, 1, min(28672, 28672 * 8192 // K)), "K": K,
                "type": rng.choice(["bf16", "fp16", "fp32"])}
    M = _between(rng, 1, 8192 if op == "mx" else 2048)
    N = _between(rng, 256, 16384, 8)
    K = _between(rng, 256, max(256, min(16384, 8192 ** 3 // (M * N))), BLOCK)
    if op == "mx":
        return {"op": op, "M": M, "N": N, "K": K, "out": rng.choice(["bf16", "fp16", "fp32"])}
    return {"op": op, "M": M, "N": N, "K": K, "type": rng.choice(["bf16", "fp16"])}


def _mx_bytes(rows, K):
    return rows * (K // 2 + K // BLOCK)


def work(case):
    M = case["M"]
    if case["op"] == "norm":
        N, t = case["N"], SIZE[case["type"]]
        b = M * N * (t + SIZE[case["out"]] + (2 * t if case["residual"] else 0)) + 2 * N * t
        return {"bytes": b + (4 * M if case["out"] == "e4m3" else 0), "flops": 8 * M * N}
    if case["op"] == "grad":
        N, t = case["N"], SIZE[case["type"]]
        return {"bytes": M * N * t * (4 if case["residual"] else 3) + N * (t + 8), "flops": 16 * M * N}
    K = case["K"]
    if case["op"] == "trip":
        # Two calls: the 4-bit form is written by one and read by the other.
        return {"bytes": 2 * M * K * SIZE[case["type"]] + 2 * _mx_bytes(M, K), "flops": 6 * M * K}
    N = case["N"]
    if case["op"] == "mx":
        return {"bytes": _mx_bytes(M, K) + _mx_bytes(N, K) + M * N * SIZE[case["out"]], "flops": 2 * M * N * K}
    t = SIZE[case["type"]]
    b = 3 * M * K * t + 2 * K * t + 2 * _mx_bytes(M, K) + _mx_bytes(N, K) + M * N * t
    return {"bytes": b, "flops": 2 * M * N * K + 8 * M * K}


# ---------------------------------------------------------------------------
# The 4-bit form in plain operations
# ---------------------------------------------------------------------------
def _powers(exponent, dtype):
    """Powers of two, exactly: pow() on the GPU rounds some of them."""
    return torch.exp2(exponent.double()).to(dtype)[:, :, None]


def _to_mx(x):
    """The rows' values in the 4-bit form, as (values of e2m1, exponents). A block's power of two is the largest one
    not above its largest magnitude, divided by 4: that magnitude becomes 4 to 8, and 6 is the most there is. Rounding
    is to nearest, ties to the even code. Powers of two alone scale the values, so every step is exact in the type
    that x is given in but the rounding to the code."""
    M, K = x.shape
    v = x.view(M, K // BLOCK, BLOCK)
    top = v.abs().amax(dim=2)
    exponent = torch.where(top > 0, torch.frexp(top).exponent.to(torch.int32) - 3, -127).clamp(-127, 127)
    q = v * _powers(-exponent, x.dtype)
    a = q.abs()
    step = 0.5 + 0.5 * (a >= 2) + (a >= 4)
    return (torch.round(a / step) * step).clamp(max=6.0).copysign(q), exponent


def _mx_values(values, exponent):
    """What the 4-bit form stands for."""
    return (values * _powers(exponent, values.dtype)).flatten(1)


def _mx_pack(values, exponent):
    """The 4-bit form as it is held: codes two a byte, and scales in rows that start at multiples of 16 bytes."""
    a = values.abs()
    code = (2 * a).clamp(max=4) + (a > 2) + (a > 3) + (a > 4) + 8 * torch.signbit(values)
    code = code.to(torch.uint8).flatten(1)
    M, blocks = exponent.shape
    scales = torch.full((M, -(-blocks // 16) * 16), 127, dtype=torch.uint8, device=exponent.device)[:, :blocks]
    scales.copy_(exponent + 127)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).view(torch.float4_e2m1fn_x2), scales.view(torch.float8_e8m0fnu)


def _mx_unpack(codes, scales):
    codes, scales = codes.view(torch.uint8), scales.view(torch.uint8)
    c = torch.stack([codes & 15, codes >> 4], dim=2).view(scales.shape[0], scales.shape[1], BLOCK)
    m = (c & 7).float()
    a = torch.where(m < 4, 0.5 * m, torch.where(m < 6, m - 2, 2 * m - 8))
    return torch.where(c > 7, -a, a), scales.to(torch.int32) - 127


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device=dev, dtype=torch.float32, generator=g)

    def loud(n):
        # Activations: a few channels are much larger than the others.
        return 1 + 10 * (torch.rand(n, device=dev, generator=g) < 0.01)

    M = case["M"]
    s = {"case": case}
    if case["op"] in ("norm", "grad", "layer"):
        t = TYPES[case["type"]]
        N = case["K"] if case["op"] == "layer" else case["N"]
        s["weight"] = (1 + 0.1 * normal(N)).to(t)
        s["bias"] = (0.1 * normal(N)).to(t)
        s["x"] = (normal(M, N) * loud(N) + 0.3 * normal(M, 1)).to(t)
        s["residual"] = normal(M, N).to(t) if case.get("residual", True) else None
        if case["op"] == "grad":
            s["dy"] = normal(M, N).to(t)
    elif case["op"] == "trip":
        s["x"] = (normal(M, case["K"]) * loud(case["K"])).to(TYPES[case["type"]])
    else:
        s["A"], s["a_scales"] = _mx_pack(*_to_mx(normal(M, case["K"]) * loud(case["K"])))
    if case["op"] in ("mx", "layer"):
        s["W"], s["w_scales"] = _mx_pack(*_to_mx(normal(case["N"], case["K"]) / math.sqrt(case["K"])))
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def _stream(s):
    """The residual stream, held in the stream's type."""
    x = s["x"]
    return x if s["residual"] is None else (x.float() + s["residual"].float()).to(x.dtype)


def _plain_norm(s, case):
    t = TYPES[case["type"]]
    h = _stream(s)
    f = h.float()
    f = f - f.mean(dim=1, keepdim=True)
    y = f * torch.rsqrt((f * f).mean(dim=1, keepdim=True) + EPS) * s["weight"].float() + s["bias"].float()
    if case["out"] == "e4m3":
        scales = y.abs().amax(dim=1).clamp_min(AMAX_MIN) / E4M3_MAX
        out = {"y": (y / scales[:, None]).to(torch.float8_e4m3fn), "scales": scales}
    else:
        out = {"y": y.to(t)}
    if s["residual"] is not None:
        out["h"] = h
    return out


def _plain_grad(s, case):
    t = TYPES[case["type"]]
    dy, w, f = s["dy"].float(), s["weight"].float(), s["x"].float()
    f = f - f.mean(dim=1, keepdim=True)
    r = torch.rsqrt((f * f).mean(dim=1, keepdim=True) + EPS)
    unit = f * r
    g = dy * w
    dx = (g - g.mean(dim=1, keepdim=True) - unit * (g * unit).mean(dim=1, keepdim=True)) * r
    if s["residual"] is not None:
        dx = dx + s["residual"].float()
    return {"dx": dx.to(t), "dweight": (dy * unit).sum(dim=0), "dbias": dy.sum(dim=0)}


def _plain_trip(s, case):
    return _mx_values(*_to_mx(s["x"].float())).to(s["x"].dtype)


def _plain_mx(s, case):
    a = _mx_values(*_mx_unpack(s["A"], s["a_scales"]))
    return (a @ _mx_values(*_mx_unpack(s["W"], s["w_scales"])).t()).to(TYPES[case["out"]])


def _plain_layer(s, case):
    h = _stream(s)
    f = h.double()  # a value next to the border between two codes goes to the one that it is nearer to
    f = f - f.mean(dim=1, keepdim=True)
    y = f * torch.rsqrt((f * f).mean(dim=1, keepdim=True) + EPS) * s["weight"].double() + s["bias"].double()
    a = _mx_values(*_to_mx(y)).float()
    return {"C": (a @ _mx_values(*_mx_unpack(s["W"], s["w_scales"])).t()).to(TYPES[case["type"]]), "h": h}


def _own_norm(s, case):
    import async_stage_tile_amd as pt
    got = pt.pipe_layernorm(s["x"], s["weight"], s["bias"], residual=s["residual"], eps=EPS, out_dtype=TYPES[case["out"]])
    names = ["y"] + (["scales"] if case["out"] == "e4m3" else []) + (["h"] if s["residual"] is not None else [])
    return dict(zip(names, got if len(names) > 1 else (got,)))


def _own_grad(s, case):
    import async_stage_tile_amd as pt
    dx, dweight, dbias = pt.pipe_layernorm_backward(s["dy"], s["x"], s["weight"], dh=s["residual"], eps=EPS)
    return {"dx": dx, "dweight": dweight, "dbias": dbias}


def _own_trip(s, case):
    import async_stage_tile_amd as pt
    codes, scales = pt.pipe_quantize_mxfp4(s["x"])
    return pt.pipe_dequantize_mxfp4(codes, scales, out_dtype=s["x"].dtype)


def _own_mx(s, case):
    import async_stage_tile_amd as pt
    return pt.pipe_gemm_mxfp4(s["A"], s["a_scales"], s["W"], s["w_scales"], out_dtype=TYPES[case["out"]])


def _own_layer(s, case):
    import async_stage_tile_amd as pt
    y, scales, h = pt.pipe_layernorm(s["x"], s["weight"], s["bias"], residual=s["residual"], eps=EPS,
                                     out_dtype=torch.float4_e2m1fn_x2)
    return {"C": pt.pipe_gemm_mxfp4(y, scales, s["W"], s["w_scales"], out_dtype=TYPES[case["type"]]), "h": h}


_PLAIN = {"norm": _plain_norm, "grad": _plain_grad, "trip": _plain_trip, "mx": _plain_mx, "layer": _plain_layer}
_OWN = {"norm": _own_norm, "grad": _own_grad, "trip": _own_trip, "mx": _own_mx, "layer": _own_layer}


def run(state):
    case = state["case"]
    return (_OWN if own else _PLAIN)[case["op"]](state, case)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _nearest(v):
    """Rows of 64-bit values, each replaced by what its 4-bit form stands for: the magnitudes' borders counted one by one
    (a border itself goes to the even one of its two codes)."""
    d = torch.float64
    b = v.unflatten(1, (-1, BLOCK))
    top = torch.maximum(b.max(dim=2, keepdim=True).values, -b.min(dim=2, keepdim=True).values)
    unit = torch.exp2(torch.floor(torch.log2(top.clamp_min(2.0 ** -125))) - 2)
    a = b.abs() / unit
    n = torch.zeros_like(a, dtype=torch.int64)
    for border, up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        n += (a >= border) if up else (a > border)
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=d, device=v.device)
    return (grid[n] * unit * torch.sign(b)).flatten(1)


def _meaning(codes, scales):
    d = torch.float64
    codes, scales = codes.view(torch.uint8), scales.view(torch.uint8)
    table = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    table = torch.tensor(table + [-v for v in table], dtype=d, device=codes.device)
    out = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=d, device=codes.device)
    out[:, 0::2] = table[(codes % 16).int()]
    out[:, 1::2] = table[torch.div(codes, 16, rounding_mode="floor").int()]
    return out * torch.repeat_interleave(torch.exp2(scales.to(d) - 127), BLOCK, dim=1)


def _normed(s, N):
    """The stream in its type, and its norm."""
    d = torch.float64
    h = s["x"] if s["residual"] is None else (s["x"].to(d) + s["residual"].to(d)).to(s["x"].dtype)
    v = h.to(d)
    centred = v - torch.sum(v, dim=1, keepdim=True) / N
    rms = torch.sqrt(torch.sum(centred ** 2, dim=1, keepdim=True) / N + EPS)
    return v, centred / rms, rms


def exact(case, seed):
    s = prepare(case, seed)
    d = torch.float64
    if case["op"] == "norm":
        v, unit, _ = _normed(s, case["N"])
        y = torch.addcmul(s["bias"].to(d), unit, s["weight"].to(d))
        out = {"y": y}
        if case["out"] == "e4m3":
            out["scales"] = torch.maximum(y.max(dim=1).values, -y.min(dim=1).values).clamp(min=AMAX_MIN) / E4M3_MAX
            out["y"] = y / out["scales"].unsqueeze(1)
        if s["residual"] is not None:
            out["h"] = v
        return out
    if case["op"] == "grad":
        N, dy = case["N"], s["dy"].to(d)
        _, unit, rms = _normed({"x": s["x"], "residual": None}, N)
        g = dy * s["weight"].to(d)
        along = torch.sum(g * unit, dim=1, keepdim=True) / N
        dx = (g - torch.sum(g, dim=1, keepdim=True) / N - unit * along) / rms
        if s["residual"] is not None:
            dx += s["residual"].to(d)
        return {"dx": dx, "dweight": torch.sum(dy * unit, dim=0), "dbias": torch.sum(dy, dim=0)}
    if case["op"] == "trip":
        return _nearest(s["x"].to(d))
    w = _meaning(s["W"], s["w_scales"])
    if case["op"] == "mx":
        return torch.mm(_meaning(s["A"], s["a_scales"]), w.t())
    v, unit, _ = _normed(s, case["K"])
    y = _nearest(torch.addcmul(s["bias"].to(d), unit, s["weight"].to(d)))
    return {"C": torch.mm(y, w.t()), "h": v}
