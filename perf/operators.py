"""The operators of a quantised linear layer: what is measured, and their plain forms.

A residual stream is added up and normalised, the result leaves in 16 bits or in e4m3 with one scale a row, and it
meets weights held in e4m3 (many rows: a prompt) or in 4 bits with a scale for each group (few rows: single tokens);
the norm also has its gradient. `run` computes a case in plain torch operations where `own` is false, and with this
repository's kernels where it is true.

A row of length K times a weight W of shape N x K is written `A @ B`, with B the K x N view of W (unit row stride).
"""
import math

import torch

own = False

E4M3_MAX = 448.0
AMAX_MIN = 2.0 ** -100  # below it a row counts as zeros: keeps the scale and its reciprocal normal numbers
EPS = 1e-6

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}


def listed():
    return [
        # One token of one sequence: latency. The 8-bit output feeds an 8-bit product.
        {"name": "norm 1x4096 e4m3", "op": "norm", "M": 1, "N": 4096, "type": "bf16", "out": "e4m3", "residual": True},
        # A batch of short prompts, an odd number of rows, a width that is no power of two; 16-bit output.
        {"name": "norm 1021x5000 fp16", "op": "norm", "M": 1021, "N": 5000, "type": "fp16", "out": "fp16", "residual": True},
        # Long prompts or a training batch.
        {"name": "norm 8192x8192 e4m3", "op": "norm", "M": 8192, "N": 8192, "type": "bf16", "out": "e4m3", "residual": True},
        # The gradient at an ordinary and at a large training step; the residual stream brings a gradient of its own.
        {"name": "grad 1021x2048 fp16", "op": "grad", "M": 1021, "N": 2048, "type": "fp16", "residual": False},
        {"name": "grad 8192x8192 bf16", "op": "grad", "M": 8192, "N": 8192, "type": "bf16", "residual": True},
        # 8-bit weights: one token, a batch of tokens, a ragged prompt, a long prompt.
        {"name": "fp8 1x4096x4096", "op": "fp8", "M": 1, "N": 4096, "K": 4096, "out": "bf16"},
        {"name": "fp8 24x8192x8192", "op": "fp8", "M": 24, "N": 8192, "K": 8192, "out": "fp16"},
        {"name": "fp8 1000x5000x4112", "op": "fp8", "M": 1000, "N": 5000, "K": 4112, "out": "bf16"},
        {"name": "fp8 8192x8192x8192", "op": "fp8", "M": 8192, "N": 8192, "K": 8192, "out": "bf16"},
        # 4-bit weights: one token at a small and at a large layer, a batch of tokens with zero points.
        {"name": "w4 1x4096x4096", "op": "w4", "M": 1, "N": 4096, "K": 4096, "group": 128, "type": "bf16", "zeros": False},
        {"name": "w4 1x28672x8192", "op": "w4", "M": 1, "N": 28672, "K": 8192, "group": 128, "type": "fp16", "zeros": True},
        {"name": "w4 47x6000x4096", "op": "w4", "M": 47, "N": 6000, "K": 4096, "group": 64, "type": "bf16", "zeros": True},
    ]


def _between(rng, low, high, step=1):
    """A multiple of `step` in [low, high], spread evenly over its logarithm."""
    v = math.exp(rng.uniform(math.log(low), math.log(high + 1)))
    return min(high // step * step, max(-(-low // step) * step, int(v) // step * step))


def draw(rng):
    op = rng.choice(["norm", "grad", "fp8", "w4"])
    if op in ("norm", "grad"):
        N = _between(rng, 256, 16384, 8)
        M = _between(rng, 1, min(8192, (1 << 26) // N))
        case = {"op": op, "M": M, "N": N, "type": rng.choice(["bf16", "fp16"]), "residual": rng.random() < 0.7}
        if op == "norm":
            case["out"] = rng.choice([case["type"], "e4m3"])
        return case
    if op == "fp8":
        M = _between(rng, 1, 8192)
        N = _between(rng, 256, 16384, 8)
        K = _between(rng, 256, max(256, min(16384, 8192 ** 3 // (M * N))), 16)
        return {"op": op, "M": M, "N": N, "K": K, "out": rng.choice(["bf16", "fp16", "fp32"])}
    group = rng.choice([32, 64, 128])
    M = _between(rng, 1, 64)
    N = _between(rng, 256, 28672, 8)
    K = _between(rng, 256, min(28672, 28672 * 8192 // N), group)
    return {"op": op, "M": M, "N": N, "K": K, "group": group, "type": rng.choice(["bf16", "fp16"]),
            "zeros": rng.random() < 0.5}


def work(case):
    M, N = case["M"], case["N"]
    if case["op"] == "norm":
        t = SIZE[case["type"]]
        b = M * N * (t + SIZE[case["out"]] + (2 * t if case["residual"] else 0)) + N * t
        return {"bytes": b + (4 * M if case["out"] == "e4m3" else 0), "flops": 5 * M * N}
    if case["op"] == "grad":
        t = SIZE[case["type"]]
        return {"bytes": M * N * t * (4 if case["residual"] else 3) + N * (t + 4), "flops": 11 * M * N}
    K = case["K"]
    if case["op"] == "fp8":
        return {"bytes": M * K + N * K + 4 * (M + N) + M * N * SIZE[case["out"]], "flops": 2 * M * N * K}
    t = SIZE[case["type"]]
    groups = N * (K // case["group"])
    return {"bytes": M * K * t + N * K // 2 + groups * (t + (1 if case["zeros"] else 0)) + M * N * t,
            "flops": 2 * M * N * K}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _e4m3_rows(w):
    """The rows of w in e4m3, and one fp32 scale a row."""
    s = w.abs().amax(dim=1).clamp_min(AMAX_MIN) / E4M3_MAX
    return (w / s[:, None]).to(torch.float8_e4m3fn), s


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device=dev, dtype=torch.float32, generator=g)

    M, N = case["M"], case["N"]
    s = {"case": case}
    if case["op"] in ("norm", "grad"):
        t = TYPES[case["type"]]
        s["weight"] = (1 + 0.1 * normal(N)).to(t)
        # Activations: a few channels are much larger than the others.
        loud = 1 + 20 * (torch.rand(N, device=dev, generator=g) < 0.01)
        s["x"] = (normal(M, N) * loud).to(t)
        s["residual"] = normal(M, N).to(t) if case["residual"] else None
        if case["op"] == "grad":
            s["dy"] = normal(M, N).to(t)
        return s
    K = case["K"]
    if case["op"] == "fp8":
        s["A"], s["a_scales"] = _e4m3_rows(normal(M, K) * (1 + 10 * (torch.rand(K, device=dev, generator=g) < 0.01)))
        w, s["b_scales"] = _e4m3_rows(normal(N, K) / math.sqrt(K))
        s["B"] = w.t()
        return s
    t = TYPES[case["type"]]
    s["A"] = normal(M, K).to(t)
    w = (normal(N, K) / math.sqrt(K)).view(N, K // case["group"], case["group"])
    if case["zeros"]:
        low, high = w.amin(dim=2), w.amax(dim=2)
        scales = ((high - low) / 15).to(t)
        zeros = (-low / scales.float()).round().clamp(0, 15)
        s["zeros"] = zeros.to(torch.uint8)
    else:
        scales = (w.abs().amax(dim=2) / 7).to(t)
        zeros = torch.full_like(scales, 8, dtype=torch.float32)
        s["zeros"] = None
    q = ((w / scales.float()[:, :, None]).round() + zeros[:, :, None]).clamp(0, 15).to(torch.uint8).view(N, K)
    s["codes"] = q[:, 0::2] | (q[:, 1::2] << 4)  # two codes a byte, the even column's in the low half
    s["scales"] = scales
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def _plain_norm(s, case):
    t = TYPES[case["type"]]
    h = s["x"]
    if s["residual"] is not None:
        h = (h.float() + s["residual"].float()).to(t)
    f = h.float()
    r = torch.rsqrt((f * f).mean(dim=1, keepdim=True) + EPS)
    y = f * r * s["weight"].float()
    if case["out"] == "e4m3":
        y, scales = _e4m3_rows(y)
        out = {"y": y, "scales": scales}
    else:
        out = {"y": y.to(t)}
    if s["residual"] is not None:
        out["h"] = h
    return out


def _plain_grad(s, case):
    t = TYPES[case["type"]]
    dy, h, w = s["dy"].float(), s["x"].float(), s["weight"].float()
    r = torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS)
    g = dy * w
    dx = g * r - h * ((g * h).mean(dim=1, keepdim=True) * r * r * r)
    if s["residual"] is not None:
        dx = dx + s["residual"].float()
    return {"dx": dx.to(t), "dweight": (dy * h * r).sum(dim=0)}


def _plain_fp8(s, case):
    c = s["A"].float() @ s["B"].float()
    return (c * s["a_scales"][:, None] * s["b_scales"][None, :]).to(TYPES[case["out"]])


def _plain_w4(s, case):
    N, K, G = case["N"], case["K"], case["group"]
    q = torch.stack([s["codes"] & 15, s["codes"] >> 4], dim=2).view(N, K // G, G).float()
    z = s["zeros"].float()[:, :, None] if s["zeros"] is not None else 8.0
    w = ((q - z) * s["scales"].float()[:, :, None]).view(N, K)
    return (s["A"].float() @ w.t()).to(TYPES[case["type"]])


def _own_norm(s, case):
    import async_stage_tile_amd as pt
    got = pt.pipe_rmsnorm(s["x"], s["weight"], residual=s["residual"], eps=EPS, out_dtype=TYPES[case["out"]])
    names = ["y"] + (["scales"] if case["out"] == "e4m3" else []) + (["h"] if s["residual"] is not None else [])
    return dict(zip(names, got if len(names) > 1 else (got,)))


def _own_grad(s, case):
    import async_stage_tile_amd as pt
    dx, dweight = pt.pipe_rmsnorm_backward(s["dy"], s["x"], s["weight"], dh=s["residual"], eps=EPS)
    return {"dx": dx, "dweight": dweight}


def _own_fp8(s, case):
    import async_stage_tile_amd as pt
    return pt.pipe_gemm_fp8(s["A"], s["a_scales"], s["B"], s["b_scales"], out_dtype=TYPES[case["out"]])


def _own_w4(s, case):
    import async_stage_tile_amd as pt
    return pt.pipe_gemm_w4(s["A"], s["codes"], s["scales"], zeros=s["zeros"])


_PLAIN = {"norm": _plain_norm, "grad": _plain_grad, "fp8": _plain_fp8, "w4": _plain_w4}
_OWN = {"norm": _own_norm, "grad": _own_grad, "fp8": _own_fp8, "w4": _own_w4}


def run(state):
    case = state["case"]
    return (_OWN if own else _PLAIN)[case["op"]](state, case)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    d = torch.float64
    if case["op"] == "norm":
        # The stream's sum is held in the stream's type: that rounding is part of the definition.
        h = s["x"] if s["residual"] is None else (s["x"].to(d) + s["residual"].to(d)).to(s["x"].dtype)
        v = h.to(d)
        y = v / torch.sqrt(torch.sum(v ** 2, dim=1) / case["N"] + EPS).unsqueeze(1) * s["weight"].to(d)
        out = {"y": y}
        if case["out"] == "e4m3":
            out["scales"] = torch.maximum(y.max(dim=1).values, -y.min(dim=1).values).clamp(min=AMAX_MIN) / E4M3_MAX
            out["y"] = y / out["scales"].unsqueeze(1)
        if s["residual"] is not None:
            out["h"] = v
        return out
    if case["op"] == "grad":
        v, dy, w = s["x"].to(d), s["dy"].to(d), s["weight"].to(d)
        rms = torch.sqrt(torch.sum(v ** 2, dim=1, keepdim=True) / case["N"] + EPS)
        unit = v / rms
        along = torch.sum(dy * w * unit, dim=1, keepdim=True) / case["N"]
        dx = (dy * w - unit * along) / rms
        if s["residual"] is not None:
            dx += s["residual"].to(d)
        return {"dx": dx, "dweight": torch.einsum("mn,mn->n", dy, unit)}
    if case["op"] == "fp8":
        a = s["A"].to(d) * s["a_scales"].to(d).unsqueeze(1)
        w = s["B"].t().to(d) * s["b_scales"].to(d).unsqueeze(1)
        return torch.mm(a, w.t())
    N, K, G = case["N"], case["K"], case["group"]
    w = torch.empty(N, K, dtype=d, device=s["codes"].device)
    w[:, 0::2] = (s["codes"] % 16).to(d)
    w[:, 1::2] = torch.div(s["codes"], 16, rounding_mode="floor").to(d)
    if s["zeros"] is None:
        w -= 8
    else:
        w -= torch.repeat_interleave(s["zeros"].to(d), G, dim=1)
    w *= torch.repeat_interleave(s["scales"].to(d), G, dim=1)
    return torch.mm(s["A"].to(d), w.t())
