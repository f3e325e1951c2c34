"""A language-model layer's projection on quantised weights, with the operators of pipe_linear.h.

One layer keeps its weights twice: in e4m3 with a scale for each row, for prompts (many rows: bound by arithmetic),
and in 4 bits with a scale and a zero point for each group of 128, for single tokens (few rows: bound by reading the
weights). `forward` adds the block's input to the residual stream, normalises it and multiplies it, choosing by the
number of rows; `backward` takes the gradient of a 16-bit training step back through the norm.

    python examples/quantised_layer.py        # needs an MI355X; compares each step with 64-bit arithmetic
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import async_stage_tile_amd as pt  # noqa: E402

EPS = 1e-6
FEW = 64        # rows that the 4-bit product is laid out for
GROUP = 128


class QuantisedLayer:
    """norm(h) @ weight.T for a weight of N rows (outputs) and K columns (inputs), K a multiple of 128."""

    def __init__(self, weight, norm_weight):
        self.weight, self.norm_weight = weight, norm_weight
        w = weight.float()
        self.row_scales = w.abs().amax(dim=1).clamp_min(2.0 ** -100) / 448
        self.e4m3 = (w / self.row_scales[:, None]).to(torch.float8_e4m3fn)
        g = w.view(w.shape[0], -1, GROUP)
        # From zero or below to zero or above: the zero point is one of the 16 codes also where a group has one sign.
        low, high = g.amin(dim=2).clamp_max(0), g.amax(dim=2).clamp_min(0)
        self.scales = ((high - low) / 15).clamp_min(torch.finfo(weight.dtype).tiny).to(weight.dtype)
        self.zeros = (-low / self.scales.float()).round().clamp(0, 15).to(torch.uint8)
        q = (g / self.scales.float()[:, :, None]).round() + self.zeros[:, :, None]
        q = q.clamp(0, 15).to(torch.uint8).view(w.shape)
        self.codes = q[:, 0::2] | (q[:, 1::2] << 4)

    def forward(self, x, residual):
        """The layer's output, and the residual stream with x added to it."""
        if x.shape[0] <= FEW:
            y, h = pt.pipe_rmsnorm(x, self.norm_weight, residual=residual, eps=EPS)
            return pt.pipe_gemm_w4(y, self.codes, self.scales, zeros=self.zeros), h
        y, y_scales, h = pt.pipe_rmsnorm(x, self.norm_weight, residual=residual, eps=EPS,
                                         out_dtype=torch.float8_e4m3fn)
        return pt.pipe_gemm_fp8(y, y_scales, self.e4m3.t(), self.row_scales, out_dtype=x.dtype), h

    def backward(self, dout, h, dh):
        """From the gradients of the output and of the stream: the gradient of both addends and of norm_weight.
        bfloat16, as the framework's 16-bit product takes it."""
        dy = pt.pipe_gemm_mainloop(dout, self.weight, out_dtype=torch.bfloat16)
        return pt.pipe_rmsnorm_backward(dy, h, self.norm_weight, dh=dh, eps=EPS)


def relative(got, ref):
    return float((got.double() - ref).norm() / ref.norm())


def run(rows, N=1024, K=2048, dtype=torch.bfloat16, seed=0):
    """One forward and (in bfloat16) one backward pass; returns their distances from 64-bit arithmetic on the
    unquantised weights (forward) and on the same dy (backward)."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    layer = QuantisedLayer((normal(N, K) / K ** 0.5).to(dtype), (1 + 0.1 * normal(K)).to(dtype))
    x, residual = normal(rows, K).to(dtype), normal(rows, K).to(dtype)
    out, h = layer.forward(x, residual)
    v = h.double()
    r = 1 / torch.sqrt((v * v).mean(dim=1, keepdim=True) + EPS)
    got = {"forward": relative(out, (v * r * layer.norm_weight.double()) @ layer.weight.double().t())}
    if dtype == torch.bfloat16:
        dout, dh = normal(rows, N).to(dtype), normal(rows, K).to(dtype)
        dx, dweight = layer.backward(dout, h, dh)
        dy = dout.double() @ layer.weight.double()
        gw = dy * layer.norm_weight.double()
        ref = r * gw - v * r ** 3 * (gw * v).mean(dim=1, keepdim=True) + dh.double()
        got["dx"] = relative(dx, ref)
        got["dweight"] = relative(dweight, (dy * v * r).sum(dim=0))
    return got


if __name__ == "__main__":
    for rows in (1, 48, 500):
        print(rows, "rows:", {k: f"{v:.2e}" for k, v in run(rows).items()}, flush=True)
