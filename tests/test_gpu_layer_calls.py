"""Calls of layer norm and the microscaled 4-bit form that their documentation allows: outputs in the place of operands in
every shape of workgroup, workspaces given, streams' memory, operands of function transforms, one operand in two places."""
import pytest
import torch

import async_stage_tile_amd as pt
from tests import test_gpu_stream_memory as memory
from tests.test_gpu_layernorm import BF, DEV, E4, F32, F4, HF, normal
from tests.test_gpu_mxfp4 import operand, values

pytestmark = pytest.mark.gpu
U8 = torch.uint8


@pytest.fixture(autouse=True)
def _name(request):
    print(f"[layer calls] {request.node.name}", flush=True)
    yield
    torch.cuda.synchronize()


SHAPES = [(5, 8), (301, 512), (5001, 504), (70, 1000), (1021, 2048), (40, 4096), (700, 4096), (2500, 4000), (33, 8192),
          (300, 5000), (4200, 8192), (600, 16384), (2100, 16384), (300, 24008), (1100, 32768)]


@pytest.mark.parametrize("M,N", SHAPES)
@pytest.mark.parametrize("dtype", (BF, HF))
def test_norm_in_place(M, N, dtype):
    """h in the place of x or of the residual, y in that of x."""
    x, res = normal((M, N), dtype, 1), normal((M, N), dtype, 2)
    w, b = normal((N,), dtype, 3), normal((N,), dtype, 4)
    y, h = pt.pipe_layernorm(x, w, b, residual=res)
    for place in (0, 1):
        t = [x.clone(), res.clone()]
        got = pt.pipe_layernorm(t[0], w, b, residual=t[1], h=t[place])
        assert got[1] is t[place] and torch.equal(got[0], y) and torch.equal(got[1], h)
        assert torch.equal(t[1 - place], (x, res)[1 - place])
    t = x.clone()
    got = pt.pipe_layernorm(t, w, b, residual=res, y=t)
    assert got[0] is t and torch.equal(t, y) and torch.equal(got[1], h)
    t = [x.clone(), res.clone()]
    pt.pipe_layernorm(t[0], w, b, residual=t[1], y=t[0], h=t[1])
    assert torch.equal(t[0], y) and torch.equal(t[1], h)
    t = x.clone()
    assert torch.equal(pt.pipe_layernorm(t, w, b, y=t), pt.pipe_layernorm(x, w, b))


@pytest.mark.parametrize("M,N", SHAPES)
@pytest.mark.parametrize("dtype", (BF, HF))
def test_grad_in_place(M, N, dtype):
    """dx in the place of dy or of dh; dh and dy the same tensor."""
    dy, x, dh = (normal((M, N), dtype, s) for s in (5, 6, 7))
    w = normal((N,), dtype, 8)
    for more in (dh, None):
        want = pt.pipe_layernorm_backward(dy, x, w, dh=more)
        t = dy.clone()
        got = pt.pipe_layernorm_backward(t, x, w, dh=more, dx=t)
        assert got[0] is t and all(torch.equal(a, b) for a, b in zip(got, want))
    want = pt.pipe_layernorm_backward(dy, x, w, dh=dh)
    t = dh.clone()
    got = pt.pipe_layernorm_backward(dy, x, w, dh=t, dx=t)
    assert got[0] is t and all(torch.equal(a, b) for a, b in zip(got, want))
    want = pt.pipe_layernorm_backward(dy, x, w, dh=dy.clone())
    t = dy.clone()
    got = pt.pipe_layernorm_backward(t, x, w, dh=t, dx=t)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("M,N,K", [(40, 256, 16384), (150, 512, 4096), (4096, 4096, 16416), (700, 520, 6016), (4100, 264, 96)])
def test_products_with_one_workspace_after_another(M, N, K):
    """A workspace given, of just the size and of a larger one's rest, filled with NaN: what it held does not matter."""
    need = pt.pipe_gemm_mxfp4_workspace_bytes(M, N, K)
    space = torch.full((need // 4 + 1024,), float("nan"), device=DEV).view(U8)
    (A, sa), (W, sw) = operand(M, K, 9), operand(N, K, 10)
    want = values(A, sa).float() @ values(W, sw).float().t()
    for ws in (space, space[:need], space[16:16 + need]):
        assert torch.equal(pt.pipe_gemm_mxfp4(A, sa, W, sw, out_dtype=F32, workspace=ws), want)
        assert torch.equal(pt.pipe_gemm_mxfp4(W[:M], sw[:M], W, sw, out_dtype=F32)[:, :8],
                           (values(W[:M], sw[:M]).float() @ values(W[:8], sw[:8]).float().t()))


def calls():
    x, w = normal((512, 1024), BF, 11), normal((1024,), BF, 12)
    (A, sa), (W, sw) = operand(40, 16384, 13), operand(256, 16384, 14)
    (B, sb), (V, sv) = operand(4096, 16416, 15), operand(4096, 16416, 16)
    assert pt.pipe_gemm_mxfp4_workspace_bytes(40, 256, 16384) > 0 and pt.pipe_layernorm_backward_workspace_bytes(512, 1024) > 0
    assert pt.pipe_gemm_mxfp4_workspace_bytes(4096, 4096, 16416) > 0
    return {
        "layernorm": lambda s: pt.pipe_layernorm(x, w, w, residual=x, out_dtype=E4, stream=s),
        "layernorm_4bit": lambda s: pt.pipe_layernorm(x, w, w, residual=x, out_dtype=F4, stream=s),
        "layernorm_backward": lambda s: pt.pipe_layernorm_backward(x, x, w, dh=x, stream=s),
        "quantize": lambda s: pt.pipe_quantize_mxfp4(x, stream=s),
        "dequantize": lambda s: pt.pipe_dequantize_mxfp4(A, sa, stream=s),
        "gemm": lambda s: pt.pipe_gemm_mxfp4(A, sa, W, sw, stream=s),
        "gemm_scales": lambda s: pt.pipe_gemm_mxfp4(B, sb, V, sv, stream=s),
    }


@pytest.mark.parametrize("name", list(("layernorm", "layernorm_4bit", "layernorm_backward", "quantize", "dequantize", "gemm",
                                       "gemm_scales")))
@pytest.mark.parametrize("check", ("test_no_output_in_memory_that_the_current_stream_still_writes",
                                   "test_no_output_reused_before_the_current_stream_has_read_it",
                                   "test_captured_on_a_stream_that_joins_the_capture"))
def test_stream_memory(monkeypatch, name, check):
    monkeypatch.setattr(memory, "calls", calls)
    getattr(memory, check)(name)


def operators():
    x, w = normal((4, 64), BF, 17), normal((64,), BF, 18)
    (A, sa), (W, sw) = operand(4, 64, 19), operand(8, 64, 20)
    return {"layernorm": (lambda a, b, c, d: pt.pipe_layernorm(a, b, c, residual=d), (x, w, w, x)),
            "layernorm_backward": (lambda a, b, c, d: pt.pipe_layernorm_backward(a, b, c, dh=d), (x, x, w, x)),
            "quantize": (pt.pipe_quantize_mxfp4, (x,)),
            "dequantize": (pt.pipe_dequantize_mxfp4, (A, sa)),
            "gemm": (pt.pipe_gemm_mxfp4, (A, sa, W, sw))}


@pytest.mark.parametrize("name", ("layernorm", "layernorm_backward", "quantize", "dequantize", "gemm"))
def test_operands_of_function_transforms_are_refused(name):
    f, args = operators()[name]
    for i, a in enumerate(args):
        with pytest.raises(RuntimeError):
            torch.func.vmap(lambda t: f(*args[:i], t, *args[i + 1:]))(a.expand((2,) + tuple(a.shape)))
        if a.dtype == BF:
            with pytest.raises(RuntimeError):
                torch.func.vjp(lambda t: f(*args[:i], t, *args[i + 1:]), a)
    out = f(*args)
    torch.cuda.synchronize()
    assert (out[0] if isinstance(out, tuple) else out).numel() > 0
