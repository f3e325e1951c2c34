"""Checks of layer norm's and the microscaled 4-bit form's entry points that need no GPU: bad arguments are refused before
anything reaches the device (the addresses below are never dereferenced)."""
import os
import re

import pytest
import torch

import async_stage_tile_amd as pt
from async_stage_tile_amd import linear
from tests.conftest import ROOT

P = 0x10000
BF, HF, F32, E4, MX = pt.PIPE_BF16, pt.PIPE_FP16, pt.PIPE_FP32, pt.PIPE_E4M3, pt.PIPE_MXFP4


def fns():
    return linear._setup()


def test_constants_of_the_header():
    txt = open(os.path.join(ROOT, "include", "pipe_linear.h")).read()
    assert int(re.search(r"#define PIPE_LAYERNORM_MAX_N (\d+)", txt).group(1)) == pt.PIPE_LAYERNORM_MAX_N
    assert int(re.search(r"PIPE_MXFP4 = (\d+)", txt).group(1)) == MX


def norm(x=P, res=0, w=P, b=0, y=P, s=0, h=0, M=4, N=64, ldx=64, ldr=64, ldy=64, lds=16, ldh=64, eps=1e-5, t=BF, o=BF):
    return fns().pipe_layernorm(x, res, w, b, y, s, h, M, N, ldx, ldr, ldy, lds, ldh, eps, t, o, None)


@pytest.mark.parametrize("change,status", [
    (dict(t=F32, o=F32), pt.PIPE_ERR_CONFIG), (dict(t=MX, o=MX), pt.PIPE_ERR_CONFIG), (dict(t=BF, o=HF), pt.PIPE_ERR_CONFIG),
    (dict(o=5), pt.PIPE_ERR_CONFIG), (dict(eps=-1.0), pt.PIPE_ERR_CONFIG), (dict(eps=float("nan")), pt.PIPE_ERR_CONFIG),
    (dict(M=-1), pt.PIPE_ERR_SHAPE), (dict(N=-8), pt.PIPE_ERR_SHAPE), (dict(N=63), pt.PIPE_ERR_SHAPE),
    (dict(M=1 << 31), pt.PIPE_ERR_SHAPE), (dict(N=pt.PIPE_LAYERNORM_MAX_N + 8, ldx=1 << 20, ldy=1 << 20), pt.PIPE_ERR_SHAPE),
    (dict(ldx=56), pt.PIPE_ERR_SHAPE), (dict(ldy=56), pt.PIPE_ERR_SHAPE), (dict(ldx=1 << 40), pt.PIPE_ERR_SHAPE),
    (dict(o=MX, s=P, N=40), pt.PIPE_ERR_SHAPE), (dict(o=MX, s=P, ldy=16), pt.PIPE_ERR_SHAPE),
    (dict(o=MX, s=P, lds=1), pt.PIPE_ERR_SHAPE), (dict(o=MX, s=P, lds=1 << 24), pt.PIPE_ERR_SHAPE),
    (dict(x=0), pt.PIPE_ERR_NULL), (dict(w=0), pt.PIPE_ERR_NULL), (dict(y=0), pt.PIPE_ERR_NULL), (dict(res=P), pt.PIPE_ERR_NULL),
    (dict(h=P), pt.PIPE_ERR_NULL), (dict(o=E4), pt.PIPE_ERR_NULL), (dict(o=MX), pt.PIPE_ERR_NULL),
    (dict(x=P + 8), pt.PIPE_ERR_ALIGN), (dict(y=P + 8), pt.PIPE_ERR_ALIGN), (dict(w=P + 2), pt.PIPE_ERR_ALIGN),
    (dict(b=P + 2), pt.PIPE_ERR_ALIGN), (dict(ldx=68), pt.PIPE_ERR_ALIGN), (dict(o=E4, s=P, y=P + 4), pt.PIPE_ERR_ALIGN),
    (dict(o=E4, s=P + 2), pt.PIPE_ERR_ALIGN), (dict(o=MX, s=P, y=P + 8), pt.PIPE_ERR_ALIGN),
    (dict(o=MX, s=P + 8), pt.PIPE_ERR_ALIGN), (dict(o=MX, s=P, lds=8), pt.PIPE_ERR_ALIGN),
    (dict(o=MX, s=P, ldy=40), pt.PIPE_ERR_ALIGN), (dict(res=P, h=P + 8), pt.PIPE_ERR_ALIGN),
    (dict(res=P, h=P, ldr=72, ldh=60), pt.PIPE_ERR_SHAPE),
    (dict(M=0, x=0, y=0, w=0), pt.PIPE_OK), (dict(N=0, x=0, y=0, w=0), pt.PIPE_OK),
])
def test_layernorm_refusals(change, status):
    assert norm(**change) == status


def grad(dy=P, x=P, w=P, dh=0, dx=P, dw=P, db=P, M=4, N=64, lddy=64, ldx=64, lddh=64, lddx=64, eps=1e-5, t=BF,
         ws=P, wsb=1 << 30):
    return fns().pipe_layernorm_backward(dy, x, w, dh, dx, dw, db, M, N, lddy, ldx, lddh, lddx, eps, t, ws, wsb, None)


@pytest.mark.parametrize("change,status", [
    (dict(t=F32), pt.PIPE_ERR_CONFIG), (dict(eps=-1.0), pt.PIPE_ERR_CONFIG), (dict(N=60), pt.PIPE_ERR_SHAPE),
    (dict(M=-4), pt.PIPE_ERR_SHAPE), (dict(lddx=8), pt.PIPE_ERR_SHAPE), (dict(dy=0), pt.PIPE_ERR_NULL),
    (dict(x=0), pt.PIPE_ERR_NULL), (dict(dx=0), pt.PIPE_ERR_NULL), (dict(w=0), pt.PIPE_ERR_NULL), (dict(dw=0), pt.PIPE_ERR_NULL),
    (dict(db=0), pt.PIPE_ERR_NULL), (dict(dw=P + 4), pt.PIPE_ERR_ALIGN), (dict(db=P + 8), pt.PIPE_ERR_ALIGN),
    (dict(dh=P + 2), pt.PIPE_ERR_ALIGN), (dict(dh=P, lddh=68), pt.PIPE_ERR_ALIGN), (dict(M=100, ws=P + 4), pt.PIPE_ERR_ALIGN),
    (dict(M=100, ws=0), pt.PIPE_ERR_WORKSPACE), (dict(M=100, wsb=16), pt.PIPE_ERR_WORKSPACE), (dict(N=0, dw=0, dy=0), pt.PIPE_OK),
])
def test_layernorm_backward_refusals(change, status):
    assert grad(**change) == status


def quant(x=P, c=P, s=P, M=4, K=64, ldx=64, ldc=32, lds=16, t=BF, name="pipe_quantize_mxfp4"):
    if name == "pipe_quantize_mxfp4":
        return fns().pipe_quantize_mxfp4(x, c, s, M, K, ldx, ldc, lds, t, None)
    return fns().pipe_dequantize_mxfp4(c, s, x, M, K, ldc, lds, ldx, t, None)


@pytest.mark.parametrize("name", ["pipe_quantize_mxfp4", "pipe_dequantize_mxfp4"])
@pytest.mark.parametrize("change,status", [
    (dict(t=E4), pt.PIPE_ERR_CONFIG), (dict(t=MX), pt.PIPE_ERR_CONFIG), (dict(t=-1), pt.PIPE_ERR_CONFIG),
    (dict(K=48), pt.PIPE_ERR_SHAPE), (dict(K=-32), pt.PIPE_ERR_SHAPE), (dict(M=-1), pt.PIPE_ERR_SHAPE),
    (dict(M=1 << 31), pt.PIPE_ERR_SHAPE), (dict(M=1 << 20, K=(1 << 20) + 32, ldx=1 << 21, ldc=1 << 20, lds=1 << 16), pt.PIPE_ERR_SHAPE),
    (dict(ldx=56), pt.PIPE_ERR_SHAPE), (dict(ldc=16), pt.PIPE_ERR_SHAPE), (dict(lds=1), pt.PIPE_ERR_SHAPE),
    (dict(lds=1 << 24), pt.PIPE_ERR_SHAPE), (dict(x=0), pt.PIPE_ERR_NULL), (dict(c=0), pt.PIPE_ERR_NULL), (dict(s=0), pt.PIPE_ERR_NULL),
    (dict(x=P + 8), pt.PIPE_ERR_ALIGN), (dict(c=P + 8), pt.PIPE_ERR_ALIGN), (dict(s=P + 4), pt.PIPE_ERR_ALIGN),
    (dict(ldx=68), pt.PIPE_ERR_ALIGN), (dict(ldc=40), pt.PIPE_ERR_ALIGN), (dict(lds=8), pt.PIPE_ERR_ALIGN),
    (dict(M=0, x=0), pt.PIPE_OK), (dict(K=0, x=0), pt.PIPE_OK),
])
def test_conversion_refusals(name, change, status):
    assert quant(name=name, **change) == status


def gemm(A=P, sa=P, W=P, sw=P, C=P, M=4, N=64, K=64, lda=32, ldsa=16, ldw=32, ldsw=16, ldc=64, o=BF, ws=0, wsb=0):
    return fns().pipe_gemm_mxfp4(A, sa, W, sw, C, M, N, K, lda, ldsa, ldw, ldsw, ldc, o, ws, wsb, None)


@pytest.mark.parametrize("change,status", [
    (dict(o=E4), pt.PIPE_ERR_CONFIG), (dict(o=MX), pt.PIPE_ERR_CONFIG), (dict(o=-1), pt.PIPE_ERR_CONFIG),
    (dict(N=60), pt.PIPE_ERR_SHAPE), (dict(K=48), pt.PIPE_ERR_SHAPE), (dict(K=-32), pt.PIPE_ERR_SHAPE),
    (dict(lda=16), pt.PIPE_ERR_SHAPE), (dict(ldw=16), pt.PIPE_ERR_SHAPE), (dict(ldc=56), pt.PIPE_ERR_SHAPE),
    (dict(lda=1 << 24), pt.PIPE_ERR_SHAPE), (dict(ldw=1 << 24), pt.PIPE_ERR_SHAPE), (dict(ldsa=1), pt.PIPE_ERR_SHAPE),
    (dict(ldsw=1 << 24), pt.PIPE_ERR_SHAPE), (dict(M=1 << 31), pt.PIPE_ERR_SHAPE),
    (dict(M=(1 << 31) - 1, N=(1 << 31) - 8, ldc=1 << 31), pt.PIPE_ERR_SHAPE),
    (dict(A=0), pt.PIPE_ERR_NULL), (dict(W=0), pt.PIPE_ERR_NULL), (dict(C=0), pt.PIPE_ERR_NULL), (dict(sa=0), pt.PIPE_ERR_NULL),
    (dict(sw=0), pt.PIPE_ERR_NULL), (dict(A=P + 8), pt.PIPE_ERR_ALIGN), (dict(lda=40), pt.PIPE_ERR_ALIGN),
    (dict(ldw=40), pt.PIPE_ERR_ALIGN), (dict(C=P + 8), pt.PIPE_ERR_ALIGN), (dict(ldc=68), pt.PIPE_ERR_ALIGN),
    (dict(sa=P + 1), pt.PIPE_ERR_ALIGN), (dict(ldsw=24), pt.PIPE_ERR_ALIGN), (dict(M=0, A=0), pt.PIPE_OK), (dict(N=0, A=0), pt.PIPE_OK),
])
def test_gemm_refusals(change, status):
    assert gemm(**change) == status


def test_workspaces():
    """Where a shape needs a workspace, a missing or short one is refused."""
    M, N, K = 40, 256, 16384
    need = pt.pipe_gemm_mxfp4_workspace_bytes(M, N, K)
    assert need > 0 and need % (4 * M * N) == 0
    kw = dict(M=M, N=N, K=K, lda=K // 2, ldw=K // 2, ldsa=K // 32, ldsw=K // 32, ldc=N)
    assert gemm(**kw) == pt.PIPE_ERR_WORKSPACE
    assert gemm(ws=P, wsb=need - 1, **kw) == pt.PIPE_ERR_WORKSPACE
    assert gemm(ws=P + 4, wsb=need, **kw) == pt.PIPE_ERR_ALIGN
    for shape in ((1, 256, 8192), (0, 256, 8192), (40, 0, 8192), (40, 256, 0)):
        assert pt.pipe_gemm_mxfp4_workspace_bytes(*shape) == 0
    for shape in ((1, 255, 64), (1, 256, 16), (-1, 256, 64)):
        with pytest.raises(pt.PipeError) as e:
            pt.pipe_gemm_mxfp4_workspace_bytes(*shape)
        assert e.value.status == pt.PIPE_ERR_SHAPE
    assert pt.pipe_layernorm_backward_workspace_bytes(1, 4096) == 0
    assert pt.pipe_layernorm_backward_workspace_bytes(100, 4096) % (2 * 4 * 4096) == 0
    for name, n in (("pipe_gemm_mxfp4_workspace_bytes", 3), ("pipe_layernorm_backward_workspace_bytes", 2)):
        assert getattr(fns(), name)(*[64] * n, None) == pt.PIPE_ERR_NULL


BF_, F4, E8, U8 = torch.bfloat16, torch.float4_e2m1fn_x2, torch.float8_e8m0fnu, torch.uint8


@pytest.fixture
def as_device(monkeypatch):
    """Host tensors in the place of device tensors, and no call."""
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    linear._setup()
    monkeypatch.setattr(linear, "_fast", None)
    monkeypatch.setattr(linear, "_call", lambda *a, **k: pytest.fail("the call went on"))


def form(rows, K, pitch=None):
    pitch = pitch or -(-K // 32 // 16) * 16
    return torch.zeros(rows, K // 2, dtype=U8).view(F4), torch.zeros(rows, pitch, dtype=U8)[:, :K // 32].view(E8)


def operands():
    x, w = torch.zeros(4, 64, dtype=BF_), torch.ones(64, dtype=BF_)
    A, sa = form(4, 64)
    W, sw = form(8, 64)
    return {
        "layernorm": (pt.pipe_layernorm, (x, w), dict(residual=x), 2),
        "layernorm_backward": (pt.pipe_layernorm_backward, (x, x, w), {}, 3),
        "quantize": (pt.pipe_quantize_mxfp4, (x,), {}, 1),
        "dequantize": (pt.pipe_dequantize_mxfp4, (A, sa), {}, 2),
        "gemm": (pt.pipe_gemm_mxfp4, (A, sa, W, sw), {}, 4),
    }


@pytest.mark.parametrize("wrong", [5, "x", [1.0]])
@pytest.mark.parametrize("name,place", [
    ("layernorm", "bias"), ("layernorm", "y"), ("layernorm", "h"), ("layernorm", "residual"), ("layernorm", "stream"),
    ("layernorm", "out_dtype"), ("layernorm_backward", "dh"), ("layernorm_backward", "dx"), ("layernorm_backward", "dweight"),
    ("layernorm_backward", "dbias"), ("layernorm_backward", "workspace"), ("layernorm_backward", "stream"),
    ("quantize", "codes"), ("quantize", "scales"), ("quantize", "stream"), ("dequantize", "out"), ("dequantize", "out_dtype"),
    ("dequantize", "stream"), ("gemm", "C"), ("gemm", "workspace"), ("gemm", "stream"), ("gemm", "out_dtype"),
])
def test_optional_arguments(as_device, name, place, wrong):
    f, args, more, _ = operands()[name]
    with pytest.raises(TypeError):
        f(*args, **{**more, place: wrong})


@pytest.mark.parametrize("name", list(operands()))
def test_operands_that_are_no_tensors_or_of_other_types(as_device, name):
    f, args, more, count = operands()[name]
    for i in range(count):
        for wrong in (None, 5, "x", args[i].to(torch.float64) if args[i].dtype is BF_ else args[i].view(U8)):
            with pytest.raises(TypeError):
                f(*args[:i], wrong, *args[i + 1:], **more)


def test_shapes_of_the_form(as_device):
    A, sa = form(4, 64)
    W, sw = form(8, 64)
    wide, wide_s = form(8, 96)
    odd = torch.zeros(4, 24, dtype=U8).view(F4)
    x = torch.zeros(4, 64, dtype=BF_)
    for args in ((A, sa, wide, wide_s), (A, sw, W, sw), (A, sa, W, sa), (A, sa[:, :1], W, sw), (odd, sa, W, sw), (A.t(), sa, W, sw)):
        with pytest.raises(ValueError):
            pt.pipe_gemm_mxfp4(*args)
    with pytest.raises(ValueError):
        pt.pipe_gemm_mxfp4(A, sa, W, sw, C=x)
    with pytest.raises(TypeError):
        pt.pipe_gemm_mxfp4(A, sa, W, sw, C=x[:, :8].double())
    with pytest.raises(ValueError):
        pt.pipe_quantize_mxfp4(x[:, :40])
    with pytest.raises(ValueError):
        pt.pipe_layernorm(x[:, :40], x[0, :40], out_dtype=F4)
    with pytest.raises(ValueError):
        pt.pipe_layernorm(x, x[0], y_scales=torch.zeros(4))
    with pytest.raises(ValueError):
        pt.pipe_layernorm(x, x[0], h=x)
    with pytest.raises(TypeError):
        pt.pipe_layernorm(x, x[0], y=torch.zeros(4, 32, dtype=U8).view(F4), out_dtype=BF_)


def test_scales_whose_memory_ends_inside_a_group(as_device):
    """Rows of scales are read 16 bytes at a time: the last row's group must lie in the tensor's memory."""
    A, sa = form(4, 64)
    W, _ = form(8, 64)
    short = torch.zeros(7 * 16 + 2, dtype=U8).as_strided((8, 2), (16, 1)).view(E8)
    with pytest.raises(ValueError, match="16 bytes"):
        pt.pipe_gemm_mxfp4(A, sa, W, short)
    with pytest.raises(ValueError, match="16 bytes"):
        pt.pipe_gemm_mxfp4(A[:1], torch.zeros(1, 2, dtype=U8).view(E8), W, form(8, 64)[1])
    with pytest.raises(ValueError, match="16 bytes"):
        pt.pipe_dequantize_mxfp4(W, short)
