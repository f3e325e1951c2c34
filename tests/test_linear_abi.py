"""Checks of the quantised linear layer's entry points that need no GPU: the
header's functions are exported and bound, and bad arguments are refused before
anything reaches the device (the addresses below are never dereferenced)."""
import ctypes
import os
import re

import pytest
import torch

import async_stage_tile_amd as pt
from async_stage_tile_amd import linear
from tests.conftest import ROOT

P = 0x10000
BF, HF, F32, E4 = pt.PIPE_BF16, pt.PIPE_FP16, pt.PIPE_FP32, pt.PIPE_E4M3


def fns():
    return linear._setup()


def test_every_declared_function_is_exported_and_bound():
    txt = open(os.path.join(ROOT, "include", "pipe_linear.h")).read()
    txt = re.sub(r"/\*.*?\*/", "", txt, flags=re.S)
    declared = sorted(set(re.findall(r"\b(pipe_[a-z0-9_]+)\s*\(", txt)))
    assert declared == sorted(pt.linear_symbols())
    for name in declared:
        assert hasattr(pt.lib(), name)
    limit = re.search(r"#define PIPE_RMSNORM_MAX_N (\d+)", txt).group(1)
    assert int(limit) == pt.PIPE_RMSNORM_MAX_N


def norm(x=P, res=0, w=P, y=P, s=0, h=0, M=4, N=64, ldx=64, ldr=64, ldy=64, ldh=64, eps=1e-6, t=BF, o=BF):
    return fns().pipe_rmsnorm(x, res, w, y, s, h, M, N, ldx, ldr, ldy, ldh, eps, t, o, None)


@pytest.mark.parametrize("change,status", [
    (dict(t=F32, o=F32), pt.PIPE_ERR_CONFIG), (dict(t=E4, o=E4), pt.PIPE_ERR_CONFIG),
    (dict(t=BF, o=HF), pt.PIPE_ERR_CONFIG), (dict(t=9, o=9), pt.PIPE_ERR_CONFIG),
    (dict(eps=-1.0), pt.PIPE_ERR_CONFIG), (dict(eps=float("nan")), pt.PIPE_ERR_CONFIG),
    (dict(M=-1), pt.PIPE_ERR_SHAPE), (dict(N=-8), pt.PIPE_ERR_SHAPE),
    (dict(N=63), pt.PIPE_ERR_SHAPE), (dict(M=1 << 31), pt.PIPE_ERR_SHAPE),
    (dict(N=pt.PIPE_RMSNORM_MAX_N + 8, ldx=1 << 20, ldy=1 << 20), pt.PIPE_ERR_SHAPE),
    (dict(ldx=56), pt.PIPE_ERR_SHAPE), (dict(ldy=56), pt.PIPE_ERR_SHAPE),
    (dict(ldx=1 << 40), pt.PIPE_ERR_SHAPE),
    (dict(x=0), pt.PIPE_ERR_NULL), (dict(w=0), pt.PIPE_ERR_NULL), (dict(y=0), pt.PIPE_ERR_NULL),
    (dict(res=P), pt.PIPE_ERR_NULL), (dict(h=P), pt.PIPE_ERR_NULL),
    (dict(o=E4), pt.PIPE_ERR_NULL),
    (dict(x=P + 8), pt.PIPE_ERR_ALIGN), (dict(y=P + 8), pt.PIPE_ERR_ALIGN),
    (dict(w=P + 2), pt.PIPE_ERR_ALIGN), (dict(ldx=68), pt.PIPE_ERR_ALIGN),
    (dict(o=E4, s=P, y=P + 4), pt.PIPE_ERR_ALIGN), (dict(o=E4, s=P + 2), pt.PIPE_ERR_ALIGN),
    (dict(res=P, h=P + 8), pt.PIPE_ERR_ALIGN), (dict(res=P, h=P, ldr=72, ldh=60), pt.PIPE_ERR_SHAPE),
    (dict(M=0, x=0, y=0, w=0), pt.PIPE_OK), (dict(N=0, x=0, y=0, w=0), pt.PIPE_OK),
])
def test_rmsnorm_refusals(change, status):
    assert norm(**change) == status


def grad(dy=P, x=P, w=P, dh=0, dx=P, dw=P, M=4, N=64, lddy=64, ldx=64, lddh=64, lddx=64, eps=1e-6, t=BF,
         ws=P, wsb=1 << 30):
    return fns().pipe_rmsnorm_backward(dy, x, w, dh, dx, dw, M, N, lddy, ldx, lddh, lddx, eps, t, ws, wsb, None)


@pytest.mark.parametrize("change,status", [
    (dict(t=F32), pt.PIPE_ERR_CONFIG), (dict(eps=-1.0), pt.PIPE_ERR_CONFIG),
    (dict(N=60), pt.PIPE_ERR_SHAPE), (dict(M=-4), pt.PIPE_ERR_SHAPE), (dict(lddx=8), pt.PIPE_ERR_SHAPE),
    (dict(dy=0), pt.PIPE_ERR_NULL), (dict(x=0), pt.PIPE_ERR_NULL), (dict(dx=0), pt.PIPE_ERR_NULL),
    (dict(w=0), pt.PIPE_ERR_NULL), (dict(dw=0), pt.PIPE_ERR_NULL),
    (dict(dw=P + 4), pt.PIPE_ERR_ALIGN), (dict(dh=P + 2), pt.PIPE_ERR_ALIGN),
    (dict(dh=P, lddh=68), pt.PIPE_ERR_ALIGN), (dict(M=100, ws=P + 4), pt.PIPE_ERR_ALIGN),
    (dict(M=100, ws=0), pt.PIPE_ERR_WORKSPACE), (dict(M=100, wsb=16), pt.PIPE_ERR_WORKSPACE),
    (dict(N=0, dw=0, dy=0), pt.PIPE_OK),
])
def test_rmsnorm_backward_refusals(change, status):
    assert grad(**change) == status


def fp8(A=P, sa=P, B=P, sb=P, C=P, M=4, N=64, K=64, lda=64, ldb=64, ldc=64, o=BF, ws=0, wsb=0):
    return fns().pipe_gemm_fp8(A, sa, B, sb, C, M, N, K, lda, ldb, ldc, o, ws, wsb, None)


@pytest.mark.parametrize("change,status", [
    (dict(o=E4), pt.PIPE_ERR_CONFIG), (dict(o=-1), pt.PIPE_ERR_CONFIG),
    (dict(N=60), pt.PIPE_ERR_SHAPE), (dict(K=56), pt.PIPE_ERR_SHAPE), (dict(K=-16), pt.PIPE_ERR_SHAPE),
    (dict(lda=48), pt.PIPE_ERR_SHAPE), (dict(ldb=48), pt.PIPE_ERR_SHAPE), (dict(ldc=56), pt.PIPE_ERR_SHAPE),
    (dict(M=1 << 31), pt.PIPE_ERR_SHAPE),
    (dict(M=(1 << 31) - 1, N=(1 << 31) - 8, ldc=1 << 31), pt.PIPE_ERR_SHAPE),
    (dict(A=0), pt.PIPE_ERR_NULL), (dict(B=0), pt.PIPE_ERR_NULL), (dict(C=0), pt.PIPE_ERR_NULL),
    (dict(sa=0), pt.PIPE_ERR_NULL), (dict(sb=0), pt.PIPE_ERR_NULL),
    (dict(A=P + 8), pt.PIPE_ERR_ALIGN), (dict(lda=72), pt.PIPE_ERR_ALIGN), (dict(ldb=72), pt.PIPE_ERR_ALIGN),
    (dict(C=P + 8), pt.PIPE_ERR_ALIGN), (dict(ldc=68), pt.PIPE_ERR_ALIGN), (dict(sa=P + 1), pt.PIPE_ERR_ALIGN),
    (dict(M=0, A=0), pt.PIPE_OK), (dict(N=0, A=0), pt.PIPE_OK),
])
def test_gemm_fp8_refusals(change, status):
    assert fp8(**change) == status


def test_gemm_fp8_workspace():
    """Where a shape needs a workspace, a missing or short one is refused."""
    M, N, K = 128, 256, 8192
    need = pt.pipe_gemm_fp8_workspace_bytes(M, N, K)
    assert need > 0 and need % (4 * M * N) == 0
    kw = dict(M=M, N=N, K=K, lda=K, ldb=K, ldc=N)
    assert fp8(**kw) == pt.PIPE_ERR_WORKSPACE
    assert fp8(ws=P, wsb=need - 1, **kw) == pt.PIPE_ERR_WORKSPACE
    assert fp8(ws=P + 4, wsb=need, **kw) == pt.PIPE_ERR_ALIGN
    assert pt.pipe_gemm_fp8_workspace_bytes(1, 256, 8192) == 0
    assert pt.pipe_gemm_fp8_workspace_bytes(0, 256, 8192) == 0
    with pytest.raises(pt.PipeError) as e:
        pt.pipe_gemm_fp8_workspace_bytes(1, 255, 64)
    assert e.value.status == pt.PIPE_ERR_SHAPE
    for name, n in (("pipe_gemm_fp8_workspace_bytes", 3), ("pipe_gemm_w4_workspace_bytes", 3), ("pipe_rmsnorm_backward_workspace_bytes", 2)):
        assert getattr(fns(), name)(*[64] * n, None) == pt.PIPE_ERR_NULL


def w4(A=P, q=P, s=P, z=0, C=P, M=4, N=64, K=256, G=64, lda=256, ldq=128, lds=4, ldz=4, ldc=64, t=BF,
       ws=0, wsb=0):
    return fns().pipe_gemm_w4(A, q, s, z, C, M, N, K, G, lda, ldq, lds, ldz, ldc, t, ws, wsb, None)


@pytest.mark.parametrize("change,status", [
    (dict(t=F32), pt.PIPE_ERR_CONFIG), (dict(t=E4), pt.PIPE_ERR_CONFIG),
    (dict(N=60), pt.PIPE_ERR_SHAPE), (dict(K=240, G=240), pt.PIPE_ERR_SHAPE), (dict(M=-1), pt.PIPE_ERR_SHAPE),
    (dict(G=16), pt.PIPE_ERR_SHAPE), (dict(G=96, K=288), pt.PIPE_ERR_SHAPE), (dict(G=0), pt.PIPE_ERR_SHAPE),
    (dict(G=512), pt.PIPE_ERR_SHAPE), (dict(G=-64), pt.PIPE_ERR_SHAPE),
    (dict(lda=248), pt.PIPE_ERR_SHAPE), (dict(ldq=112), pt.PIPE_ERR_SHAPE), (dict(lds=3), pt.PIPE_ERR_SHAPE),
    (dict(z=P, ldz=3), pt.PIPE_ERR_SHAPE), (dict(ldc=56), pt.PIPE_ERR_SHAPE),
    (dict(A=0), pt.PIPE_ERR_NULL), (dict(q=0), pt.PIPE_ERR_NULL), (dict(s=0), pt.PIPE_ERR_NULL),
    (dict(C=0), pt.PIPE_ERR_NULL),
    (dict(A=P + 8), pt.PIPE_ERR_ALIGN), (dict(q=P + 8), pt.PIPE_ERR_ALIGN), (dict(ldq=136), pt.PIPE_ERR_ALIGN),
    (dict(lda=260), pt.PIPE_ERR_ALIGN), (dict(s=P + 1), pt.PIPE_ERR_ALIGN), (dict(C=P + 4), pt.PIPE_ERR_ALIGN),
    (dict(M=0, A=0), pt.PIPE_OK), (dict(N=0, q=0), pt.PIPE_OK),
])
def test_gemm_w4_refusals(change, status):
    assert w4(**change) == status


def test_gemm_w4_workspace():
    M, N, K = 40, 256, 4096
    need = pt.pipe_gemm_w4_workspace_bytes(M, N, K)
    assert need > 0 and need % (4 * M * N) == 0
    kw = dict(M=M, N=N, K=K, G=128, lda=K, ldq=K // 2, lds=32, ldc=N)
    assert w4(**kw) == pt.PIPE_ERR_WORKSPACE
    assert w4(ws=P, wsb=need - 1, **kw) == pt.PIPE_ERR_WORKSPACE
    assert w4(ws=P + 8, wsb=need, **kw) == pt.PIPE_ERR_ALIGN
    assert pt.pipe_gemm_w4_workspace_bytes(1, N, K) == 0


def test_wrappers_refuse_host_tensors_and_wrong_types():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.ones(64, dtype=torch.bfloat16)
    f = torch.ones(64)
    with pytest.raises(ValueError):
        pt.pipe_rmsnorm(x, w)
    with pytest.raises(TypeError):
        pt.pipe_rmsnorm(x.float(), w)
    with pytest.raises(TypeError):
        pt.pipe_rmsnorm("x", w)
    with pytest.raises(ValueError):
        pt.pipe_rmsnorm_backward(x, x, w)
    e = torch.zeros(4, 64, dtype=torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        pt.pipe_gemm_fp8(e, f[:4], e.t(), f[:4])
    with pytest.raises(TypeError):
        pt.pipe_gemm_fp8(x, f[:4], e.t(), f[:4])
    with pytest.raises(ValueError):
        pt.pipe_gemm_w4(x, torch.zeros(8, 32, dtype=torch.uint8), x[:, :1])
    with pytest.raises(TypeError):
        pt.pipe_gemm_w4(x.float(), torch.zeros(8, 32, dtype=torch.uint8), x[:, :1])


def test_binding_is_built_and_hands_back_what_it_does_not_take():
    """The C++ marshalling is in place (the build makes it), and gives host tensors, other types and other
    arguments back to the Python wrappers, without an error set."""
    linear._setup()
    fast = linear._fast
    assert fast is not None
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.ones(64, dtype=torch.bfloat16)
    e, f = torch.zeros(4, 64, dtype=torch.float8_e4m3fn), torch.ones(4)
    q = torch.zeros(8, 32, dtype=torch.uint8)
    for args in ((x, w, None, 1e-6, None), (None, w, None, 1e-6, None), (x, w, x, "eps", "type"), (x[0], w, None, 1e-6, None)):
        assert fast.rmsnorm(*args) is NotImplemented
    for args in ((x, x, w, None, 1e-6), (1, 2, 3, 4, 5)):
        assert fast.rmsnorm_backward(*args) is NotImplemented
    for args in ((e, f, e.t(), f, None), (x, f, e.t(), f, None), (e, f, e, f, 3)):
        assert fast.gemm_fp8(*args) is NotImplemented
    for args in ((x, q, x[:, :1], None), (x, None, None, None)):
        assert fast.gemm_w4(*args) is NotImplemented
    assert fast.gemm_w4(x) is NotImplemented and fast.rmsnorm() is NotImplemented
    with pytest.raises(TypeError):
        fast.bind(None)
    with pytest.raises(ValueError):
        fast.bind(None, 0, 0, 0, 0, 0, 0, 0)
