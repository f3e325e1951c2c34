"""Layer norm and its gradient in every shape of workgroup and on both sides of the size up to which rows stay in the
last-level cache. Calls past it are compared bit for bit with calls on some of their rows alone (a row's y, h and dx do not
depend on the others), the gradient's sums over the rows with 64-bit ones."""
import pytest
import torch

import async_stage_tile_amd as pt
from tests.test_gpu_layernorm import BF, E4, F32, F4, HF, check_grad, check_norm, normal

pytestmark = pytest.mark.gpu
KEPT = 128 << 20       # bytes of a call that stay


@pytest.fixture(autouse=True)
def _name(request):
    print(f"[layer shapes] {request.node.name}", flush=True)
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def rows_past(N, sides):
    return KEPT // (2 * N * sides) + 5


def ends(M):
    return slice(0, 5), slice(M // 2, M // 2 + 3), slice(M - 5, M)


def raw(t):
    return t.contiguous().view(torch.uint8)


@pytest.mark.parametrize("N", (512, 1024, 2048, 4096, 6144, 8192, 16384, 32768))
@pytest.mark.parametrize("residual", (True, False))
@pytest.mark.parametrize("dtype", (BF, HF))
def test_norm_past_the_cache(N, residual, dtype):
    M = rows_past(N, 4 if residual else 2)
    x = normal((M, N), dtype, 1) + 0.5
    res = normal((M, N), dtype, 2) if residual else None
    w, b = normal((N,), dtype, 3), normal((N,), dtype, 4)
    for out in (dtype, E4, F4):
        got = pt.pipe_layernorm(x, w, b, residual=res, out_dtype=out)
        for e in ends(M):
            want = pt.pipe_layernorm(x[e], w, b, residual=None if res is None else res[e], out_dtype=out)
            pairs = zip(got, want) if isinstance(got, tuple) else ((got, want),)
            assert all(torch.equal(raw(g[e]), raw(v)) for g, v in pairs), (out, e)


@pytest.mark.parametrize("M,N", [(4096, 8192), (8192, 8192), (1100, 32768)])
@pytest.mark.parametrize("dtype", (BF, HF))
@pytest.mark.parametrize("eighths", (True, False))
def test_norm_past_the_cache_by_its_formula(M, N, dtype, eighths):
    w = (1 + 0.1 * normal((N,), F32, 5)).to(dtype)
    check_norm(normal((M, N), dtype, 6) + 0.5, w, normal((N,), dtype, 7), normal((M, N), dtype, 8), E4 if eighths else dtype)


@pytest.mark.parametrize("N", (512, 1024, 2048, 4096, 8192, 16384, 32768, 20008))
@pytest.mark.parametrize("residual", (True, False))
@pytest.mark.parametrize("dtype", (BF, HF))
def test_grad_past_the_cache(N, residual, dtype):
    M = rows_past(N, 4 if residual else 3)
    dy, x = normal((M, N), dtype, 9), normal((M, N), dtype, 10) - 0.5
    dh = normal((M, N), dtype, 11) if residual else None
    w = (1 + 0.1 * normal((N,), F32, 12)).to(dtype)
    check_grad(dy, x, w, dh)
    dx = pt.pipe_layernorm_backward(dy, x, w, dh=dh)[0]
    for e in ends(M):
        assert torch.equal(dx[e], pt.pipe_layernorm_backward(dy[e], x[e], w, dh=None if dh is None else dh[e])[0])


@pytest.mark.parametrize("M,N", [(4095, 512), (4096, 512), (4097, 8), (4100, 64), (9001, 264), (9000, 512), (9001, 8), (4095, 8)])
@pytest.mark.parametrize("dtype,residual", [(BF, True), (HF, False), (HF, True), (BF, False)])
def test_grad_of_many_narrow_rows(M, N, dtype, residual):
    """Four rows a workgroup below 4096 rows of up to 512, eight from there on."""
    w = (1 + 0.1 * normal((N,), F32, 13)).to(dtype)
    check_grad(normal((M, N), dtype, 14), normal((M, N), dtype, 15) - 0.5, w, normal((M, N), dtype, 16) if residual else None)


@pytest.mark.parametrize("N", (512, 1024, 2016, 4096, 5024, 8192, 16384, 20000, 32768))
@pytest.mark.parametrize("dtype,out", [(HF, HF), (HF, E4), (BF, E4), (HF, F4), (BF, F4)])
def test_rows_do_not_depend_on_the_others(N, dtype, out):
    M = 9000 if N <= 4096 else 2500
    x, res, dy = (normal((M, N), dtype, s) for s in (17, 18, 19))
    w, b = normal((N,), dtype, 20), normal((N,), dtype, 21)
    y = pt.pipe_layernorm(x, w, b, residual=res, out_dtype=out)
    dx = pt.pipe_layernorm_backward(dy, x, w, dh=res)[0]
    for rows in (1, 40, 300, 1021, 2049):
        got = pt.pipe_layernorm(x[:rows], w, b, residual=res[:rows], out_dtype=out)
        assert all(torch.equal(raw(g), raw(v[:rows])) for g, v in zip(got, y)), rows
        if out == dtype:
            assert torch.equal(pt.pipe_layernorm_backward(dy[:rows], x[:rows], w, dh=res[:rows])[0], dx[:rows]), rows
