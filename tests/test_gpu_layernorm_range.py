"""Layer norm and its gradient on bf16 rows of very large finite values.

A row whose squared deviations add up past fp32's range has r = 0 and u = 0: y is the bias and dx the residual stream's gradient
alone, as for a row of zeros, with which each is compared bit for bit. What infinities come up on the way (a sum
of values, of deviations or of their products with dy) must not reach the outputs, nor the rows beside it."""
import pytest
import torch

import async_stage_tile_amd as pt
from tests.test_gpu_layernorm import BF, D, DEV, E4, F4, HALF, TINY, UP, close, grad_reference, norm_reference, normal

pytestmark = pytest.mark.gpu
LOW, HIGH = torch.finfo(BF).min, torch.finfo(BF).max


@pytest.fixture(autouse=True)
def _name(request):
    print(f"[layernorm range] {request.node.name}", flush=True)
    yield
    torch.cuda.synchronize()


def large_rows(N):
    """Rows of finite values whose squared deviations pass fp32's range, a plain row after each."""
    base = normal((10, N), BF, 1).float()
    base[0, N // 3] = LOW                       # a mask's value
    base[1, ::3] = LOW                          # many of them: the values' sum passes the range too
    base[2, :N // 2] = LOW
    base[3, 1], base[3, N - 2] = HIGH, LOW
    base[4, ::2], base[4, 1::2] = HIGH, LOW
    base[5, :-1] = HIGH
    base[5, -1] = LOW
    base[6] *= 1e28
    base[7] *= 1e30
    base[8] = (base[8] * 1e38).clamp(LOW, HIGH)
    base[9] = base[9] * 1e-3 * HIGH + 0.9 * HIGH
    rows = torch.stack([base.clamp(LOW, HIGH).to(BF), normal((10, N), BF, 2)], dim=1).flatten(0, 1)
    assert bool(torch.isfinite(rows).all())
    return rows


def raw(t):
    return t.contiguous().view(torch.uint8)


WIDTHS = (8, 512, 1000, 1024, 2048, 4096, 5000, 8192, 16384, 24000, 32768)


@pytest.mark.parametrize("N", WIDTHS)
@pytest.mark.parametrize("out,residual,bias", [(BF, False, True), (BF, True, False), (E4, True, True), (F4, False, True)])
def test_norm(N, out, residual, bias):
    if out == F4:
        N = max(N // 32 * 32, 32)
    x = large_rows(N)
    small = x.clone()
    small[0::2] = 0
    w, b = normal((N,), BF, 3), normal((N,), BF, 4) if bias else None
    res = torch.zeros_like(x) if residual else None
    got = pt.pipe_layernorm(x, w, b, residual=res, out_dtype=out)
    want = pt.pipe_layernorm(small, w, b, residual=res, out_dtype=out)
    if residual:
        assert torch.equal(got[-1], x)
        got, want = got[:-1], want[:-1]
    for g, v in zip(got if isinstance(got, tuple) else (got,), want if isinstance(want, tuple) else (want,)):
        assert torch.equal(raw(g), raw(v))


@pytest.mark.parametrize("N", WIDTHS)
@pytest.mark.parametrize("M", (20, 300, 4200))
@pytest.mark.parametrize("residual", (True, False))
def test_grad(M, N, residual):
    if M * N > 1 << 24:
        M = 300
    x = large_rows(N).repeat(-(-M // 20), 1)[:M]
    small = x.clone()
    small[0::2] = 0
    w, dy = normal((N,), BF, 5), 3 * normal((M, N), BF, 6)
    dh = normal((M, N), BF, 7) if residual else None
    got = pt.pipe_layernorm_backward(dy, x, w, dh=dh)
    want = pt.pipe_layernorm_backward(dy, small, w, dh=dh)
    assert torch.equal(got[0][1::2], want[0][1::2])
    assert torch.equal(got[0][0::2], dh[0::2] if residual else torch.zeros_like(got[0][0::2]))
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])


@pytest.mark.parametrize("N", (1000, 4096, 8192, 20000))
def test_rows_whose_squares_just_fit(N):
    """Deviations of 5e16 and of 1e17: the sums of their squares stay below 2^128, so the formula holds as elsewhere."""
    x = normal((6, N), BF, 8)
    x[1] *= 5e16
    x[3] *= 1e17
    x[4] = (x[4].float() * 1e15 + 1e17).to(BF)
    assert float((x.to(D) ** 2).sum(dim=1).max()) < 2.0 ** 127.9
    w, b, dy = normal((N,), BF, 9), normal((N,), BF, 10), normal((6, N), BF, 11)
    _, ref, tol = norm_reference(x, w, b, None, 1e-5)
    close(pt.pipe_layernorm(x, w, b), ref, ref.abs() * HALF[BF] + tol * UP + TINY[BF], "y")
    dx, dw, db, tol, tol_w, tol_b = grad_reference(dy, x, w, None, 1e-5)
    got = pt.pipe_layernorm_backward(dy, x, w)
    close(got[0], dx, dx.abs() * HALF[BF] * UP + tol * UP + TINY[BF], "dx")
    close(got[1], dw, tol_w, "dweight")
    close(got[2], db, tol_b, "dbias")
