"""Operands past 4 GiB and pitches near 2^24: offsets of layer norm's and the microscaled 4-bit form's kernels beyond 32 bits.
The rows at both ends are compared with those of a call on these rows alone."""
import pytest
import torch

import async_stage_tile_amd as pt
from tests.test_gpu_mxfp4 import BF, DEV, E8, F4, F32, U8, gen, normal, operand, values

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _name(request):
    print(f"[extent] {request.node.name}", flush=True)
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def filled(rows, columns, dtype, seed):
    """A large matrix of few random rows, each 4099th one the same."""
    small = normal((4099, columns), dtype, seed)
    t = torch.empty(rows, columns, dtype=dtype, device=DEV)
    for i in range(0, rows, 4099):
        t[i:i + 4099] = small[:min(4099, rows - i)]
    return t


def test_norm_and_conversion_of_large_matrices():
    M, N = 560_003, 4096       # 4.3 GiB
    x = filled(M, N, BF, 1)
    w, b = normal((N,), BF, 2), normal((N,), BF, 3)
    ends = (slice(0, 5), slice(M - 5, M), slice(M // 2, M // 2 + 3))
    y, h = pt.pipe_layernorm(x, w, b, residual=x)
    c, s = pt.pipe_quantize_mxfp4(x)
    back = pt.pipe_dequantize_mxfp4(c, s)
    y4, s4 = pt.pipe_layernorm(x, w, b, out_dtype=F4)
    for e in ends:
        part = x[e].contiguous()
        want = pt.pipe_layernorm(part, w, b, residual=part)
        assert torch.equal(y[e], want[0]) and torch.equal(h[e], want[1])
        cw, sw = pt.pipe_quantize_mxfp4(part)
        assert torch.equal(c.view(U8)[e], cw.view(U8)) and torch.equal(s.view(U8)[e], sw.view(U8))
        assert torch.equal(back[e], pt.pipe_dequantize_mxfp4(cw, sw))
        yw, tw = pt.pipe_layernorm(part, w, b, out_dtype=F4)
        assert torch.equal(y4.view(U8)[e], yw.view(U8)) and torch.equal(s4.view(U8)[e], tw.view(U8))
    del y, h, c, s, back, y4, s4
    dx, dw, db = pt.pipe_layernorm_backward(x, x, w, dh=x)
    for e in ends:
        part = x[e].contiguous()
        assert torch.equal(dx[e], pt.pipe_layernorm_backward(part, part, w, dh=part)[0])
    assert bool(torch.isfinite(dw).all()) and bool(torch.isfinite(db).all())


@pytest.mark.parametrize("M,N", [(1_100_000, 64), (8, 1_100_008), (1, 1_100_008), (40, 1_100_008)])
def test_product_of_large_operands(M, N):
    """4.2 GiB of codes on one side."""
    K = 8192
    big = torch.randint(0, 256, (1021, K // 2), dtype=torch.int16, device=DEV, generator=gen(4)).to(U8)
    scale = torch.randint(126, 129, (1021, K // 32), dtype=torch.int16, device=DEV, generator=gen(5)).to(U8)
    rows = max(M, N)
    codes, scales = torch.empty(rows, K // 2, dtype=U8, device=DEV), torch.empty(rows, K // 32, dtype=U8, device=DEV)
    for i in range(0, rows, 1021):
        codes[i:i + 1021] = big[:min(1021, rows - i)]
        scales[i:i + 1021] = scale[:min(1021, rows - i)]
    small = operand(min(M, N), K, 6)
    large = (codes.view(F4), scales.view(E8))
    C = pt.pipe_gemm_mxfp4(*(large if M > N else small), *(small if M > N else large), out_dtype=F32)
    a, w = values(big.view(F4), scale.view(E8)).float(), values(*small).float()
    want = a @ w.t() if M > N else w @ a.t()
    for i in (0, rows // 1021 // 2 * 1021, rows // 1021 * 1021 - 1021):
        got = C[i:i + 1021] if M > N else C[:, i:i + 1021]
        assert torch.equal(got, want), i
    last = rows % 1021
    assert torch.equal(C[-last:] if M > N else C[:, -last:], want[:last] if M > N else want[:, :last])


@pytest.mark.parametrize("M,N", [(257, 136), (130, 264), (70, 40)])
def test_product_of_rows_far_apart(M, N):
    """Pitches just below 2^24 bytes, of codes and of scales: a tile's rows lie up to 4 GiB apart."""
    K, pitch = 1056, (1 << 24) - 16
    (A, sa), (W, sw) = operand(M, K, 7), operand(N, K, 8)
    want = values(A, sa).float() @ values(W, sw).float().t()

    def apart(t, rows, kind):
        wide = torch.empty((rows - 1) * pitch + 1024, dtype=U8, device=DEV).as_strided((rows, t.shape[1]), (pitch, 1))
        wide.copy_(t.view(U8))
        return wide.view(kind)

    got = pt.pipe_gemm_mxfp4(apart(A, M, F4), apart(sa, M, E8), W, sw, out_dtype=F32)
    assert torch.equal(got, want)
    got = pt.pipe_gemm_mxfp4(A, sa, apart(W, N, F4), apart(sw, N, E8), out_dtype=F32)
    assert torch.equal(got, want)


def test_large_product_on_another_stream():
    """The largest kind of product, whose scales are laid out anew first, on streams of its own, and captured."""
    M, N, K = 4096, 4096, 16416
    (A, sa), (W, sw) = operand(M, K, 9), operand(N, K, 10)
    assert pt.pipe_gemm_mxfp4_workspace_bytes(M, N, K) > 0
    want = pt.pipe_gemm_mxfp4(A, sa, W, sw)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = [pt.pipe_gemm_mxfp4(A, sa, W, sw, stream=s) for s in streams]
        torch.cuda.synchronize()
        assert all(torch.equal(g, want) for g in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = pt.pipe_gemm_mxfp4(A, sa, W, sw)
    for turn in range(3):
        A.view(U8).bitwise_xor_(0x88)      # every sign changes
        eager = pt.pipe_gemm_mxfp4(A, sa, W, sw).clone()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(captured, eager) and torch.equal(captured.abs(), want.abs())
