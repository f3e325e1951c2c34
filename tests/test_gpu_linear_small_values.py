"""Operands and results below the normal range of their types: no kernel may take them for zeros. Small integers times the
type's smallest step are exact in every product and sum here, and the results have to match bit for bit."""
import pytest
import torch

import async_stage_tile_amd as pt
from tests.test_gpu_linear import BF, D, E4, F32, HF, codes_of, gen, normal, w4_weights

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
STEP = {HF: 2.0 ** -24, BF: 2.0 ** -133, E4: 2.0 ** -9}


@pytest.fixture(autouse=True)
def _name(request):
    print(f"[linear small values] {request.node.name}", flush=True)
    yield
    torch.cuda.synchronize()


def small(shape, seed):
    return torch.randint(-4, 5, shape, device=DEV, generator=gen(seed)).to(D)


@pytest.mark.parametrize("M,N,K", [(1, 264, 256), (3, 264, 2048), (24, 520, 1040), (60, 1000, 512), (200, 520, 4112), (1500, 520, 528)])
@pytest.mark.parametrize("out", [F32, BF, HF])
def test_fp8_operands(M, N, K, out):
    """Both operands below 2^-6, results of whole steps of 2^-18 below 2^-2."""
    a, w = small((M, K), 400), small((N, K), 401)
    A, W = (a * STEP[E4]).float().to(E4), (w * STEP[E4]).float().to(E4)
    assert torch.equal(A.to(D), a * STEP[E4])
    one = torch.ones(max(M, N), device=DEV)
    got = pt.pipe_gemm_fp8(A, one[:M], W.t(), one[:N], out_dtype=out)
    assert torch.equal(got, (a @ w.t() * STEP[E4] ** 2).to(out))


@pytest.mark.parametrize("M,N,K,G", [(1, 4096, 8192, 128), (2, 8200, 4096, 64), (1, 264, 1024, 32), (3, 264, 1024, 64), (8, 520, 2048, 128),
                                     (16, 264, 512, 32), (40, 520, 1024, 64), (64, 18432, 512, 128)])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("zeros", [True, False])
def test_w4_activations(M, N, K, G, dtype, zeros):
    """Activations of whole steps below the normal range. bf16's products with scales of 1 are below it too: scales of
    2^20 bring the results into it."""
    a = small((M, K), 402)
    A = (a * STEP[dtype]).to(F32).to(dtype)
    assert torch.equal(A.to(D), a * STEP[dtype])
    q, codes = codes_of(N, K, 403)
    up = 2.0 ** 20 if dtype is BF else 1.0
    s = (up * 2.0 ** torch.randint(-2, 1, (N, K // G), device=DEV, generator=gen(404)).float()).to(dtype)
    z = torch.randint(0, 16, (N, K // G), device=DEV, generator=gen(405), dtype=torch.uint8) if zeros else None
    ref = a @ w4_weights(q, z, s, G).t() * STEP[dtype]
    assert torch.equal(pt.pipe_gemm_w4(A, codes, s, zeros=z), ref.to(F32).to(dtype))


@pytest.mark.parametrize("dtype", [BF, HF])
def test_norm_of_small_rows(dtype):
    """Rows of the smallest steps: eps carries the factor, and outputs below the normal range keep their steps."""
    M, N, eps = 5, 2056, 1e-6
    v = small((M, N), 406) * STEP[dtype]
    x = v.to(F32).to(dtype)
    w = torch.full((N,), 2.0, device=DEV).to(dtype)
    y = pt.pipe_rmsnorm(x, w, eps=eps)
    r = 1 / torch.sqrt((v * v).mean(dim=1, keepdim=True) + eps)
    ref = v * r * 2
    half = {BF: 2.0 ** -8, HF: 2.0 ** -11}[dtype]
    assert bool(((y.to(D) - ref).abs() <= ref.abs() * (half + 2.0 ** -20) + STEP[dtype] / 2 * (1 + 2.0 ** -20)).all())
