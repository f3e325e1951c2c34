"""More shapes of the microscaled 4-bit product, on both sides of rules that choose a kernel's tiles."""
import pytest
import torch

import async_stage_tile_amd as pt
from tests.test_gpu_mxfp4 import BF, F32, HF, SHAPES, operand, values

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _name(request):
    print(f"[mxfp4 shapes] {request.node.name}", flush=True)
    yield
    torch.cuda.synchronize()


def check_exact(M, N, K):
    """Scales of 1/2, 1 and 2: every sum is a multiple of 1/16; where the sums of magnitudes stay below 2^20 they are
    exact in fp32 in any order."""
    (A, sa), (W, sw) = operand(M, K, 10), operand(N, K, 11)
    a, w = values(A, sa).float(), values(W, sw).float()
    assert float((a.abs() @ w.abs().t()).max()) < 2 ** 20 * (1 - 2 ** -8)      # fp32 sums of magnitudes, off by less
    ref = a @ w.t()
    for out in (F32, BF, HF):
        got = pt.pipe_gemm_mxfp4(A, sa, W, sw, out_dtype=out)
        assert got.dtype == out and torch.equal(got, ref.to(out)), out


@pytest.mark.parametrize("M,N,K", [(3, 8192, 544), (3, 8200, 544), (24, 8192, 4128), (24, 8200, 4128), (32, 10240, 96),
                                   (33, 8192, 1056), (33, 8200, 1056), (64, 11008, 2080), (64, 12288, 64), (64, 12296, 64),
                                   (17, 9216, 16416), (64, 16384, 416)])
def test_few_rows_by_columns(M, N, K):
    """Tiles of 32 columns up to 8192, of 64 past them."""
    check_exact(M, N, K)


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_sums_that_are_compared_bit_for_bit_are_exact(M, N, K):
    """What makes every order of adding up right in test_exact_sums: all its sums of magnitudes stay below 2^20."""
    (A, sa), (W, sw) = operand(M, K, 10), operand(N, K, 11)
    a, w = values(A, sa).float().abs(), values(W, sw).float().abs()
    assert float((a @ w.t()).max()) < 2 ** 20 * (1 - 2 ** -8)      # its fp32 sums are off by less
