"""The products at row counts next to the end of 32 bits, where the last tile's rows end past it. The rows at that end are
checked, and as many at the start."""
import pytest
import torch

import async_stage_tile_amd as pt

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
END = (1 << 31) - 1


@pytest.fixture(autouse=True)
def _memory(request):
    torch.cuda.empty_cache()
    free = torch.cuda.mem_get_info()[0]
    if free < 200 << 30:
        pytest.skip(f"{free >> 30} GiB of device memory free, 200 needed")
    print(f"[linear extent] {request.node.name}", flush=True)
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def small(shape, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(-4, 5, shape, device=DEV, generator=g).float()


@pytest.mark.parametrize("M", [END, END - 70])
def test_fp8_rows_to_the_end_of_32_bits(M):
    N, K, tail = 8, 16, 400
    A = torch.zeros((M, K), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    a, w = small((tail, K), 1), small((N, K), 2)
    A.view(torch.uint8)[-tail:] = a.to(torch.float8_e4m3fn).view(torch.uint8)
    scales = torch.ones(M, device=DEV)
    scales[-tail:] = 2.0 ** torch.arange(tail, device=DEV).remainder(7)
    C = pt.pipe_gemm_fp8(A, scales, w.to(torch.float8_e4m3fn).t(), torch.ones(N, device=DEV))
    assert torch.equal(C[-tail:], ((a @ w.t()) * scales[-tail:, None]).to(torch.bfloat16))
    assert not bool(C[:tail].any())


def test_w4_rows_to_the_end_of_32_bits():
    M, N, K, tail = END, 8, 32, 400
    A = torch.zeros((M, K), dtype=torch.bfloat16, device=DEV)
    A[-tail:] = small((tail, K), 3).to(torch.bfloat16)
    q = small((N, K), 4).add(8).to(torch.uint8)
    C = pt.pipe_gemm_w4(A, q[:, 0::2] | (q[:, 1::2] << 4), torch.ones((N, 1), dtype=torch.bfloat16, device=DEV))
    assert torch.equal(C[-tail:], (A[-tail:].float() @ (q.float() - 8).t()).to(torch.bfloat16))
    assert not bool(C[:tail].any())
