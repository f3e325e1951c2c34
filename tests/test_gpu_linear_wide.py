"""The norm's gradient for rows wider than 16384, several rows for each workgroup, against the formula in 64 bits."""
import pytest
import torch

from tests.test_gpu_linear import BF, F32, HF, check_grad, normal, padded

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N", [(300, 24584), (520, 32768), (257, 16392), (1, 32768), (9, 20000)])
@pytest.mark.parametrize("dtype,residual,pad", [(BF, True, 8), (HF, False, 0)])
def test_wide_rows(M, N, dtype, residual, pad):
    print(f"[linear wide] {M} {N} {dtype}", flush=True)
    w = (1 + 0.1 * normal((N,), F32, 300)).to(dtype)
    dy, x, dh = (normal((M, N), dtype, seed) for seed in (301, 302, 303))
    if pad:
        dy, x, dh = padded(dy, pad), padded(x, 2 * pad), padded(dh, pad)
    check_grad(dy, x, w, dh if residual else None)
