"""The bounds of test_gpu_linear_sums.py reject what they are there for. Without a device: the operators' results are made
here in 64 bits with a planted loss of bits, and the bounds must see it; without the loss they must hold."""
import pytest
import torch

from tests import test_gpu_linear_sums as sums

BF, HF, D = torch.bfloat16, torch.float16, torch.float64


def seen(got, ref, err):
    try:
        sums.check_mean(got, ref, err, "C")
    except AssertionError:
        return True
    return False


@pytest.mark.parametrize("kind", sums.KINDS)
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("M,N,K,G", [(4, 1000, 1024, 64), (40, 500, 2048, 128)])
def test_w4_weights_and_sums_in_16_bits(M, N, K, G, dtype, kind):
    a, w = sums.values(kind, M, N, K, 1, "cpu")
    A = a.to(dtype)
    q, s, z = sums.four_bits(w / K ** 0.5, G, dtype)
    ref, size = sums.w4_reference(A, q, s, z)
    err = size * ((K ** 0.5 + 4) * sums.U)
    assert not seen(ref.to(dtype), ref, err)
    assert not seen(ref.float().to(dtype), ref, err)
    exact = (q - z[:, :, None]).to(D) * s.to(D)[:, :, None]
    rounded = exact.to(dtype).to(D).view(N, K)                      # each weight rounded to 16 bits
    assert seen((A.to(D) @ rounded.t()).to(dtype), ref, err)
    groups = torch.einsum("mgk,ngk->mng", A.to(D).view(M, K // G, G), exact)
    part = torch.zeros(M, N, dtype=D)
    for g in range(K // G):                                         # accumulators of 16 bits
        part = (part + groups[:, :, g]).to(dtype).to(D)
    assert seen(part.to(dtype), ref, err)


@pytest.mark.parametrize("kind", sums.KINDS)
def test_fp8_sums_in_fewer_bits(kind):
    M, N, K = 24, 256, 2048
    a, w = sums.values(kind, M, N, K, 2, "cpu")
    (A, sa), (W, sb) = sums.e4m3_rows(a), sums.e4m3_rows(w)
    scale = sa.to(D)[:, None] * sb.to(D)[None, :]
    groups = torch.einsum("mgk,ngk->mng", A.to(D).view(M, K // 64, 64), W.to(D).view(N, K // 64, 64))
    ref = groups.sum(dim=2) * scale
    squares, linear = sums.largest_of_eights(A, W, torch.arange(M))
    mean = (squares * (7 / 3)).sqrt() * 2.0 ** -13
    if kind == "positive":
        mean = mean + linear * (7 * 2.0 ** -14)
    mag = (A.to(D).abs() @ W.to(D).abs().t()) * scale
    err = mean * scale + mag * (4 * sums.U)
    assert not seen(ref.to(BF), ref, err)
    part = torch.zeros(M, N, dtype=D)
    for g in range(K // 64):
        part = (part + groups[:, :, g]).to(BF).to(D)
    assert seen((part * scale).to(BF), ref, err)
