"""How exact the sums inside the quantised linear layer's products are, on values that exact-integer inputs do not
reach: loud channels, operands of one sign, sums that cancel, long K.

What a sum was before C's rounding shows in the mean: the rounded outputs are whole steps apart, and an error e much
below a step u moves an output to a neighbour with probability |e| / u, so the mean of |got - rounded(reference)| is
the mean of |e|, with a variance of at most the largest step times that sum. The bounds below are the bound B on
sum |e| and six standard deviations, 6 sqrt(u_max B)."""
import pytest
import torch

import async_stage_tile_amd as pt

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
D = torch.float64
BF, HF, F32, E4 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
HALF = {BF: 2.0 ** -8, HF: 2.0 ** -11}


@pytest.fixture(autouse=True)
def _name(request):
    print(f"[linear sums] {request.node.name}", flush=True)
    yield
    torch.cuda.synchronize()


def values(kind, M, N, K, seed, device=DEV):
    """Rows of activations and of weights."""
    g = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device=device, generator=g)

    a, w = normal(M, K), normal(N, K)
    if kind == "positive":
        a, w = a.abs(), w.abs()
    elif kind == "loud":        # every 100th channel 11 times the others
        a[:, ::100] *= 11
    elif kind == "louder":      # every 500th channel 300 times the others
        a[:, ::500] *= 300
    elif kind == "cancelling":  # halves that cancel but for 2 %
        h = K // 2
        a[:, h:2 * h] = a[:, :h]
        w[:, h:2 * h] = -w[:, :h] * (1 + 0.02 * normal(N, h))
    return a, w


def e4m3_rows(v):
    s = v.abs().amax(dim=1) / 448
    return (v / s[:, None]).to(E4), s


def check_mean(got, ref, err, what):
    """got: outputs in 16 bits; ref: in 64 bits; err: what each sum may be off on average (64 bits)."""
    step = 2 * HALF[got.dtype] * float(ref.abs().max())
    total = float(err.sum())
    off = float((got.to(D) - ref.to(got.dtype).to(D)).abs().sum())
    assert off <= total + 6 * (step * total) ** 0.5, \
        f"{what}: {off:.3e} in all, bound {total:.3e} + {6 * (step * total) ** 0.5:.3e}"


# The few-row kernel at both widths, its splits of K, and every tile of the kernel for many rows.
SUM_SHAPES = [(24, 2048, 1040), (60, 1000, 16384), (40, 12400, 512), (150, 4096, 2064), (300, 2000, 8192), (1000, 2000, 1040),
              (2000, 4096, 528), (4096, 4096, 272)]
KINDS = ["normal", "positive", "loud", "louder", "cancelling"]


@pytest.mark.parametrize("M,N,K", SUM_SHAPES + [(1, 8192, 4096), (4, 4096, 1040)])
@pytest.mark.parametrize("kind", KINDS)
def test_fp8_fp16_output_holds_fp32_sums(M, N, K, kind):
    """K roundings of 2^-24 of the partial sums: sqrt(K) of them as independent errors. A partial sum is as large
    as the root of the squared products' sum, or, where all have one sign, as the result."""
    a, w = values(kind, M, N, K, 200)
    (A, sa), (W, sb) = e4m3_rows(a), e4m3_rows(w)
    ref = A.to(D) @ W.to(D).t()
    size = (A.to(D) ** 2 @ (W.to(D) ** 2).t()).sqrt()
    scale = sa.to(D)[:, None] * sb.to(D)[None, :]
    big = float((ref * scale).abs().max())
    sb = sb * (60000 / big if big > 60000 else 1.0)     # within fp16's range
    scale = sa.to(D)[:, None] * sb.to(D)[None, :]
    got = pt.pipe_gemm_fp8(A, sa, W.t(), sb, out_dtype=HF)
    check_mean(got, ref * scale, torch.maximum(size, ref.abs()) * scale * ((K ** 0.5 + 4) * U), "C")


def largest_of_eights(A, W, rows):
    """Sum over the groups of eight k's of the largest product's square, for the given rows of A; and of the largest
    product itself."""
    M, K = A.shape
    a, w = A.float()[rows].view(-1, 1, K // 8, 8), W.float().view(1, -1, K // 8, 8)
    squares, linear = [], []
    for part in range(0, w.shape[1], 64):
        top = (a * w[:, part:part + 64]).abs().amax(dim=3)
        squares.append((top.to(D) ** 2).sum(dim=2))
        linear.append(top.to(D).sum(dim=2))
    return torch.cat(squares, dim=1), torch.cat(linear, dim=1)


@pytest.mark.parametrize("M,N,K", [(24, 512, 1040), (60, 200, 16384), (150, 512, 2064), (300, 264, 8192), (1000, 1000, 400)])
@pytest.mark.parametrize("kind", KINDS)
def test_fp8_bf16_output_holds_13_bits_of_each_eight_products(M, N, K, kind):
    """bf16 C, five rows and more. Of each eight products the largest is exact, the others are off by less than 2^-13
    of it, toward zero. In the worst case these add up. On average they are uniform: as independent errors a third
    of the squares, and their mean of half where all have one sign."""
    a, w = values(kind, M, N, K, 210)
    (A, sa), (W, sb) = e4m3_rows(a), e4m3_rows(w)
    rows = torch.arange(0, M, max(1, M // 24), device=DEV)[:24]
    squares, linear = largest_of_eights(A, W, rows)
    scale = (sa.to(D)[:, None] * sb.to(D)[None, :])[rows]
    ref = (A.to(D)[rows] @ W.to(D).t()) * scale
    mag = (A.to(D).abs()[rows] @ W.to(D).abs().t()) * scale
    got = pt.pipe_gemm_fp8(A, sa, W.t(), sb)[rows]
    worst = linear * scale * (7 * 2.0 ** -13) + mag * (K * 2 * U + 4 * U)
    off = (got.to(D) - ref).abs() - ref.abs() * (HALF[BF] * (1 + 2 ** -10)) - worst * (1 + HALF[BF])
    assert float(off.max()) <= 0
    mean = (squares * (7 / 3)).sqrt() * 2.0 ** -13
    if kind == "positive":
        mean = mean + linear * (7 * 2.0 ** -14)
    check_mean(got, ref, mean * scale + mag * (4 * U), "C")


def four_bits(w, G, dtype):
    """Codes, scales and zero points of weights in groups of G, and the weights that they stand for."""
    N, K = w.shape
    g = w.view(N, K // G, G)
    low, high = g.amin(dim=2).clamp_max(0), g.amax(dim=2).clamp_min(0)
    s = ((high - low) / 15).to(dtype)
    z = (-low / s.float()).round().clamp(0, 15)
    q = ((g / s.float()[:, :, None]).round() + z[:, :, None]).clamp(0, 15)
    return q, s, z


def w4_reference(A, q, s, z, chunk=256):
    """The product in 64 bits, and the size of what its sums pass through: for each group the terms a q and z a and their
    sums, whichever is larger, scaled; the groups' as independent errors."""
    M, (N, groups, G) = A.shape[0], q.shape
    a = A.to(D).view(M, groups, G)
    total, squares = a.sum(dim=2), (a * a).sum(dim=2)
    ref, size = [], []
    for n in range(0, N, chunk):
        Q, S, Z = (t[n:n + chunk].to(D) for t in (q, s, z))
        P = torch.matmul(a.transpose(0, 1).contiguous(), Q.permute(1, 2, 0).contiguous())       # groups, M, N
        terms = torch.matmul((a * a).transpose(0, 1).contiguous(), (Q * Q).permute(1, 2, 0).contiguous())
        S, Z, T = S.t()[:, None, :], Z.t()[:, None, :], total.t()[:, :, None]
        ref.append((S * (P - Z * T)).sum(dim=0))
        part = torch.maximum(terms, P * P) + Z * Z * torch.maximum(squares.t()[:, :, None], T * T)
        size.append((S * S * part).sum(dim=0).sqrt())
    return torch.cat(ref, dim=1), torch.cat(size, dim=1)


# The vector units, the small matrix instructions with both numbers of loads, the tiles of both widths.
W4_SUM_SHAPES = [(1, 4096, 8192, 128), (2, 8200, 4096, 64), (1, 4096, 2048, 32), (4, 2048, 4096, 128), (8, 2056, 4096, 64),
                 (16, 2048, 1024, 32), (40, 2000, 4096, 128), (64, 18432, 512, 64), (200, 1000, 2048, 2048)]


@pytest.mark.parametrize("M,N,K,G", W4_SUM_SHAPES)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_w4_holds_fp32_sums_of_unrounded_weights(M, N, K, G, kind, dtype):
    """K roundings of 2^-24 of the sums that codes and zero points enter apart."""
    a, w = values(kind, M, N, K, 220)
    A = a.to(dtype)
    q, s, z = four_bits(w / K ** 0.5, G, dtype)
    codes = q.to(torch.uint8).view(N, K)
    codes = codes[:, 0::2] | (codes[:, 1::2] << 4)
    ref, size = w4_reference(A, q, s, z)
    got = pt.pipe_gemm_w4(A, codes, s, zeros=z.to(torch.uint8))
    check_mean(got, ref, size * ((K ** 0.5 + 4) * U), "C")
