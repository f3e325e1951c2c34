"""The quantised linear layer's operators against their formulas in 64 bits.

Tolerances are bounds, derived from the arithmetic: a rounding to a type is off
by at most half a step (eps / 2 of the value, and half the smallest step for
values below the normal range); an fp32 sum of n terms in the kernels' order is
off by at most (longest chain of additions) * 2^-24 of the sum of the terms'
magnitudes (2^-23 where the matrix instructions may truncate). Products of
small integers with scales that are powers of two are exact in every step
and have to match bit for bit."""
import pytest
import torch

import async_stage_tile_amd as pt

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
D = torch.float64
BF, HF, F32, E4 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
HALF = {BF: 2.0 ** -8, HF: 2.0 ** -11, F32: 2.0 ** -24, E4: 2.0 ** -4}     # half a step of 1
TINY = {BF: 2.0 ** -134, HF: 2.0 ** -25, F32: 2.0 ** -150, E4: 2.0 ** -10}  # half the smallest step


@pytest.fixture(autouse=True)
def _name(request):
    print(f"[linear] {request.node.name}", flush=True)
    yield
    torch.cuda.synchronize()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(shape, dtype, seed):
    return torch.randn(shape, device=DEV, generator=gen(seed)).to(dtype)


def padded(t, pad):
    """The same matrix as a view of a wider one."""
    wide = torch.full((t.shape[0], t.shape[1] + pad), 0, device=t.device, dtype=torch.float32).to(t.dtype)
    if t.element_size() == 1:
        wide.view(torch.uint8)[:, :t.shape[1]] = t.view(torch.uint8)
    else:
        wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def close(got, ref, tol, what):
    got, ref = got.to(D), ref.to(D)
    assert got.shape == ref.shape, what
    bad = ~((got - ref).abs() <= tol)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()}, worst " \
        f"{float(((got - ref).abs() / tol.clamp_min(1e-300)).max()):.3f} of the bound at {bad.nonzero()[0].tolist()}"


# ---------------------------------------------------------------------------
# RMS norm
# ---------------------------------------------------------------------------
# fp32 chain of a row's sum: at most 32 elements a thread, 6 steps of the wave, 16 waves; r takes
# half of that and a few roundings of its own; h w, its product with r and the scale's a few more.
NORM_U = (32 + 6 + 16) / 2 + 10


def norm_reference(x, w, res, eps):
    h = x if res is None else (x.float() + res.float()).to(x.dtype)
    v = h.to(D)
    r = 1 / torch.sqrt((v * v).mean(dim=1, keepdim=True) + eps)
    return h, v * r * w.to(D)


def check_norm(x, w, res, out, eps=1e-6, **kw):
    h, ref = norm_reference(x, w, res, eps)
    got = pt.pipe_rmsnorm(x, w, residual=res, eps=eps, out_dtype=out, **kw)
    got = list(got) if isinstance(got, tuple) else [got]
    y = got.pop(0)
    if out == E4:
        s = got.pop(0)
        want = ref.abs().amax(dim=1).clamp_min(2.0 ** -100) / 448
        close(s, want, want * (NORM_U * U), "scales")
        ref = ref / want[:, None]
    close(y, ref, ref.abs() * (HALF[out] * (1 + 2 ** -10) + 2 * NORM_U * U) + TINY[out], "y")
    if res is not None:
        assert torch.equal(got.pop(0).view(torch.int16), h.view(torch.int16))
    assert not got


@pytest.mark.parametrize("M,N", [(1, 8), (1, 4096), (3, 504), (5, 520), (4, 1024), (7, 1032), (2, 2048), (3, 2056),
                                 (2, 4104), (1, 8192), (3, 8200), (1, 16384), (2, 16392), (2, 32768), (1021, 256),
                                 (600, 5000)])
@pytest.mark.parametrize("dtype,out,residual", [(BF, BF, True), (HF, HF, False), (BF, E4, True), (HF, E4, False),
                                                (HF, E4, True), (BF, BF, False)])
def test_norm(M, N, dtype, out, residual):
    x = normal((M, N), dtype, 1)
    w = (1 + 0.1 * normal((N,), F32, 2)).to(dtype)
    check_norm(x, w, normal((M, N), dtype, 3) if residual else None, out)


@pytest.mark.parametrize("out", [BF, E4])
def test_norm_strided_in_place_and_given_outputs(out):
    M, N = 37, 1000
    x, res = padded(normal((M, N), BF, 4), 24), padded(normal((M, N), BF, 5), 40)
    w = normal((N,), BF, 6)
    check_norm(x, w, res, out)
    h, ref = norm_reference(x, w, res, 1e-5)
    base = torch.full((M, N + 16), 7.0, device=DEV).to(out)
    y = base[:, :N]
    got = pt.pipe_rmsnorm(x, w, residual=res, eps=1e-5, out_dtype=out, y=y, h=res)
    assert got[0] is y and got[-1] is res
    assert torch.equal(res, h)
    assert bool((base[:, N:].float() == 7).all())          # nothing written past the row
    scale = got[1].to(D)[:, None] if out == E4 else 1.0
    want = ref / scale
    close(y, want, want.abs() * (HALF[out] * (1 + 2 ** -10) + 2 * NORM_U * U) + TINY[out], "y")


def test_norm_special_rows():
    """Zeros, tiny and huge rows, NaN and infinities: row by row, without touching their neighbours."""
    M, N = 8, 2056
    x = normal((M, N), BF, 7)
    x[1] = 0
    x[2] = 1e-30
    x[3] = 1e4
    x[4, 77] = float("nan")
    x[5, 78] = float("inf")
    w = normal((N,), BF, 8)
    y, s = pt.pipe_rmsnorm(x, w, out_dtype=E4)
    y16 = pt.pipe_rmsnorm(x, w)
    good = [0, 1, 2, 3, 6, 7]
    _, ref = norm_reference(x, w, None, 1e-6)
    want = ref.abs().amax(dim=1).clamp_min(2.0 ** -100) / 448
    close(s[good], want[good], want[good] * (NORM_U * U), "scales")
    scaled = ref / want[:, None]
    close(y[good], scaled[good], scaled[good].abs() * (HALF[E4] * (1 + 2 ** -10) + 2 * NORM_U * U) + TINY[E4], "y")
    close(y16[good], ref[good], ref[good].abs() * (HALF[BF] + 2 * NORM_U * U) + TINY[BF], "y16")
    assert bool((y[1].float() == 0).all()) and float(s[1]) == float(torch.tensor(2.0 ** -100) / 448)
    for r in (4, 5):
        assert bool(torch.isnan(s[r])) and bool(torch.isnan(y[r].float()).all())
    assert bool(torch.isnan(y16[4]).all())
    assert bool(torch.isnan(y16[5, 78])) and bool((y16[5, :78] == 0).all())
    w[5] = float("nan")     # a NaN weight makes every row's maximum NaN
    y, s = pt.pipe_rmsnorm(x, w, out_dtype=E4)
    assert bool(torch.isnan(s).all()) and bool(torch.isnan(y.float()).all())


def test_norm_empty_and_refusals():
    w = torch.ones(64, dtype=BF, device=DEV)
    x = torch.ones(4, 64, dtype=BF, device=DEV)
    y, s, h = pt.pipe_rmsnorm(x[:0], w, residual=x[:0], out_dtype=E4)
    assert y.shape == (0, 64) and s.shape == (0,) and h.shape == (0, 64)
    dx, dw = pt.pipe_rmsnorm_backward(x[:0], x[:0], w)
    assert dx.shape == (0, 64) and bool((dw == 0).all())
    with pytest.raises(TypeError):
        pt.pipe_rmsnorm(x, w.half())
    with pytest.raises(TypeError):
        pt.pipe_rmsnorm(x, w, out_dtype=HF)
    with pytest.raises(ValueError):
        pt.pipe_rmsnorm(x, w[:32])
    with pytest.raises(ValueError):
        pt.pipe_rmsnorm(x, w, residual=x[:2])
    with pytest.raises(ValueError):
        pt.pipe_rmsnorm(x.t(), w)
    with pytest.raises(ValueError):
        pt.pipe_rmsnorm(x, w, h=x)
    with pytest.raises(ValueError):
        pt.pipe_rmsnorm(x[0], w)
    with pytest.raises(pt.PipeError) as e:
        pt.pipe_rmsnorm(x[:, :60], w[:60])
    assert e.value.status == pt.PIPE_ERR_SHAPE
    with pytest.raises(pt.PipeError) as e:
        pt.pipe_rmsnorm(x[:, 4:60], w[:56])
    assert e.value.status == pt.PIPE_ERR_ALIGN


# ---------------------------------------------------------------------------
# Gradient
# ---------------------------------------------------------------------------
def grad_reference(dy, x, w, dh, eps):
    """dx, dweight, and the magnitudes that their fp32 errors scale with."""
    v, g = x.to(D), dy.to(D) * w.to(D)
    N = x.shape[1]
    r = 1 / torch.sqrt((v * v).mean(dim=1, keepdim=True) + eps)
    dx = r * g - v * r ** 3 * (g * v).sum(dim=1, keepdim=True) / N
    mag = r * g.abs() + v.abs() * r ** 3 * (g * v).abs().sum(dim=1, keepdim=True) / N
    if dh is not None:
        dx, mag = dx + dh.to(D), mag + dh.to(D).abs()
    return dx, (dy.to(D) * v * r).sum(dim=0), mag, (dy.to(D) * v * r).abs().sum(dim=0)


def check_grad(dy, x, w, dh, eps=1e-6):
    dx, dw, mag, mag_w = grad_reference(dy, x, w, dh, eps)
    got, got_w = pt.pipe_rmsnorm_backward(dy, x, w, dh=dh, eps=eps)
    chain = 3 * NORM_U + 54
    close(got, dx, dx.abs() * HALF[x.dtype] * (1 + 2 ** -10) + mag * (chain * U) + TINY[x.dtype], "dx")
    # a workgroup's rows (256 workgroups or more where there are as many rows, and at least one in 16), its
    # partial's place among the others
    chain = max(x.shape[0] / 256, 16) + 64 + NORM_U
    close(got_w, dw, mag_w * (chain * U) + 1e-300, "dweight")
    again, again_w = pt.pipe_rmsnorm_backward(dy, x, w, dh=dh, eps=eps)
    assert torch.equal(got, again) and torch.equal(got_w, again_w)


@pytest.mark.parametrize("M,N", [(1, 8), (1, 4096), (5, 512), (6, 1000), (5, 2048), (3, 4096), (4, 8200), (2, 16384),
                                 (3, 16400), (2, 32768), (2100, 264), (1500, 2056), (1021, 2048), (16, 512), (17, 512), (18, 4096),
                                 (9, 8192), (700, 5000), (4100, 2056), (4099, 8192), (600, 16384)])
@pytest.mark.parametrize("dtype,residual", [(BF, True), (HF, False), (HF, True)])
def test_grad(M, N, dtype, residual):
    w = (1 + 0.1 * normal((N,), F32, 12)).to(dtype)
    check_grad(normal((M, N), dtype, 10), normal((M, N), dtype, 11), w,
               normal((M, N), dtype, 13) if residual else None)


def test_grad_strided_and_in_place():
    M, N = 70, 776
    dy, x, dh = (padded(normal((M, N), BF, s), p) for s, p in ((14, 8), (15, 16), (16, 24)))
    w = normal((N,), BF, 17)
    check_grad(dy, x, w, dh)
    want, want_w = pt.pipe_rmsnorm_backward(dy, x, w, dh=dh)
    got, got_w = pt.pipe_rmsnorm_backward(dy, x, w, dh=dh, dx=dh)
    assert got is dh and torch.equal(dh, want) and torch.equal(got_w, want_w)


def test_grad_against_differences():
    """dx and dweight against central differences of the 64-bit forward pass, along random directions; the
    difference quotient of step t is off by O(t^2), far below the outputs' rounding."""
    M, N, eps, t = 6, 264, 1e-5, 1e-4
    dy, x, dh = (normal((M, N), HF, s) for s in (20, 21, 22))
    w = normal((N,), HF, 23)
    dx, dw = pt.pipe_rmsnorm_backward(dy, x, w, dh=dh, eps=eps)

    def loss(v, weight):
        r = 1 / torch.sqrt((v * v).mean(dim=1, keepdim=True) + eps)
        return (v * r * weight * dy.to(D)).sum() + (v * dh.to(D)).sum()

    _, _, mag, mag_w = grad_reference(dy, x, w, dh, eps)
    for seed in (24, 25, 26):
        ex, ew = normal((M, N), D, seed), normal((N,), D, seed + 10)
        quot = (loss(x.to(D) + t * ex, w.to(D)) - loss(x.to(D) - t * ex, w.to(D))) / (2 * t)
        tol = ((dx.to(D).abs() * HALF[HF] + mag * (200 * U)) * ex.abs()).sum() + 1e-5
        assert abs(float(quot - (dx.to(D) * ex).sum())) <= float(tol)
        quot = (loss(x.to(D), w.to(D) + t * ew) - loss(x.to(D), w.to(D) - t * ew)) / (2 * t)
        assert abs(float(quot - (dw.to(D) * ew).sum())) <= float((mag_w * (200 * U) * ew.abs()).sum()) + 1e-5


# ---------------------------------------------------------------------------
# e4m3 products
# ---------------------------------------------------------------------------
def small_e4m3(shape, seed):
    return torch.randint(-4, 5, shape, device=DEV, generator=gen(seed)).float().to(E4)


def powers(n, seed):
    return 2.0 ** torch.randint(-3, 4, (n,), device=DEV, generator=gen(seed)).float()


FP8_SHAPES = [(1, 8, 16), (1, 4096, 4096), (2, 24, 48), (15, 264, 400), (16, 256, 128), (17, 248, 1040), (24, 512, 2048),
              (33, 40, 4112), (64, 304, 256), (65, 136, 64), (66, 128, 8192), (128, 256, 4096), (129, 520, 1040),
              (200, 1000, 4112), (300, 2056, 272), (257, 264, 80), (130, 8, 16), (500, 504, 5008),
              (4096, 4104, 192), (4100, 4096, 336), (8192, 2048, 64), (2048, 3904, 272), (700, 2000, 6000),
              (4096, 4096, 400), (8192, 4096, 144), (3, 520, 272), (4, 200, 512), (2, 72, 1040), (32, 13000, 1040),
              (64, 12400, 528), (5, 1000, 16384)]


# Large tiles of every shape at their edges, and the few-row kernel's second and later rows of tiles.
FP8_MORE = [(65, 136, 8256), (129, 520, 9232), (257, 264, 8208), (130, 8, 8224), (500, 504, 13200), (66, 4104, 336),
            (1000, 1000, 400), (600, 2056, 2064), (65, 4088, 8192), (128, 4096, 1040), (1000, 504, 1552), (4100, 40, 80),
            (200, 4096, 1552), (1500, 520, 528), (1300, 2000, 2064), (2000, 4120, 400)]


@pytest.mark.parametrize("M,N,K", FP8_SHAPES + FP8_MORE)
def test_fp8_exact_integers(M, N, K):
    A, W = small_e4m3((M, K), 30), small_e4m3((N, K), 31)
    sa, sb = powers(M, 32), powers(N, 33)
    ref = (A.float().cpu().to(F32) @ W.float().cpu().t()).to(DEV) if M * N * K < 1 << 28 else \
        A.float() @ W.float().t()
    ref = ref * sa[:, None] * sb[None, :]      # integers below 2^24 and powers of two: exact
    for out in (F32, BF, HF):
        got = pt.pipe_gemm_fp8(A, sa, W.t(), sb, out_dtype=out)
        assert got.dtype == out and torch.equal(got, ref.to(out)), out


@pytest.mark.parametrize("M,N,K,out", [(1, 512, 4096, BF), (24, 264, 1040, HF), (50, 512, 512, F32), (200, 264, 4112, BF),
                                       (300, 264, 2048, F32), (4096, 4096, 512, BF)])
def test_fp8_random(M, N, K, out):
    A, W = normal((M, K), F32, 34).mul(30).to(E4), normal((N, K), F32, 35).mul(30).to(E4)
    sa, sb = normal((M,), F32, 36).abs() + 0.1, normal((N,), F32, 37).abs() + 0.1
    scale = sa.to(D)[:, None] * sb.to(D)[None, :]
    ref = (A.to(D) @ W.to(D).t()) * scale
    mag = (A.to(D).abs() @ W.to(D).abs().t()) * scale
    got = pt.pipe_gemm_fp8(A, sa, W.t(), sb, out_dtype=out)
    tol = ref.abs() * HALF[out] * (1 + 2 ** -10) + mag * (K * 2 * U + 4 * U) + TINY[out]
    if out == HF:       # 65520 and more round to infinity in fp16, and some of these products are larger
        over = ref.abs() - tol > 65520
        assert bool(over.any()) and torch.equal(got[over], (ref[over].sign() * float("inf")).to(HF))
        near = (ref.abs() + tol > 65504) & ~over
        assert bool((got[near].float().abs() > 65000).all())
        got, ref, tol = got[~over & ~near], ref[~over & ~near], tol[~over & ~near]
    close(got, ref, tol, "C")
    got = pt.pipe_gemm_fp8(A, sa, W.t(), sb, out_dtype=out)
    assert torch.equal(got, pt.pipe_gemm_fp8(A, sa, W.t(), sb, out_dtype=out))


@pytest.mark.parametrize("M,N,K", [(1, 512, 4096), (24, 512, 4096), (60, 13000, 4096), (150, 512, 4096), (300, 1000, 8192),
                                   (1000, 5000, 1040), (4096, 4096, 528)])
def test_fp8_fp32_sums(M, N, K):
    """fp32 C holds fp32 sums: the errors of K independent roundings add up to sqrt(K) * 2^-24 of the result's
    norm, which sums of fewer bits pass many times over."""
    A, W = normal((M, K), F32, 38).mul(30).to(E4), normal((N, K), F32, 39).mul(30).to(E4)
    one = torch.ones(max(M, N), device=DEV)
    ref = A.to(D) @ W.to(D).t()
    got = pt.pipe_gemm_fp8(A, one[:M], W.t(), one[:N], out_dtype=F32).to(D)
    assert float((got - ref).norm() / ref.norm()) <= K ** 0.5 * U


@pytest.mark.parametrize("M,N,K", [(5, 72, 144), (40, 136, 528), (150, 200, 1040), (4096, 4104, 80)])
def test_fp8_strided(M, N, K):
    """Padded rows whose padding is NaN: nothing past a row's K bytes may enter a sum."""
    A, W = padded(small_e4m3((M, K), 40), 48), padded(small_e4m3((N, K), 41), 16)
    for t in (A, W):
        wide = torch.as_strided(t.view(torch.uint8), (t.shape[0], t.stride(0)), (t.stride(0), 1))
        wide[:, t.shape[1]:] = 0x7F
    sa, sb = powers(M + 3, 42)[3:], powers(N + 1, 43)[1:]
    ref = (A.float() @ W.float().t()) * sa[:, None] * sb[None, :]
    base = torch.full((M, N + 24), 5.0, device=DEV)
    got = pt.pipe_gemm_fp8(A, sa, W.t(), sb, C=base[:, :N])
    assert torch.equal(got, ref) and bool((base[:, N:] == 5).all())


def test_fp8_nan_stays_in_its_row_and_column():
    for M in (3, 40, 150):
        N, K = 200, 272
        A, W = small_e4m3((M, K), 44), small_e4m3((N, K), 45)
        one = torch.ones(max(M, N), device=DEV)
        ref = A.float() @ W.float().t()
        A.view(torch.uint8)[1, 100] = 0x7F
        W.view(torch.uint8)[7, 200] = 0x7F
        got = pt.pipe_gemm_fp8(A, one[:M], W.t(), one[:N], out_dtype=F32)
        bad = torch.isnan(got)
        assert bool(bad[1].all()) and bool(bad[:, 7].all())
        bad[1] = True
        bad[:, 7] = True
        assert torch.equal(got[~bad], ref[~bad])


def test_fp8_empty_and_refusals():
    e, f = small_e4m3((8, 64), 46), torch.ones(64, device=DEV)
    assert pt.pipe_gemm_fp8(e[:0], f[:0], e.t(), f[:8]).shape == (0, 8)
    z = pt.pipe_gemm_fp8(e[:, :0], f[:8], e[:, :0].t(), f[:8], out_dtype=F32)
    assert z.shape == (8, 8) and bool((z == 0).all())
    with pytest.raises(TypeError):
        pt.pipe_gemm_fp8(e, f[:8], e.t(), f[:8], out_dtype=E4)
    with pytest.raises(ValueError):
        pt.pipe_gemm_fp8(e, f[:8], e, f[:8])               # row-major B
    with pytest.raises(ValueError):
        pt.pipe_gemm_fp8(e, f[:7], e.t(), f[:8])
    with pytest.raises(ValueError):
        pt.pipe_gemm_fp8(e, f[:16:2], e.t(), f[:8])
    with pytest.raises(ValueError):
        pt.pipe_gemm_fp8(e, f[:8], small_e4m3((8, 80), 1).t(), f[:8])
    with pytest.raises(pt.PipeError) as err:
        pt.pipe_gemm_fp8(e[:, 8:56], f[:8], e[:, 8:56].t(), f[:8])
    assert err.value.status == pt.PIPE_ERR_ALIGN


# ---------------------------------------------------------------------------
# 4-bit products
# ---------------------------------------------------------------------------
def codes_of(N, K, seed):
    q = torch.randint(0, 16, (N, K), device=DEV, generator=gen(seed), dtype=torch.uint8)
    return q, q[:, 0::2] | (q[:, 1::2] << 4)


def w4_weights(q, z, s, G):
    N, K = q.shape
    v = q.view(N, K // G, G).to(D) - (8.0 if z is None else z.to(D)[:, :, None])
    return (v * s.to(D)[:, :, None]).view(N, K)


W4_SHAPES = [(1, 8, 32, 32), (1, 264, 4096, 128), (1, 504, 1024, 64), (2, 24, 96, 32), (3, 40, 192, 64), (5, 136, 2048, 32),
             (16, 256, 256, 256), (17, 248, 640, 128), (7, 72, 288, 288), (24, 264, 1056, 32), (32, 40, 4096, 64),
             (33, 520, 1152, 128), (47, 120, 4096, 64), (64, 304, 512, 512), (65, 200, 544, 32), (200, 136, 768, 256),
             (1, 512, 8192, 8192), (9, 128, 64, 64), (64, 64, 2080, 32)]


@pytest.mark.parametrize("M,N,K,G", W4_SHAPES)
@pytest.mark.parametrize("dtype,zeros", [(BF, True), (HF, False), (BF, False), (HF, True)])
def test_w4_exact_integers(M, N, K, G, dtype, zeros):
    A = torch.randint(-4, 5, (M, K), device=DEV, generator=gen(50)).to(dtype)
    q, codes = codes_of(N, K, 51)
    s = (2.0 ** torch.randint(-2, 1, (N, K // G), device=DEV, generator=gen(52)).float()).to(dtype)
    z = torch.randint(0, 16, (N, K // G), device=DEV, generator=gen(53), dtype=torch.uint8) if zeros else None
    ref = A.to(D) @ w4_weights(q, z, s, G).t()      # multiples of 1/4 below 2^22: exact in fp32 too
    assert torch.equal(pt.pipe_gemm_w4(A, codes, s, zeros=z), ref.to(dtype))


# Wide layers, whose tiles are of 128 weight rows, also for three and four rows of many weights.
W4_WIDE = [(5, 16520, 288, 32), (20, 16648, 256, 128), (33, 16456, 640, 64), (40, 16648, 512, 128), (64, 16400, 1056, 32),
           (200, 5000, 320, 64), (3, 12312, 8192, 128), (4, 49160, 2080, 32), (5, 16520, 1600, 32),
           (2, 4120, 8224, 32)]


# Two to eight rows: one or two turns through K, blocks that K leaves empty, both numbers of loads, ends of N.
W4_FEW = [(2, 2056, 4096, 64), (3, 2072, 4608, 128), (4, 4104, 96, 32), (5, 2064, 160, 32), (6, 72, 8256, 64),
          (7, 4112, 256, 256), (8, 1000, 5120, 128), (8, 3000, 8192, 1024), (4, 8, 32, 32), (2, 40, 64, 64), (1, 2056, 1024, 64), (1, 4104, 256, 32),
          (1, 24, 4128, 32), (1, 4104, 4096, 128), (2, 33000, 1024, 128), (1, 5000, 18432, 256)]


@pytest.mark.parametrize("M,N,K,G", W4_WIDE + W4_FEW)
@pytest.mark.parametrize("dtype,zeros", [(BF, True), (HF, False)])
def test_w4_wide_exact_integers(M, N, K, G, dtype, zeros):
    test_w4_exact_integers(M, N, K, G, dtype, zeros)


@pytest.mark.parametrize("M,N,K,G", [(1, 512, 4096, 128), (13, 264, 2048, 32), (30, 136, 1024, 64), (60, 264, 4096, 128)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_w4_random(M, N, K, G, dtype):
    A = normal((M, K), dtype, 54)
    q, codes = codes_of(N, K, 55)
    s = (0.01 * (normal((N, K // G), F32, 56).abs() + 0.1)).to(dtype)
    z = torch.randint(4, 12, (N, K // G), device=DEV, generator=gen(57), dtype=torch.uint8)
    ref = A.to(D) @ w4_weights(q, z, s, G).t()
    # codes and zero points enter apart: magnitudes |a| (q + z) s
    big = ((q.view(N, K // G, G).to(D) + z.to(D)[:, :, None]) * s.to(D)[:, :, None]).view(N, K)
    mag = A.to(D).abs() @ big.t()
    got = pt.pipe_gemm_w4(A, codes, s, zeros=z)
    close(got, ref, ref.abs() * HALF[dtype] * (1 + 2 ** -10) + mag * (K * 2 * U + 8 * U) + TINY[dtype], "C")
    assert torch.equal(got, pt.pipe_gemm_w4(A, codes, s, zeros=z))


@pytest.mark.parametrize("M,G", [(1, 32), (20, 64), (50, 128)])
def test_w4_strided(M, G):
    """Padded rows: codes, scales and activations past a row are NaN or 255 and must not be read into a sum."""
    N, K, dtype = 104, 640, BF
    A = torch.randint(-4, 5, (M, K), device=DEV, generator=gen(58)).to(dtype)
    q, codes = codes_of(N, K, 59)
    s = (2.0 ** torch.randint(-2, 1, (N, K // G), device=DEV, generator=gen(60)).float()).to(dtype)
    z = torch.randint(0, 16, (N, K // G), device=DEV, generator=gen(61), dtype=torch.uint8)

    def wide(t, pad, fill):
        w = torch.full((t.shape[0], t.shape[1] + pad), fill, device=DEV, dtype=t.dtype)
        w[:, :t.shape[1]] = t
        return w[:, :t.shape[1]]

    nan = float("nan")
    ref = (A.to(D) @ w4_weights(q, z, s, G).t()).to(dtype)
    base = torch.full((M, N + 8), 3.0, device=DEV, dtype=dtype)
    got = pt.pipe_gemm_w4(wide(A, 24, nan), wide(codes, 48, 255), wide(s, 3, nan), zeros=wide(z, 5, 255),
                          C=base[:, :N])
    assert torch.equal(got, ref) and bool((base[:, N:] == 3).all())


def test_w4_special_values_stay_in_their_rows():
    N, K, G = 72, 320, 64
    for M in (3, 20, 40):
        A = torch.randint(-4, 5, (M, K), device=DEV, generator=gen(62)).to(HF)
        q, codes = codes_of(N, K, 63)
        s = torch.ones((N, K // G), device=DEV, dtype=HF)
        ref = (A.to(D) @ w4_weights(q, None, s, G).t()).to(HF)
        A[1, 70] = float("nan")
        s[9, 2] = float("inf")
        got = pt.pipe_gemm_w4(A, codes, s)
        assert bool(torch.isnan(got[1]).all()) and not bool(torch.isfinite(got[:, 9]).any())
        keep = torch.ones_like(got, dtype=torch.bool)
        keep[1] = False
        keep[:, 9] = False
        assert torch.equal(got[keep], ref[keep])


def test_w4_empty_and_refusals():
    A = torch.ones(4, 64, dtype=BF, device=DEV)
    c = torch.zeros(8, 32, dtype=torch.uint8, device=DEV)
    s = torch.ones(8, 2, dtype=BF, device=DEV)
    assert pt.pipe_gemm_w4(A[:0], c, s).shape == (0, 8)
    z = pt.pipe_gemm_w4(A[:, :0], c[:, :0], s[:, :0])
    assert z.shape == (4, 8) and bool((z == 0).all())
    with pytest.raises(TypeError):
        pt.pipe_gemm_w4(A, c, s.half())
    with pytest.raises(TypeError):
        pt.pipe_gemm_w4(A, c.to(torch.int8), s)
    with pytest.raises(ValueError):
        pt.pipe_gemm_w4(A, c[:, :16], s)
    with pytest.raises(ValueError):
        pt.pipe_gemm_w4(A, c, s[:4])
    with pytest.raises(ValueError):
        pt.pipe_gemm_w4(A, c, s, zeros=c[:, :1])
    with pytest.raises(pt.PipeError) as err:
        pt.pipe_gemm_w4(A, c, torch.ones(8, 4, dtype=BF, device=DEV))    # groups of 16
    assert err.value.status == pt.PIPE_ERR_SHAPE


# ---------------------------------------------------------------------------
# Streams, graphs, long extents
# ---------------------------------------------------------------------------
def _layer_inputs(M=100, N=512, K=4096, seed=70):
    x, res, dy = (normal((M, K), BF, seed + i) for i in range(3))
    w = normal((K,), BF, seed + 3)
    W, sb = small_e4m3((N, K), seed + 4), powers(N, seed + 5)
    q, codes = codes_of(N, K, seed + 6)
    s = normal((N, K // 64), BF, seed + 7)
    return x, res, dy, w, W, sb, codes, s


def _layer(x, res, dy, w, W, sb, codes, s, stream=None):
    y, ys, h = pt.pipe_rmsnorm(x, w, residual=res, out_dtype=E4, stream=stream)
    y16 = pt.pipe_rmsnorm(h, w, stream=stream)
    C = pt.pipe_gemm_fp8(y, ys, W.t(), sb, stream=stream)
    C4 = pt.pipe_gemm_w4(y16[:40], codes, s, stream=stream)
    dx, dw = pt.pipe_rmsnorm_backward(dy, h, w, dh=res, stream=stream)
    return y.float(), ys, h, C, C4, dx, dw


def test_operators_on_a_side_stream():
    ins = _layer_inputs()
    want = _layer(*ins)
    assert pt.pipe_gemm_fp8_workspace_bytes(100, 512, 4096) > 0    # the workspace too is held for the side stream
    torch.cuda.synchronize()
    side = torch.cuda.Stream(device=DEV)
    side.wait_stream(torch.cuda.current_stream())
    got = _layer(*ins, stream=side)[1:]
    for _ in range(8):
        torch.full((1 << 20,), 7.0, device=DEV).add_(1.0)
    side.synchronize()
    torch.cuda.synchronize()
    for a, b in zip(got, want[1:]):
        assert torch.equal(a, b)


def test_operators_captured_and_replayed():
    ins = _layer_inputs(seed=80)
    x = ins[0]
    _layer(*ins)
    torch.cuda.synchronize()
    side = torch.cuda.Stream(device=DEV)
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            outs = _layer(*ins)
    torch.cuda.current_stream().wait_stream(side)
    for seed in (90, 91, 92, 93):
        x.copy_(normal(tuple(x.shape), BF, seed))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = _layer(*ins)
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b), seed


def test_offsets_past_32_bits():
    """Operands of more than 4 GiB: rows at both ends against the same rows alone."""
    M, N = 70000, 32768
    x = torch.empty((M, N), dtype=BF, device=DEV)
    x[:] = normal((1, N), BF, 100)
    x[-3:] = normal((3, N), BF, 101)
    w = normal((N,), BF, 102)
    y = pt.pipe_rmsnorm(x, w)
    assert torch.equal(y[-3:], pt.pipe_rmsnorm(x[-3:].clone(), w)) and torch.equal(y[:1], y[M - 4:M - 3])
    del x, y
    N, K = 300000, 16384
    W = torch.empty((N, K), dtype=torch.uint8, device=DEV)
    W[:] = small_e4m3((1, K), 103).view(torch.uint8)
    W[-16:] = small_e4m3((16, K), 104).view(torch.uint8)
    one = torch.ones(N, device=DEV)
    for M in (2, 80):
        A = small_e4m3((M, K), 105)
        got = pt.pipe_gemm_fp8(A, one[:M], W.view(E4).t(), one, out_dtype=F32)
        assert torch.equal(got[:, -16:], A.float() @ W[-16:].view(E4).float().t())
        assert torch.equal(got[:, 0], got[:, N - 17])
    A = torch.randint(-4, 5, (3, 2 * K), device=DEV, generator=gen(106)).to(HF)
    s = torch.full((N, 2), 2.0 ** -6, device=DEV, dtype=HF)
    got = pt.pipe_gemm_w4(A, W, s)
    q = torch.stack([W[-16:] & 15, W[-16:] >> 4], dim=2).view(16, 2 * K)
    assert torch.equal(got[:, -16:], (A.to(D) @ w4_weights(q, None, s[-16:], K).t()).to(HF))
    assert torch.equal(got[:, 0], got[:, N - 17])
