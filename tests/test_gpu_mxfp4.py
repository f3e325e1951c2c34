"""The microscaled 4-bit form and its product against their definitions in 64 bits.

Bringing values into the form and back is exact but for the rounding to the code (and to fp16), so those have to match bit
for bit. So do products whose sums are exact in fp32. Others are off by at most the fp32 additions: a block's 32 products
add up exactly, then at most (K / 32 + joins) additions, each 2^-23 of the sum of the magnitudes (the matrix instructions
may truncate), and the rounding of C."""
import pytest
import torch

import async_stage_tile_amd as pt

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
D = torch.float64
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
F4, E8, U8 = torch.float4_e2m1fn_x2, torch.float8_e8m0fnu, torch.uint8
HALF = {BF: 2.0 ** -8, HF: 2.0 ** -11, F32: 2.0 ** -24}
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
NAN = float("nan")


@pytest.fixture(autouse=True)
def _name(request):
    print(f"[mxfp4] {request.node.name}", flush=True)
    yield
    torch.cuda.synchronize()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(shape, dtype, seed):
    return torch.randn(shape, device=DEV, generator=gen(seed)).to(dtype)


def same(a, b):
    """The same values, NaN in the same places."""
    return a.dtype == b.dtype and a.shape == b.shape and bool(((a == b) | (torch.isnan(a) & torch.isnan(b))).all())


def nibbles(codes):
    c = codes.view(U8)
    return torch.stack([c & 15, c >> 4], dim=2).flatten(1)


def pack(nib):
    return (nib[:, 0::2] | (nib[:, 1::2] << 4)).view(F4)


def scale_view(bytes_, pad=16, fill=255):
    """e8m0 scales in rows that start at multiples of 16 bytes; what lies between is `fill`: NaN."""
    rows, blocks = bytes_.shape
    wide = torch.full((rows, -(-blocks // 16) * 16 + (pad - 16)), fill, dtype=U8, device=DEV)
    wide[:, :blocks] = bytes_
    return wide[:, :blocks].view(E8)


def values(codes, scales):
    """What the form stands for, in 64 bits."""
    table = torch.tensor(E2M1 + [-v for v in E2M1], dtype=D, device=DEV)
    s = scales.view(U8).to(D)
    p = torch.where(s == 255, NAN, torch.exp2(s - 127))     # pow() on the GPU rounds some powers of two
    return table[nibbles(codes).long()] * p.repeat_interleave(32, dim=1)


def quantised(x):
    """(codes a nibble each, scale bytes) of x by the definition, borders counted one by one."""
    v = x.to(D).unflatten(1, (-1, 32))
    top = v.abs().amax(dim=2)
    bad = ~torch.isfinite(v).all(dim=2)
    e = torch.floor(torch.log2(torch.where(bad | (top == 0), 1.0, top))) - 2
    e = torch.where(top == 0, -127.0, e).clamp(-127, 127)
    a = v.abs() / torch.exp2(e[:, :, None])
    n = torch.zeros_like(a, dtype=U8)
    for border, even_up in ((0.25, 0), (0.75, 1), (1.25, 0), (1.75, 1), (2.5, 0), (3.5, 1), (5.0, 0)):
        n += (a >= border) if even_up else (a > border)
    n += 8 * torch.signbit(v).to(U8)
    return n.flatten(1), torch.where(bad, 255, e + 127).to(U8)


def check_quantise(x, **kw):
    codes, scales = pt.pipe_quantize_mxfp4(x, **kw)
    n, s = quantised(x)
    assert codes.dtype == F4 and scales.dtype == E8 and codes.shape == (x.shape[0], x.shape[1] // 2)
    assert torch.equal(scales.view(U8), s)
    good = (s != 255).repeat_interleave(32, dim=1)
    assert torch.equal(nibbles(codes)[good], n[good])
    return codes, scales


@pytest.mark.parametrize("M,K", [(1, 32), (3, 64), (5, 96), (7, 512), (2, 4128), (33, 1056), (1021, 2080), (300, 8192), (4, 16384),
                                 (1, 65536), (2049, 32)])
@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_quantise(M, K, dtype):
    x = normal((M, K), F32, 1) * 2.0 ** torch.randint(-12, 12, (M, 1), device=DEV, generator=gen(2)).float()
    x[:, ::5] *= 30
    x = x.to(dtype)
    codes, scales = check_quantise(x)
    assert scales.stride(0) % 16 == 0
    want = values(codes, scales)
    for out in (BF, HF, F32):
        assert same(pt.pipe_dequantize_mxfp4(codes, scales, out_dtype=out), want.float().to(out))


@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_quantise_borders_and_special_values(dtype):
    """Every border between two codes and its neighbours, zeros of both signs, the type's largest, smallest and subnormal
    values, NaN and infinities: each in blocks of its own, beside a block that stays as it is."""
    info = torch.finfo(dtype)
    rows = []
    base = torch.tensor([0.0, 0.25, 0.5, 0.75, 1.0, 1.25, 1.5, 1.75, 2.0, 2.5, 3.0, 3.5, 4.0, 5.0, 6.0, 7.0], dtype=dtype)
    for shift in (-8, 0, 5):
        b = base * 2.0 ** shift
        up = torch.nextafter(b.float(), torch.tensor(9e9)) if dtype == F32 else (b.view(torch.int16) + 1).view(dtype)
        down = torch.where(b > 0, torch.nextafter(b.float(), torch.tensor(-9e9)) if dtype == F32 else
                           (b.view(torch.int16) - 1).view(dtype).where(b > 0, b), b)
        rows += [torch.cat([b, -b]), torch.cat([up.to(dtype), -up.to(dtype)]), torch.cat([down.to(dtype), -down.to(dtype)])]
    zero = torch.zeros(32, dtype=dtype)
    rows += [zero, -zero]
    sub = info.smallest_normal * info.eps     # the smallest subnormal
    for v in (info.max, info.smallest_normal, sub, 3 * sub, 7.99 * info.smallest_normal, 4 * info.smallest_normal):
        r = zero.clone()
        r[3], r[9], r[30] = v, -v / 3, v / 8
        rows.append(r)
    for v in (NAN, float("inf"), -float("inf")):
        r = torch.arange(32).to(dtype)
        r[17] = v
        rows.append(r)
    block = torch.stack(rows).to(DEV)
    plain = normal((len(rows), 32), dtype, 3)
    codes, scales = check_quantise(torch.cat([plain, block, plain], dim=1))
    assert bool((scales.view(U8)[:, 1][-3:] == 255).all()) and bool((scales.view(U8)[:, 1][:-3] != 255).all())
    assert bool((scales.view(U8)[:, 0] != 255).all())
    back = pt.pipe_dequantize_mxfp4(codes, scales, out_dtype=F32)
    assert bool(torch.isnan(back[-3:, 32:64]).all()) and not bool(torch.isnan(back[:-3]).any())


def test_dequantise_every_code_and_scale():
    """All codes with all scales: fp32 and bf16 hold every value within their range, fp16 rounds and overflows."""
    nib = torch.arange(16, dtype=U8, device=DEV).repeat(2).repeat(256, 1)
    s = scale_view(torch.arange(256, dtype=U8, device=DEV)[:, None])
    want = values(pack(nib), s)
    for out in (F32, BF, HF):
        got = pt.pipe_dequantize_mxfp4(pack(nib), s, out_dtype=out)
        assert same(got, want.to(F32).to(out))
    # Nothing is rounded up to 6 * 2^125 (scale 252); 2 * 2^127 = 2^128 is past fp32.
    assert torch.equal(pt.pipe_dequantize_mxfp4(pack(nib), s, out_dtype=F32)[:253].to(D), want[:253])


def test_conversions_strided_and_given():
    M, K = 21, 1056
    wide = torch.zeros(M, K + 40, device=DEV, dtype=BF)
    wide[:, :K] = normal((M, K), BF, 4)
    x = wide[:, :K]
    want = check_quantise(x)
    c = torch.full((M, K // 2 + 32), 5, dtype=U8, device=DEV)
    s = torch.full((M, 64), 6, dtype=U8, device=DEV)
    codes, scales = c[:, :K // 2].view(F4), s[:, :K // 32].view(E8)
    got = pt.pipe_quantize_mxfp4(x, codes=codes, scales=scales)
    assert got[0] is codes and got[1] is scales
    assert torch.equal(codes.view(U8), want[0].view(U8)) and torch.equal(scales.view(U8), want[1].view(U8))
    assert bool((c[:, K // 2:] == 5).all()) and bool((s[:, K // 32:] == 6).all())
    out = torch.full((M, K + 8), 9.0, device=DEV)
    assert pt.pipe_dequantize_mxfp4(codes, scales, out=out[:, :K]).data_ptr() == out.data_ptr()
    assert torch.equal(out[:, :K].to(D), values(*want)) and bool((out[:, K:] == 9).all())


def test_empty():
    x = torch.ones(4, 64, dtype=BF, device=DEV)
    for part, shape in ((x[:0], (0, 64)), (x[:, :0], (4, 0))):
        codes, scales = pt.pipe_quantize_mxfp4(part)
        assert codes.shape == (shape[0], shape[1] // 2) and scales.shape == (shape[0], shape[1] // 32)
        assert pt.pipe_dequantize_mxfp4(codes, scales).shape == shape
    A, sa = pt.pipe_quantize_mxfp4(x)
    W, sw = pt.pipe_quantize_mxfp4(normal((8, 64), BF, 5))
    none = pt.pipe_quantize_mxfp4(x[:0])
    assert pt.pipe_gemm_mxfp4(*none, W, sw).shape == (0, 8)
    assert pt.pipe_gemm_mxfp4(A, sa, *none).shape == (4, 0)
    for out in (BF, F32):
        C = torch.full((4, 16), 3.0, dtype=out, device=DEV)
        k0 = pt.pipe_quantize_mxfp4(x[:, :0])
        w0 = pt.pipe_quantize_mxfp4(torch.ones(8, 0, dtype=BF, device=DEV))
        pt.pipe_gemm_mxfp4(*k0, *w0, C=C[:, :8])
        assert bool((C[:, :8] == 0).all()) and bool((C[:, 8:] == 3).all())


# ---------------------------------------------------------------------------
# Product
# ---------------------------------------------------------------------------
def operand(rows, K, seed, spread=1, pad_codes=0):
    """Random codes, scales of 2^-spread .. 2^spread, NaN between the rows of scales; the codes' rows padded."""
    nib = torch.randint(0, 16, (rows, K), dtype=U8, device=DEV, generator=gen(seed))
    s = torch.randint(127 - spread, 128 + spread, (rows, K // 32), device=DEV, generator=gen(seed + 1000)).to(U8)
    codes = pack(nib).view(U8)
    if pad_codes:
        wide = torch.randint(0, 256, (rows, K // 2 + pad_codes), dtype=torch.int16, device=DEV, generator=gen(seed + 1)).to(U8)
        wide[:, :K // 2] = codes
        codes = wide[:, :K // 2]
    return codes.view(F4), scale_view(s, pad=16 + pad_codes)


SHAPES = [(1, 8, 32), (1, 4096, 4096), (2, 24, 96), (3, 520, 544), (4, 200, 512), (2, 72, 1056), (1, 16, 1024), (4, 40, 8192),
          (5, 8, 32), (15, 264, 416), (16, 256, 128), (17, 248, 1056), (24, 512, 2048), (33, 40, 4128), (64, 304, 256),
          (65, 136, 64), (66, 128, 8192), (128, 256, 4096), (129, 520, 1056), (200, 1000, 4128), (300, 2056, 288), (257, 264, 96),
          (130, 8, 32), (500, 504, 5024), (4096, 4104, 192), (4100, 4096, 352), (8192, 2048, 64), (2048, 3904, 288),
          (700, 2000, 6016), (4096, 4096, 416), (8192, 4096, 160), (32, 13000, 1056), (64, 12400, 544), (5, 1000, 16384),
          (65, 136, 16416), (129, 520, 18464), (257, 264, 16416), (130, 8, 16448), (500, 504, 26432), (66, 4104, 352),
          (1000, 1000, 416), (600, 2056, 4128), (65, 4088, 16384), (128, 4096, 2080), (1000, 504, 3104), (4100, 40, 96),
          (200, 4096, 3104), (1500, 520, 1056), (1300, 2000, 4128), (2000, 4120, 800), (24, 512, 16416), (40, 1000, 9248),
          (6, 4096, 9216), (4104, 4096, 992), (4096, 4096, 4128), (1021, 5000, 1056), (20, 20000, 544), (64, 16640, 1056),
          (8190, 8200, 4192), (4096, 4096, 16416), (2, 512, 96), (2, 88, 4128), (3, 20000, 96), (2, 20008, 1056), (4, 8, 16384)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_exact_sums(M, N, K):
    """Scales of 1/2, 1 and 2: every sum is a multiple of 1/16 and below 2^20, exact in fp32 in any order."""
    (A, sa), (W, sw) = operand(M, K, 10), operand(N, K, 11)
    a, w = values(A, sa), values(W, sw)
    assert K * 144 < 2 ** 24 or float((a.abs() @ w.abs().t()[:, :8]).max()) < 2 ** 19
    ref = a.float() @ w.float().t()
    for out in (F32, BF, HF):
        got = pt.pipe_gemm_mxfp4(A, sa, W, sw, out_dtype=out)
        assert got.dtype == out and torch.equal(got, ref.to(out)), out


@pytest.mark.parametrize("M,N,K,out", [(1, 512, 4096, BF), (4, 264, 1056, HF), (24, 264, 1056, HF), (50, 512, 512, F32),
                                       (200, 264, 4128, BF), (300, 264, 2048, F32), (4096, 4096, 512, BF), (700, 3000, 4128, F32),
                                       (40, 512, 16384, F32)])
def test_random_scales(M, N, K, out):
    """Scales from 2^-12 to 2^12: fp32 sums of very different blocks."""
    (A, sa), (W, sw) = operand(M, K, 12, spread=12), operand(N, K, 13, spread=12)
    if out == HF:     # into fp16's range
        sa.view(U8).sub_(8), sw.view(U8).sub_(8)
    a, w = values(A, sa), values(W, sw)
    ref, mag = a @ w.t(), a.abs() @ w.abs().t()
    got = pt.pipe_gemm_mxfp4(A, sa, W, sw, out_dtype=out)
    tol = ref.abs() * HALF[out] * (1 + 2 ** -10) + mag * ((K / 32 + 16) * 2 * U) + 2.0 ** -25
    assert bool(((got.to(D) - ref).abs() <= tol).all())
    assert torch.equal(got, pt.pipe_gemm_mxfp4(A, sa, W, sw, out_dtype=out))


@pytest.mark.parametrize("M,N,K", [(1, 512, 4096), (4, 264, 8192), (24, 512, 4096), (60, 13000, 4096), (150, 512, 4096),
                                   (300, 1000, 8192), (1000, 5000, 1056), (4096, 4096, 544)])
def test_fp32_sums(M, N, K):
    """fp32 C holds fp32 sums: the errors of K / 32 independent roundings add up to sqrt(K / 32) * 2^-24 of the sums on
    the way, themselves no larger than the result's norm; twice that for truncations."""
    A, sa = pt.pipe_quantize_mxfp4(normal((M, K), F32, 14))
    W, sw = pt.pipe_quantize_mxfp4(normal((N, K), F32, 15))
    ref = values(A, sa) @ values(W, sw).t()
    got = pt.pipe_gemm_mxfp4(A, sa, W, sw, out_dtype=F32).to(D)
    assert float((got - ref).norm() / ref.norm()) <= 2 * (K / 32) ** 0.5 * U


@pytest.mark.parametrize("M,N,K", [(1, 72, 160), (3, 264, 1056), (5, 72, 160), (40, 136, 544), (150, 200, 1056), (4096, 4104, 96)])
def test_strided(M, N, K):
    """Padded rows, with NaN scales and other codes between them: nothing past a row's K may enter a sum."""
    (A, sa), (W, sw) = operand(M, K, 16, pad_codes=48), operand(N, K, 17, pad_codes=16)
    ref = values(A, sa).float() @ values(W, sw).float().t()
    base = torch.full((M, N + 24), 5.0, device=DEV)
    got = pt.pipe_gemm_mxfp4(A, sa, W, sw, C=base[:, :N])
    assert torch.equal(got, ref) and bool((base[:, N:] == 5).all())


@pytest.mark.parametrize("M", [2, 40, 150, 700])
def test_nan_stays_in_its_row_and_column(M):
    N, K = 264, 1056
    (A, sa), (W, sw) = operand(M, K, 18), operand(N, K, 19)
    clean = pt.pipe_gemm_mxfp4(A, sa, W, sw, out_dtype=F32)
    sa.view(U8)[1, 7] = 255
    sw.view(U8)[30, K // 32 - 1] = 255
    got = pt.pipe_gemm_mxfp4(A, sa, W, sw, out_dtype=F32)
    hit = torch.zeros(M, N, dtype=torch.bool, device=DEV)
    hit[1], hit[:, 30] = True, True
    assert torch.equal(torch.isnan(got), hit) and torch.equal(got[~hit], clean[~hit])
    A.view(U8).zero_()      # zeros times a NaN scale are NaN too
    got = pt.pipe_gemm_mxfp4(A, sa, W, sw, out_dtype=F32)
    assert torch.equal(torch.isnan(got), hit) and bool((got[~hit] == 0).all())


@pytest.mark.parametrize("M", [1, 4, 24, 300])
def test_extreme_scales(M):
    """Powers of two whose exponents meet in the middle, and products past either end of fp32."""
    N, K = 64, 512
    A = torch.full((M, K // 2), 0x22, dtype=U8, device=DEV).view(F4)      # ones
    W = torch.full((N, K // 2), 0x22, dtype=U8, device=DEV).view(F4)
    for ea, ew, want in ((254, 0, 512.0), (0, 254, 512.0), (127, 127, 512.0), (254, 254, float("inf")), (0, 0, 0.0),
                         (20, 30, 0.0), (10, 127, 2.0 ** -108)):
        sa, sw = (scale_view(torch.full((r, K // 32), e, dtype=U8, device=DEV)) for r, e in ((M, ea), (N, ew)))
        assert bool((pt.pipe_gemm_mxfp4(A, sa, W, sw, out_dtype=F32) == want).all()), (ea, ew)


# ---------------------------------------------------------------------------
# Together, on streams and in graphs
# ---------------------------------------------------------------------------
def layer(x, res, w, b, W, sw, out=None):
    y, s, h = pt.pipe_layernorm(x, w, b, residual=res, out_dtype=F4)
    return pt.pipe_gemm_mxfp4(y, s, W, sw, out_dtype=out or x.dtype), h, y, s


@pytest.mark.parametrize("M,N,K,dtype", [(1, 512, 1024, BF), (4, 264, 4128, HF), (37, 512, 992, BF), (300, 520, 2048, HF)])
def test_layer(M, N, K, dtype):
    """The norm's 4-bit rows into the product, and the gradient of the same stream: the product is that of the values
    which the rows stand for, and the norm without 4 bits, brought into them, gives the same rows up to its rounding."""
    x, res = normal((M, K), dtype, 20), normal((M, K), dtype, 21)
    w, b = normal((K,), dtype, 22), normal((K,), dtype, 23)
    W, sw = pt.pipe_quantize_mxfp4(normal((N, K), F32, 24))
    C, h, y, s = layer(x, res, w, b, W, sw)
    a, v = values(y, s), values(W, sw)
    ref, mag = a @ v.t(), a.abs() @ v.abs().t()
    assert bool(((C.to(D) - ref).abs() <= ref.abs() * HALF[dtype] * (1 + 2 ** -10) + mag * ((K / 32 + 16) * 2 * U)).all())
    assert torch.equal(h, (x.float() + res.float()).to(dtype))
    back = pt.pipe_dequantize_mxfp4(y, s, out_dtype=F32)
    assert torch.equal(back.to(D), a)
    # Half a step of a code next to its block's largest is at most a quarter of that, past 6 a third of 6 (8 at most).
    plain = pt.pipe_layernorm(h, w, b).to(D)
    top = plain.abs().unflatten(1, (-1, 32)).amax(dim=2).repeat_interleave(32, dim=1)
    assert bool(((a - plain).abs() <= top / 4 * (1 + 2 * HALF[dtype]) + plain.abs() * HALF[dtype] * 2).all())
    dC = normal((M, N), F32, 25)
    dy = (dC @ pt.pipe_dequantize_mxfp4(W, sw, out_dtype=F32)).to(dtype)
    dx, dw, db = pt.pipe_layernorm_backward(dy, h, w, dh=res)
    assert dx.shape == h.shape and bool(torch.isfinite(dx).all()) and torch.isfinite(dw).all() and torch.isfinite(db).all()


@pytest.mark.parametrize("M", [1, 24, 300])
def test_captured_and_replayed(M):
    """Captured once and replayed with other inputs, eager work between the replays: every replay is the eager result."""
    N, K = 512, 16384
    W, sw = pt.pipe_quantize_mxfp4(normal((N, K), F32, 26))
    x, res, dy = (normal((M, K), BF, s) for s in (27, 28, 29))
    w, b = normal((K,), BF, 30), normal((K,), BF, 31)

    def work():
        C, h, y, s = layer(x, res, w, b, W, sw)
        back = pt.pipe_dequantize_mxfp4(*pt.pipe_quantize_mxfp4(h))
        return (C, h, y.view(U8), s.view(U8), back, *pt.pipe_layernorm_backward(dy, h, w, dh=res))

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = work()
    for turn in range(4):
        for t, seed in ((x, 40), (res, 50), (dy, 60)):
            t.copy_(normal(t.shape, BF, seed + turn))
        want = [t.clone() for t in work()]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, want)), turn


def test_on_another_stream_and_two_at_once():
    """Two streams at once, each with outputs and workspaces of its own."""
    M, N, K = 40, 512, 16384
    W, sw = pt.pipe_quantize_mxfp4(normal((N, K), F32, 32))
    w, b = normal((K,), BF, 33), normal((K,), BF, 34)
    xs = [normal((M, K), BF, 35 + i) for i in range(2)]

    def work(x, stream):
        y, s, h = pt.pipe_layernorm(x, w, b, residual=x, out_dtype=F4, stream=stream)
        C = pt.pipe_gemm_mxfp4(y, s, W, sw, stream=stream)
        codes = pt.pipe_quantize_mxfp4(h, stream=stream)
        return (C, pt.pipe_dequantize_mxfp4(*codes, stream=stream), *pt.pipe_layernorm_backward(x, h, w, dh=x, stream=stream))

    want = [work(x, None) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(5):
        got = [work(x, s) for x, s in zip(xs, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, v in zip(got, want) for a, b in zip(g, v))
