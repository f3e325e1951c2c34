"""Layer norm and its gradient against their formulas in 64 bits.

Tolerances are bounds, derived from the arithmetic. With U = 2^-24 and a row's sum off by at most CHAIN * U of the sum of
its terms' magnitudes (32 elements a thread, 6 steps of the wave, 16 waves, and a few roundings of the terms):
the mean m0 is off by delta <= CHAIN U mean|h|, which the second turn's mean of d = h - m0 corrects up to CHAIN U (mean|h -
m| + delta); the deviation itself is rounded once more or twice; the variance is off by CHAIN U (var + delta^2), r by half
of that and a few roundings. A rounding to a type is off by at most half a step."""
import pytest
import torch

import async_stage_tile_amd as pt

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
D = torch.float64
BF, HF, F32, E4, F4 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn, torch.float4_e2m1fn_x2
HALF = {BF: 2.0 ** -8, HF: 2.0 ** -11, F32: 2.0 ** -24, E4: 2.0 ** -4}     # half a step of 1
TINY = {BF: 2.0 ** -134, HF: 2.0 ** -25, F32: 2.0 ** -150, E4: 2.0 ** -10}  # half the smallest step
CHAIN = 32 + 6 + 16 + 4
UP = 1 + 2 ** -10   # a rounding's share of a value that is itself a little off


@pytest.fixture(autouse=True)
def _name(request):
    print(f"[layernorm] {request.node.name}", flush=True)
    yield
    torch.cuda.synchronize()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(shape, dtype, seed):
    return torch.randn(shape, device=DEV, generator=gen(seed)).to(dtype)


def padded(t, pad):
    """The same matrix as a view of a wider one."""
    wide = torch.zeros((t.shape[0], t.shape[1] + pad), device=t.device, dtype=t.dtype)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def close(got, ref, tol, what):
    got, ref = got.to(D), ref.to(D)
    assert got.shape == ref.shape, what
    bad = ~((got - ref).abs() <= tol)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()}, worst " \
        f"{float(((got - ref).abs() / tol.clamp_min(1e-300)).max()):.3f} of the bound at {bad.nonzero()[0].tolist()}"


def mean(v):
    return v.mean(dim=1, keepdim=True)


class Stats:
    """A row's u = (h - m) r in 64 bits, and how far the kernels' may be off."""

    def __init__(self, h, eps):
        v = h.to(D)
        self.m = mean(v)
        self.d = v - self.m
        var = mean(self.d ** 2)
        self.r = 1 / torch.sqrt(var + eps)
        self.u = self.d * self.r
        delta = CHAIN * U * mean(v.abs())
        self.rel_r = U * (CHAIN / 2 * (1 + delta ** 2 / (var + eps)) + 8)
        self.off = U * (CHAIN * (mean(self.d.abs()) + delta) + 2 * (self.d.abs() + delta)) * self.r
        self.tol = self.off + self.u.abs() * self.rel_r


def norm_reference(x, w, b, res, eps):
    """h, y and how far y may be off before its rounding."""
    h = x if res is None else (x.float() + res.float()).to(x.dtype)
    s = Stats(h, eps)
    bias = torch.zeros_like(w).to(D) if b is None else b.to(D)
    y = s.u * w.to(D) + bias
    return h, y, w.to(D).abs() * s.tol + 3 * U * ((s.u * w.to(D)).abs() + bias.abs())


E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
STEP = [0.25, 0.25, 0.25, 0.25, 0.5, 0.5, 1.0, 2.0]    # the longer half of the two steps next to it; past 6 up to 8


def form_parts(codes, scales):
    """(values, half steps, powers of two) of the 4-bit form, in 64 bits."""
    c = codes.view(torch.uint8)
    c = torch.stack([c & 15, c >> 4], dim=2).flatten(1).long()
    value = torch.tensor(E2M1 + [-v for v in E2M1], dtype=D, device=c.device)[c]
    step = torch.tensor(STEP + STEP, dtype=D, device=c.device)[c]
    p = torch.exp2(scales.view(torch.uint8).to(D) - 127)
    return value, step, p.repeat_interleave(32, dim=1)


def check_form(codes, scales, ref, tol):
    """Each code is the nearest to a value within tol of ref, and so is each block's power of two."""
    value, step, p = form_parts(codes, scales)
    close(value * p, ref, step * p + tol, "values")
    top = ref.abs().unflatten(1, (-1, 32)).amax(dim=2)
    slack = tol.unflatten(1, (-1, 32)).amax(dim=2)
    p = p[:, ::32]
    assert bool(((4 * p <= top + slack) | (p == 2.0 ** -127)).all()) and bool((top - slack < 8 * p).all())


def check_norm(x, w, b, res, out, eps=1e-5, **kw):
    h, ref, tol = norm_reference(x, w, b, res, eps)
    got = pt.pipe_layernorm(x, w, b, residual=res, eps=eps, out_dtype=out, **kw)
    got = list(got) if isinstance(got, tuple) else [got]
    y = got.pop(0)
    if out == F4:
        check_form(y, got.pop(0), ref, tol)
    elif out == E4:
        s = got.pop(0)
        top = ref.abs().amax(dim=1).clamp_min(2.0 ** -100)
        rel = tol.amax(dim=1) / top + 4 * U
        close(s, top / 448, top / 448 * rel, "scales")
        scale = (top / 448)[:, None]
        close(y, ref / scale, (ref / scale).abs() * (HALF[E4] * UP + rel[:, None]) + tol / scale * UP + TINY[E4], "y")
    else:
        close(y, ref, ref.abs() * HALF[out] + tol * UP + TINY[out], "y")
    if res is not None:
        assert torch.equal(got.pop(0).view(torch.int16), h.view(torch.int16))
    assert not got


@pytest.mark.parametrize("M,N", [(1, 8), (1, 32), (1, 4096), (3, 504), (3, 512), (5, 520), (4, 1024), (7, 1056), (2, 2048), (3, 2080),
                                 (2, 4128), (1, 8192), (3, 8224), (1, 16384), (2, 16416), (2, 32768), (1021, 256), (600, 5024),
                                 (5, 6144), (3, 6176), (2, 10016), (3, 20000), (9, 1536)])
@pytest.mark.parametrize("dtype,out,residual,bias", [(BF, BF, True, True), (HF, HF, False, True), (BF, E4, True, False),
                                                     (HF, E4, False, True), (BF, BF, False, False), (BF, F4, True, True),
                                                     (HF, F4, False, False), (HF, HF, True, False)])
def test_norm(M, N, dtype, out, residual, bias):
    if out == F4 and N % 32:
        N = N // 32 * 32 or 32
    x = normal((M, N), dtype, 1) + 0.5
    w = (1 + 0.1 * normal((N,), F32, 2)).to(dtype)
    check_norm(x, w, normal((N,), dtype, 4) if bias else None, normal((M, N), dtype, 3) if residual else None, out)


@pytest.mark.parametrize("out", [HF, E4, F4])
@pytest.mark.parametrize("center,spread", [(1000.0, 1.0), (-30000.0, 40.0), (100.0, 0.05), (0.001, 1e-4)])
def test_norm_of_rows_far_from_zero(out, center, spread):
    """Means many times the deviations: what the mean's own rounding would cost is corrected."""
    M, N = 9, 4128
    x = (center + spread * normal((M, N), F32, 5)).to(HF)
    check_norm(x, normal((N,), HF, 6), normal((N,), HF, 7), None, out, eps=1e-12)


def test_norm_of_equal_values():
    """No deviation at all: y is the bias, whatever the mean."""
    for value in (0.0, 1.0, 1000.0, 60000.0, 0.3):
        x = torch.full((3, 5000), value, device=DEV, dtype=HF)
        w, b = normal((5000,), HF, 8), normal((5000,), HF, 9)
        _, ref, tol = norm_reference(x, w, b, None, 1e-5)
        assert float((ref - b.to(D)).abs().max()) < 1e-9
        got = pt.pipe_layernorm(x, w, b)
        close(got, ref, ref.abs() * HALF[HF] + tol * UP + TINY[HF], f"rows of {value}")


@pytest.mark.parametrize("out", [BF, E4, F4])
def test_norm_strided_in_place_and_given_outputs(out):
    M, N = 37, 992
    x, res = padded(normal((M, N), BF, 10), 24), padded(normal((M, N), BF, 11), 40)
    w, b = normal((N,), BF, 12), normal((N,), BF, 13)
    check_norm(x, w, b, res, out)
    want = pt.pipe_layernorm(x, w, b, residual=res, out_dtype=out)
    cols = N // 2 if out == F4 else N
    base = torch.full((M, (cols + 16) * (2 if out == BF else 1)), 77, device=DEV, dtype=torch.uint8)
    y = base.view(out)[:, :cols]
    kw = {}
    if out == F4:
        pad = torch.full((M, 48), 99, device=DEV, dtype=torch.uint8)
        kw["y_scales"] = pad[:, :N // 32].view(torch.float8_e8m0fnu)
    elif out == E4:
        kw["y_scales"] = torch.empty(M, device=DEV)
    got = pt.pipe_layernorm(x, w, b, residual=res, out_dtype=out, y=y, h=res, **kw)
    assert got[0] is y and got[-1] is res and torch.equal(res, want[-1])
    assert bool((base[:, cols * (2 if out == BF else 1):] == 77).all())      # nothing written past the row
    assert torch.equal(y.contiguous().view(torch.uint8) if out == BF else y.view(torch.uint8).contiguous(),
                       want[0].view(torch.uint8))
    if out == F4:
        assert bool((pad[:, N // 32:] == 99).all())
    if out != BF:
        assert torch.equal(got[1].view(torch.uint8), want[1].view(torch.uint8))
    else:
        x0 = x.clone()
        assert torch.equal(pt.pipe_layernorm(x, w, b, y=x), pt.pipe_layernorm(x0, w, b))


def test_norm_special_rows():
    """Zeros, tiny and huge rows, NaN and infinities: row by row, without touching their neighbours."""
    M, N = 8, 2080
    x = normal((M, N), BF, 14)
    x[1] = 0
    x[2] *= 1e-30
    x[3] *= 1e15
    x[4, 77] = float("nan")
    x[5, 78] = float("inf")
    x[6, 79] = float("-inf")
    w, b = normal((N,), BF, 15), normal((N,), BF, 16)
    good = [0, 1, 2, 3, 7]
    _, ref, tol = norm_reference(x[good], w, b, None, 1e-5)
    y = pt.pipe_layernorm(x, w, b)
    close(y[good], ref, ref.abs() * HALF[BF] + tol * UP + TINY[BF], "y")
    assert bool(torch.isnan(y[4:7]).all())
    y8, s8 = pt.pipe_layernorm(x, w, b, out_dtype=E4)
    assert bool(torch.isnan(s8[4:7]).all()) and bool(torch.isnan(y8[4:7].float()).all())
    assert bool(torch.isfinite(s8[good]).all()) and bool(torch.isfinite(y8.float()[good]).all())
    y4, s4 = pt.pipe_layernorm(x, w, b, out_dtype=F4)
    assert bool((s4.view(torch.uint8)[4:7] == 255).all())
    check_form(y4.view(torch.uint8)[good].view(F4), s4.view(torch.uint8)[good].view(torch.float8_e8m0fnu), ref, tol)
    b[3] = float("inf")     # an infinite value in every row: e4m3's scale is NaN, of the 4-bit form its block's
    _, s8 = pt.pipe_layernorm(x, w, b, out_dtype=E4)
    assert bool(torch.isnan(s8).all())
    _, s4 = pt.pipe_layernorm(x, w, b, out_dtype=F4)
    assert bool((s4.view(torch.uint8)[:, 0] == 255).all()) and bool((s4.view(torch.uint8)[good][:, 1:] != 255).all())
    x[:] = 0
    b[:] = 0
    y8, s8 = pt.pipe_layernorm(x, w, b, out_dtype=E4)
    assert bool((y8.float() == 0).all()) and bool((s8 == torch.tensor(2.0 ** -100, device=DEV) / 448).all())
    y4, s4 = pt.pipe_layernorm(x, w, out_dtype=F4)
    assert bool(((y4.view(torch.uint8) & 0x77) == 0).all()) and bool((s4.view(torch.uint8) == 0).all())


def test_norm_empty_and_refusals():
    w = torch.ones(64, dtype=BF, device=DEV)
    x = torch.ones(4, 64, dtype=BF, device=DEV)
    y, s, h = pt.pipe_layernorm(x[:0], w, residual=x[:0], out_dtype=E4)
    assert y.shape == (0, 64) and s.shape == (0,) and h.shape == (0, 64)
    y, s = pt.pipe_layernorm(x[:0], w, out_dtype=F4)
    assert y.shape == (0, 32) and s.shape == (0, 2)
    dx, dw, db = pt.pipe_layernorm_backward(x[:0], x[:0], w)
    assert dx.shape == (0, 64) and bool((dw == 0).all()) and bool((db == 0).all())
    for bad, kind in (((x, w.half()), TypeError), ((x, w[:32]), ValueError), ((x.t(), w), ValueError), ((x[0], w), ValueError),
                      ((x, w, w.half()), TypeError), ((x, w, w[:32]), ValueError)):
        with pytest.raises(kind):
            pt.pipe_layernorm(*bad)
    with pytest.raises(TypeError):
        pt.pipe_layernorm(x, w, out_dtype=HF)
    with pytest.raises(ValueError):
        pt.pipe_layernorm(x, w, residual=x[:2])
    for view, status in ((x[:, :60], pt.PIPE_ERR_SHAPE), (x[:, 4:60], pt.PIPE_ERR_ALIGN)):
        with pytest.raises(pt.PipeError) as e:
            pt.pipe_layernorm(view, w[:view.shape[1]])
        assert e.value.status == status


# ---------------------------------------------------------------------------
# Gradient
# ---------------------------------------------------------------------------
def grad_reference(dy, x, w, dh, eps):
    """dx, dweight and dbias, and how far each may be off before its rounding."""
    s = Stats(x, eps)
    g = dy.to(D)
    gw = g * w.to(D)
    along = mean(gw * s.u)
    dx = s.r * (gw - mean(gw) - s.u * along)
    # The sums of the second turn are of g d, with d off by U (|d| + delta) and by its mean's own error, which the
    # correction by mean(g) takes out.
    sum_off = U * (CHAIN + 6) * (mean((gw * s.u).abs()) + mean(s.off / U / CHAIN) * mean(gw.abs()))
    tol = s.r * (U * (CHAIN + 4) * mean(gw.abs()) + 4 * U * gw.abs() + s.tol * along.abs() + s.u.abs() *
                 (sum_off + along.abs() * (s.rel_r + 4 * U))) + (dx.abs() * (s.rel_r + 4 * U))
    if dh is not None:
        dx = dx + dh.to(D)
        tol = tol + 2 * U * dx.abs()
    # A workgroup's rows (256 workgroups or more where there are as many rows, and at least one in 16), its
    # partial's place among the others.
    chain = max(x.shape[0] / 256, 16) + 64 + 4
    tol_w = (g.abs() * s.tol).sum(dim=0) + U * chain * (g * s.u).abs().sum(dim=0) + 1e-300
    return dx, (g * s.u).sum(dim=0), g.sum(dim=0), tol, tol_w, U * chain * g.abs().sum(dim=0) + 1e-300


def check_grad(dy, x, w, dh, eps=1e-5):
    dx, dw, db, tol, tol_w, tol_b = grad_reference(dy, x, w, dh, eps)
    got = pt.pipe_layernorm_backward(dy, x, w, dh=dh, eps=eps)
    close(got[0], dx, dx.abs() * HALF[x.dtype] * UP + tol * UP + TINY[x.dtype], "dx")
    close(got[1], dw, tol_w, "dweight")
    close(got[2], db, tol_b, "dbias")
    again = pt.pipe_layernorm_backward(dy, x, w, dh=dh, eps=eps)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("M,N", [(1, 8), (1, 4096), (5, 512), (6, 1000), (5, 2048), (3, 4096), (4, 8200), (2, 16384), (3, 16400),
                                 (2, 32768), (2100, 264), (1500, 2056), (1021, 2048), (16, 512), (17, 512), (18, 4096), (9, 8192),
                                 (700, 5000), (4100, 2056), (4099, 8192), (600, 16384), (300, 24008),
                                 (2047, 1000), (2049, 1000), (2050, 2048), (3001, 512), (2048, 504), (4097, 4104), (4096, 5000), (700, 1024)])
@pytest.mark.parametrize("dtype,residual", [(BF, True), (HF, False), (HF, True), (BF, False)])
def test_grad(M, N, dtype, residual):
    w = (1 + 0.1 * normal((N,), F32, 20)).to(dtype)
    check_grad(normal((M, N), dtype, 21), normal((M, N), dtype, 22) - 0.5, w,
               normal((M, N), dtype, 23) if residual else None)


def test_grad_of_rows_far_from_zero():
    x = (1000 + normal((33, 4104), F32, 24)).to(HF)
    check_grad(normal((33, 4104), HF, 25), x, normal((4104,), HF, 26), None)


def test_grad_strided_in_place_and_given():
    M, N = 70, 776
    dy, x, dh = (padded(normal((M, N), BF, s), p) for s, p in ((27, 8), (28, 16), (29, 24)))
    w = normal((N,), BF, 30)
    check_grad(dy, x, w, dh)
    want = pt.pipe_layernorm_backward(dy, x, w, dh=dh)
    dw, db = torch.empty(N, device=DEV), torch.empty(N, device=DEV)
    space = torch.empty(pt.pipe_layernorm_backward_workspace_bytes(M, N), dtype=torch.uint8, device=DEV)
    got = pt.pipe_layernorm_backward(dy, x, w, dh=dh, dx=dh, dweight=dw, dbias=db, workspace=space)
    assert got[0] is dh and got[1] is dw and got[2] is db
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(pt.PipeError) as e:
        pt.pipe_layernorm_backward(dy, x, w, workspace=space[:16])
    assert e.value.status == pt.PIPE_ERR_WORKSPACE


def test_grad_nan_stays_in_its_row():
    M, N = 12, 1000
    dy, x = normal((M, N), HF, 31), normal((M, N), HF, 32)
    w = normal((N,), HF, 33)
    clean = pt.pipe_layernorm_backward(dy, x, w)[0]
    x[3, 5], dy[7, 9] = float("nan"), float("inf")
    dx, dw, db = pt.pipe_layernorm_backward(dy, x, w)
    keep = [i for i in range(M) if i not in (3, 7)]
    assert torch.equal(dx[keep], clean[keep]) and bool(torch.isnan(dx[3]).all()) and not bool(torch.isfinite(dx[7]).any())
    assert bool(torch.isnan(dw).all()) and bool(torch.isfinite(db[:9]).all()) and not bool(torch.isfinite(db[9]))


def test_grad_against_differences():
    """The gradients against central differences of the 64-bit forward pass, along random directions; the difference
    quotient of step t is off by O(t^2), far below the outputs' rounding."""
    M, N, eps, t = 6, 264, 1e-5, 1e-4
    dy, x, dh = (normal((M, N), HF, s) for s in (34, 35, 36))
    w = normal((N,), HF, 37)
    dx, dw, db = pt.pipe_layernorm_backward(dy, x, w, dh=dh, eps=eps)

    def loss(v, weight, bias):
        d = v - mean(v)
        return ((d / torch.sqrt(mean(d * d) + eps) * weight + bias) * dy.to(D)).sum() + (v * dh.to(D)).sum()

    zero = torch.zeros(N, dtype=D, device=DEV)
    _, _, _, tol, tol_w, tol_b = grad_reference(dy, x, w, dh, eps)
    for seed in (38, 39, 40):
        ex, ew, eb = normal((M, N), D, seed), normal((N,), D, seed + 10), normal((N,), D, seed + 20)
        for e, grad, bound in (((ex, zero, zero), (dx.to(D) * ex).sum(), ((dx.to(D).abs() * HALF[HF] * UP + tol) * ex.abs()).sum()),
                               ((0 * ex, ew, zero), (dw.to(D) * ew).sum(), (tol_w * ew.abs()).sum()),
                               ((0 * ex, zero, eb), (db.to(D) * eb).sum(), (tol_b * eb.abs()).sum())):
            quot = (loss(x.to(D) + t * e[0], w.to(D) + t * e[1], t * e[2]) -
                    loss(x.to(D) - t * e[0], w.to(D) - t * e[1], -t * e[2])) / (2 * t)
            assert abs(float(quot - grad)) <= float(bound) + 1e-5


@pytest.mark.parametrize("residual", (True, False))
@pytest.mark.parametrize("N", (512, 1024, 2048, 4096, 5000, 8192, 16384))
def test_rows_do_not_depend_on_the_others(N, residual):
    """A row's y, h and dx are the same bits however many rows the call has: threads and chunks go by the width."""
    M = 9000 if N <= 4096 else 5000
    x, dy, dh = (normal((M, N), BF, s) for s in (41, 42, 43))
    w, b = normal((N,), BF, 44), normal((N,), BF, 45)
    more = dh if residual else None
    y, dx = pt.pipe_layernorm(x, w, b, residual=more), pt.pipe_layernorm_backward(dy, x, w, dh=more)[0]
    for rows in (1, 40, 300, 1021, 2500):
        few = None if more is None else more[:rows]
        got = pt.pipe_layernorm(x[:rows], w, b, residual=few)
        if residual:
            assert torch.equal(got[0], y[0][:rows]) and torch.equal(got[1], y[1][:rows])
        else:
            assert torch.equal(got, y[:rows])
        assert torch.equal(pt.pipe_layernorm_backward(dy[:rows], x[:rows], w, dh=few)[0], dx[:rows])
