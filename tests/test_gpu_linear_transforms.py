"""Operands that a function transform wraps are refused by the wrappers, in every place, and the process goes on."""
import pytest
import torch

import async_stage_tile_amd as pt

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, E4 = torch.bfloat16, torch.float8_e4m3fn


def operators():
    x, w = torch.ones(4, 64, dtype=BF, device=DEV), torch.ones(64, dtype=BF, device=DEV)
    e, f = torch.ones(8, 64, device=DEV).to(E4), torch.ones(8, device=DEV)
    codes, scales = torch.zeros(8, 32, dtype=torch.uint8, device=DEV), torch.ones(8, 2, dtype=BF, device=DEV)
    return {"rmsnorm": (lambda a, b, c: pt.pipe_rmsnorm(a, b, residual=c), (x, w, x)),
            "rmsnorm_backward": (lambda a, b, c, d: pt.pipe_rmsnorm_backward(a, b, c, dh=d), (x, x, w, x)),
            "gemm_fp8": (pt.pipe_gemm_fp8, (e, f, e.t(), f)),
            "gemm_w4": (pt.pipe_gemm_w4, (x, codes, scales))}


@pytest.mark.parametrize("name", ["rmsnorm", "rmsnorm_backward", "gemm_fp8", "gemm_w4"])
def test_wrapped_operands(name):
    print(f"[linear transforms] {name}", flush=True)
    f, args = operators()[name]
    for i, a in enumerate(args):
        with pytest.raises(RuntimeError):
            torch.func.vmap(lambda t: f(*args[:i], t, *args[i + 1:]))(a.expand((2,) + tuple(a.shape)))
        if a.dtype in (BF, torch.float32):
            with pytest.raises(RuntimeError):
                torch.func.vjp(lambda t: f(*args[:i], t, *args[i + 1:]), a)
    out = f(*args)
    torch.cuda.synchronize()
    assert torch.isfinite((out[0] if isinstance(out, tuple) else out).float()).all()
