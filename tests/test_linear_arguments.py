"""Arguments that are no tensors, streams or numbers are refused with TypeError before anything else happens, whichever
optional argument they stand in. Without a device: host tensors stand for device tensors by a patched device number."""
import pytest
import torch

import async_stage_tile_amd as pt
from async_stage_tile_amd import linear

BF, E4 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture
def as_device(monkeypatch):
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    linear._setup()
    monkeypatch.setattr(linear, "_fast", None)
    monkeypatch.setattr(linear, "_call", lambda *a, **k: pytest.fail("the call went on"))


def operands():
    x, w = torch.zeros(4, 64, dtype=BF), torch.ones(64, dtype=BF)
    e, f = torch.zeros(8, 64, dtype=E4), torch.ones(8)
    codes, scales = torch.zeros(8, 32, dtype=torch.uint8), torch.ones(8, 2, dtype=BF)
    return {
        "rmsnorm": (pt.pipe_rmsnorm, (x, w), dict(residual=x)),
        "rmsnorm_backward": (pt.pipe_rmsnorm_backward, (x, x, w), {}),
        "gemm_fp8": (pt.pipe_gemm_fp8, (e, f, e.t(), f), {}),
        "gemm_w4": (pt.pipe_gemm_w4, (x, codes, scales), {}),
    }


@pytest.mark.parametrize("wrong", [5, "x", [1.0]])
@pytest.mark.parametrize("name,place", [
    ("rmsnorm", "y"), ("rmsnorm", "h"), ("rmsnorm", "residual"), ("rmsnorm", "stream"), ("rmsnorm", "out_dtype"),
    ("rmsnorm_backward", "dh"), ("rmsnorm_backward", "dx"), ("rmsnorm_backward", "dweight"),
    ("rmsnorm_backward", "workspace"), ("rmsnorm_backward", "stream"),
    ("gemm_fp8", "C"), ("gemm_fp8", "workspace"), ("gemm_fp8", "stream"), ("gemm_fp8", "out_dtype"),
    ("gemm_w4", "zeros"), ("gemm_w4", "C"), ("gemm_w4", "workspace"), ("gemm_w4", "stream"),
])
def test_optional_arguments(as_device, name, place, wrong):
    f, args, more = operands()[name]
    with pytest.raises(TypeError):
        f(*args, **{**more, place: wrong})


@pytest.mark.parametrize("name,wrong", [("rmsnorm", "x"), ("rmsnorm", [1e-6]), ("rmsnorm_backward", "x")])
def test_eps(as_device, name, wrong):
    f, args, more = operands()[name]
    with pytest.raises((TypeError, ValueError)):
        f(*args, eps=wrong, **more)


@pytest.mark.parametrize("name,count", [("rmsnorm", 2), ("rmsnorm_backward", 3), ("gemm_fp8", 4), ("gemm_w4", 3)])
def test_operands(as_device, name, count):
    f, args, more = operands()[name]
    for i in range(count):
        for wrong in (None, 5, "x"):
            with pytest.raises(TypeError):
                f(*args[:i], wrong, *args[i + 1:], **more)
