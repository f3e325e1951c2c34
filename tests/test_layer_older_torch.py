"""A PyTorch without one of the 4-bit form's types: the operators that do not use it work as ever, the others say what they
need. Without a device, in a process of its own: host tensors stand for device tensors by a patched device number."""
import subprocess
import sys

import pytest

from tests.conftest import ROOT

CODE = """
import sys
sys.path.insert(0, {root!r})
import torch
f4, e8 = torch.float4_e2m1fn_x2, torch.float8_e8m0fnu
delattr(torch, {lacking!r})
import async_stage_tile_amd as pt
from async_stage_tile_amd import linear

assert pt.pipe_gemm_mxfp4_workspace_bytes(1, 256, 8192) == 0
linear._fast = None
torch.Tensor.get_device = lambda self: 0
class Done(Exception):
    pass
def call(fn, name, *args):
    raise Done(name)
linear._call = call
bf, e4 = torch.bfloat16, torch.float8_e4m3fn
x, w = torch.zeros(4, 64, dtype=bf), torch.ones(64, dtype=bf)
e, s = torch.zeros(8, 64, dtype=e4), torch.ones(8)
codes, scales = torch.zeros(8, 32, dtype=torch.uint8), torch.ones(8, 2, dtype=bf)
def goes_on(f, *args, **kw):
    try:
        f(*args, **kw)
    except Done as d:
        assert d.args[0] == f.__name__
        return
    raise AssertionError(f.__name__)
goes_on(pt.pipe_rmsnorm, x, w, out_dtype=e4)
goes_on(pt.pipe_rmsnorm_backward, x, x, w, workspace=s)
goes_on(pt.pipe_gemm_fp8, e, s, e.t(), s)
goes_on(pt.pipe_gemm_w4, x, codes, scales)
goes_on(pt.pipe_layernorm, x, w, w, residual=x)
goes_on(pt.pipe_layernorm, x, w, out_dtype=e4)
goes_on(pt.pipe_layernorm_backward, x, x, w, workspace=s)
A, sa = codes.view(f4), torch.zeros(8, 16, dtype=torch.uint8)[:, :2].view(e8)
for f, args in ((pt.pipe_quantize_mxfp4, (x,)), (pt.pipe_dequantize_mxfp4, (A, sa)), (pt.pipe_gemm_mxfp4, (A, sa, A, sa))):
    try:
        f(*args)
    except RuntimeError as r:
        assert {lacking!r} in str(r)
    else:
        raise AssertionError(f.__name__)
for f in (pt.pipe_layernorm, pt.pipe_rmsnorm):
    try:
        f(x, w, out_dtype=f4)
    except TypeError:
        pass
    else:
        raise AssertionError(f.__name__)
print("ok")
"""


@pytest.mark.parametrize("lacking", ["float4_e2m1fn_x2", "float8_e8m0fnu"])
def test_without(lacking):
    res = subprocess.run([sys.executable, "-c", CODE.format(root=ROOT, lacking=lacking)], capture_output=True, text=True,
                         timeout=120)
    assert res.returncode == 0 and res.stdout.strip() == "ok", f"{res.stdout}{res.stderr[-2000:]}"
