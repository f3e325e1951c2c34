"""The C++ marshalling of layer norm's and the microscaled 4-bit form's calls without a device, as in
test_linear_binding.py: host tensors that carry a device's mark, and counting stubs for the library's functions."""
import subprocess
import sys

import pytest
import torch

from async_stage_tile_amd import linear
from tests.conftest import ROOT
from tests.test_linear_binding import helper  # noqa: F401  (a fixture)

PROLOGUE = """
import ctypes, sys
sys.path[:0] = [{root!r}, {helper!r}]
import torch
import marked_tensors
from async_stage_tile_amd import _linear as fast

calls = []
stub = ctypes.CFUNCTYPE(ctypes.c_int)(lambda: (calls.append(1), 0)[1])
address = ctypes.cast(stub, ctypes.c_void_p).value
bf, u8, f4, e8 = torch.bfloat16, torch.uint8, torch.float4_e2m1fn_x2, torch.float8_e8m0fnu

def dev(t):
    return marked_tensors.marked(t)

x, w = dev(torch.zeros(4, 64, dtype=bf)), dev(torch.zeros(64, dtype=bf))
A, W = dev(torch.zeros(4, 32, dtype=u8)).view(f4), dev(torch.zeros(8, 32, dtype=u8)).view(f4)
sa, sw = dev(torch.zeros(4, 16, dtype=u8))[:, :2].view(e8), dev(torch.zeros(8, 16, dtype=u8))[:, :2].view(e8)
OPERATORS = {{
    "layernorm": (fast.layernorm, (x, w, w, x, 1e-5, f4)),
    "layernorm_backward": (fast.layernorm_backward, (x, x, w, x, 1e-5)),
    "quantize_mxfp4": (fast.quantize_mxfp4, (x,)),
    "dequantize_mxfp4": (fast.dequantize_mxfp4, (A, sa, None)),
    "gemm_mxfp4": (fast.gemm_mxfp4, (A, sa, W, sw, None)),
}}
name = {operator!r}
f, args = OPERATORS[name]
places = [i for i, a in enumerate(args) if isinstance(a, torch.Tensor)]
assert f(*args) is NotImplemented and not calls     # not bound yet
fast.bind(lambda device: 0, *[address] * 7)
assert f(*args) is NotImplemented and not calls
fast.bind_layer(*[address] * 7)
out = f(*args)
assert out is not NotImplemented and len(calls) >= 1     # the plain call goes through
"""

PLAIN = """
for t in out if isinstance(out, tuple) else (out,):
    if t.dtype is e8:
        assert t.shape == (4, 2) and t.stride() == (16, 1) and t.untyped_storage().nbytes() == 64
print("ok")
"""

WRAPPED = """
calls.clear()
for i in places:
    seen = []

    def call(t):
        seen.append(f(*args[:i], t, *args[i + 1:]))
        return t

    torch.func.vmap(call)(args[i].detach().expand((2,) + tuple(args[i].shape)))
    if args[i].dtype is bf:
        torch.func.vjp(call, args[i])
        torch.func.jvp(call, (args[i],), (args[i],))
    assert seen and all(s is NotImplemented for s in seen), (name, i)
    ctypes.pythonapi.PyGILState_Check.restype = ctypes.c_int
    assert ctypes.pythonapi.PyGILState_Check() == 1
# Nothing was enqueued: only the workspace's size may have been asked for.
assert len(calls) <= len(places) * 3 * (name in ("layernorm_backward", "gemm_mxfp4")), calls
print("ok")
"""

SUBCLASS = """
class Mine(torch.Tensor):
    pass

calls.clear()
for i in places:
    assert f(*args[:i], args[i].as_subclass(Mine), *args[i + 1:]) is NotImplemented, (name, i)
assert not calls
for i in places:    # a parameter is no subclass to the binding
    if args[i].dtype is bf:
        assert f(*args[:i], torch.nn.Parameter(args[i]), *args[i + 1:]) is not NotImplemented
print("ok")
"""

REFUSED = """
calls.clear()
short = dev(torch.zeros(7 * 16 + 2, dtype=u8)).as_strided((8, 2), (16, 1)).view(e8)     # ends inside a group of 16
narrow, single, double = dev(torch.zeros(4, 40, dtype=bf)), dev(torch.zeros(4, 64)), dev(torch.zeros(4, 64, dtype=torch.float64))
others = {{
    "layernorm": [(x, w, w, x, 1e-5, torch.float16), (narrow, w[:40], None, None, 1e-5, f4), (x, w[:32], None, None, 1e-5, None),
                  (x, w, None, None, "eps", None), (x, w, None, None, 1e-5, "type"), (single, w, None, None, 1e-5, None)],
    "layernorm_backward": [(x, x[:2], w, None, 1e-5), (x, x, w, x[:2], 1e-5), (x, single, w, None, 1e-5), (x, x, w, None, None)],
    "quantize_mxfp4": [(narrow,), (x.view(torch.int16),), (x[0],), (double,)],
    "dequantize_mxfp4": [(A, sw, None), (A, sa.view(u8), None), (A.view(u8), sa, None), (A, sa, f4), (W, short, None), (A, None, None)],
    "gemm_mxfp4": [(A, sa, W, short, None), (A, sw, W, sw, None), (A, sa, W, sw, f4), (A, sa, W[:, :16], sw, None), (A, sa, None, None, None),
                   (A.view(u8), sa, W, sw, None)],
}}
for other in others[name]:
    assert f(*other) is NotImplemented, (name, [getattr(o, "shape", o) for o in other])
assert f() is NotImplemented and not calls
print("ok")
"""


@pytest.mark.parametrize("body", [PLAIN, WRAPPED, SUBCLASS, REFUSED], ids=["plain", "wrapped", "subclass", "refused"])
@pytest.mark.parametrize("operator", ["layernorm", "layernorm_backward", "quantize_mxfp4", "dequantize_mxfp4", "gemm_mxfp4"])
def test_calls(helper, operator, body):  # noqa: F811
    code = PROLOGUE.format(root=ROOT, helper=helper, operator=operator) + body.replace("{{", "{").replace("}}", "}")
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=120)
    assert res.returncode == 0 and res.stdout.strip() == "ok", f"exit {res.returncode}\n{res.stdout}{res.stderr[-2000:]}"


def test_bind_layer_refuses():
    linear._setup()
    fast = linear._fast
    assert fast is not None
    with pytest.raises(TypeError):
        fast.bind_layer(1)
    with pytest.raises(ValueError):
        fast.bind_layer(*[0] * 7)
    host = torch.zeros(4, 64, dtype=torch.bfloat16)
    assert fast.quantize_mxfp4(host) is NotImplemented
