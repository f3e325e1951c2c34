"""The C++ marshalling of the linear layer's calls (_linear.so) without a device: host tensors that carry a device's
mark, and counting stubs for the library's functions. Each case runs in a process of its own: a fault would end it, and
the helper replaces the process's device guard."""
import os
import subprocess
import sys
import sysconfig

import pytest
import torch

from async_stage_tile_amd import build
from tests.conftest import ROOT

PROLOGUE = """
import ctypes, sys
sys.path[:0] = [{root!r}, {helper!r}]
import torch
import marked_tensors
from async_stage_tile_amd import _linear as fast

calls = []
stub = ctypes.CFUNCTYPE(ctypes.c_int)(lambda: (calls.append(1), 0)[1])
fast.bind(lambda device: 0, *[ctypes.cast(stub, ctypes.c_void_p).value] * 7)

def dev(t):
    return marked_tensors.marked(t)

bf, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
x, w, vec = dev(torch.zeros(4, 64, dtype=bf)), dev(torch.zeros(64, dtype=bf)), dev(torch.zeros(4, dtype=f32))
e = dev(torch.zeros(4, 64, dtype=u8)).view(torch.float8_e4m3fn)
B = dev(torch.zeros(8, 64, dtype=u8)).view(torch.float8_e4m3fn).t()
b = dev(torch.zeros(8, dtype=f32))
codes, scales, zeros = dev(torch.zeros(8, 32, dtype=u8)), dev(torch.zeros(8, 2, dtype=bf)), dev(torch.zeros(8, 2, dtype=u8))
OPERATORS = {{
    "rmsnorm": (fast.rmsnorm, (x, w, x, 1e-6, None)),
    "rmsnorm_backward": (fast.rmsnorm_backward, (x, x, w, x, 1e-6)),
    "gemm_fp8": (fast.gemm_fp8, (e, vec, B, b, None)),
    "gemm_w4": (fast.gemm_w4, (x, codes, scales, zeros)),
}}
name = {operator!r}
f, args = OPERATORS[name]
places = [i for i, a in enumerate(args) if isinstance(a, torch.Tensor)]
assert f(*args) is not NotImplemented and len(calls) >= 1     # the plain call goes through
"""

WRAPPED = """
def with_operand(i, t):
    return f(*args[:i], t, *args[i + 1:])

calls.clear()
for i in places:
    seen = []
    batch = args[i].detach().expand((2,) + tuple(args[i].shape))
    torch.func.vmap(lambda t: (seen.append(with_operand(i, t)), t)[1])(batch)
    if args[i].dtype.is_floating_point:
        torch.func.vjp(lambda t: (seen.append(with_operand(i, t)), t)[1], args[i])
        torch.func.jvp(lambda t: (seen.append(with_operand(i, t)), t)[1], (args[i],), (args[i],))
    assert seen and all(s is NotImplemented for s in seen), (name, i)
    # the interpreter lock and the thread's state are in order
    ctypes.pythonapi.PyGILState_Check.restype = ctypes.c_int
    assert ctypes.pythonapi.PyGILState_Check() == 1
# Nothing was enqueued: only the workspace's size may have been asked for.
assert len(calls) <= len(places) * 3 * (name != "rmsnorm"), calls
print("ok")
"""

SUBCLASS = """
class Mine(torch.Tensor):
    pass

calls.clear()
for i in places:
    out = f(*args[:i], args[i].as_subclass(Mine), *args[i + 1:])
    assert out is NotImplemented, (name, i, type(out))
assert not calls
for i in places:    # a parameter is no subclass to the binding
    if args[i].dtype.is_floating_point:
        assert f(*args[:i], torch.nn.Parameter(args[i]), *args[i + 1:]) is not NotImplemented
print("ok")
"""


@pytest.fixture(scope="module")
def helper(tmp_path_factory):
    where = tmp_path_factory.mktemp("helper")
    t = os.path.dirname(torch.__file__)
    cxx = os.environ.get("CXX") or "g++"
    subprocess.run([cxx, "-O0", "-std=c++17", "-fPIC", "-shared",
                    f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                    "-I", sysconfig.get_paths()["include"], "-I", os.path.join(t, "include"),
                    "-I", os.path.join(t, "include", "torch", "csrc", "api", "include"), "-L", os.path.join(t, "lib"),
                    "-o", str(where / "marked_tensors.so"), os.path.join(ROOT, "tests", "marked_tensors.cpp"),
                    "-ltorch_python", "-ltorch_cpu", "-lc10"], check=True, capture_output=True)
    return str(where)


def run(helper, operator, body):
    assert os.path.exists(build.BINDING)
    code = PROLOGUE.format(root=ROOT, helper=helper, operator=operator) + body
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=120)
    assert res.returncode == 0 and res.stdout.strip() == "ok", f"exit {res.returncode}\n{res.stdout}{res.stderr[-2000:]}"


@pytest.mark.parametrize("operator", ["rmsnorm", "rmsnorm_backward", "gemm_fp8", "gemm_w4"])
def test_operands_of_function_transforms_are_handed_back(helper, operator):
    """A tensor that a function transform wraps has no storage of its own: its address cannot be read, in whichever
    place it stands. The call goes back to the Python wrapper, which words the refusal."""
    run(helper, operator, WRAPPED)


@pytest.mark.parametrize("operator", ["rmsnorm", "rmsnorm_backward", "gemm_fp8", "gemm_w4"])
def test_operands_of_subclasses_are_handed_back(helper, operator):
    run(helper, operator, SUBCLASS)
