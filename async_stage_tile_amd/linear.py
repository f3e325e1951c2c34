"""The operators of a quantised linear layer (``include/pipe_linear.h``):

    pipe_rmsnorm(x, weight, residual=None, ...)        -> y [, scales] [, h]
    pipe_rmsnorm_backward(dy, x, weight, dh=None, ...) -> dx, dweight
    pipe_gemm_fp8(A, a_scales, B, b_scales, ...)       -> C
    pipe_gemm_w4(A, codes, scales, zeros=None, ...)    -> C
    pipe_layernorm(x, weight, bias=None, residual=None, ...)  -> y [, scales] [, h]
    pipe_layernorm_backward(dy, x, weight, dh=None, ...)      -> dx, dweight, dbias

and, in ``mxfp4.py``, those of the microscaled 4-bit form.

Argument marshalling only, as in the package's other functions: the work is
done by the HIP kernels of the shared library, on the given stream or the
current one. Outputs that are not given are allocated, and so are the
workspaces that a shape needs, from the memory pool of the stream that the work
goes to. Wrong arguments raise TypeError or ValueError here, or PipeError with
the library's status, and then nothing is enqueued.

The common case (contiguous operands, outputs made here, the current stream)
goes through ``_linear.so``, the same marshalling in C++, which the build makes
next to the library; it hands back what it does not take.
"""
from __future__ import annotations

import ctypes
import threading

import async_stage_tile_amd as _pt

PIPE_BF16 = 0
PIPE_FP16 = 1
PIPE_FP32 = 2
PIPE_E4M3 = 3
PIPE_MXFP4 = 4
PIPE_RMSNORM_MAX_N = 32768
PIPE_LAYERNORM_MAX_N = 32768

_c = ctypes
_V, _L, _F, _I, _Z = _c.c_void_p, _c.c_int64, _c.c_float, _c.c_int, _c.c_size_t
_LINEAR_SIGS = {
    "pipe_rmsnorm": [_V] * 6 + [_L] * 6 + [_F, _I, _I, _V],
    "pipe_rmsnorm_backward_workspace_bytes": [_L, _L, _c.POINTER(_Z)],
    "pipe_rmsnorm_backward": [_V] * 6 + [_L] * 6 + [_F, _I, _V, _Z, _V],
    "pipe_gemm_fp8_workspace_bytes": [_L, _L, _L, _c.POINTER(_Z)],
    "pipe_gemm_fp8": [_V] * 5 + [_L] * 6 + [_I, _V, _Z, _V],
    "pipe_gemm_w4_workspace_bytes": [_L, _L, _L, _c.POINTER(_Z)],
    "pipe_gemm_w4": [_V] * 5 + [_L] * 9 + [_I, _V, _Z, _V],
    "pipe_layernorm": [_V] * 7 + [_L] * 7 + [_F, _I, _I, _V],
    "pipe_layernorm_backward_workspace_bytes": [_L, _L, _c.POINTER(_Z)],
    "pipe_layernorm_backward": [_V] * 7 + [_L] * 6 + [_F, _I, _V, _Z, _V],
    "pipe_quantize_mxfp4": [_V] * 3 + [_L] * 5 + [_I, _V],
    "pipe_dequantize_mxfp4": [_V] * 3 + [_L] * 5 + [_I, _V],
    "pipe_gemm_mxfp4_workspace_bytes": [_L, _L, _L, _c.POINTER(_Z)],
    "pipe_gemm_mxfp4": [_V] * 5 + [_L] * 8 + [_I, _V, _Z, _V],
}
_FORM = ("float4_e2m1fn_x2", "float8_e8m0fnu")     # the 4-bit form's codes and scales in torch
_FIRST = 7      # the C++ marshalling's bind() takes so many, bind_layer() the rest

_fns = None
_lock = threading.Lock()
_torch = None
_codes = {}         # torch dtype -> pipe_dtype_t
_current_stream = None      # address of a device's current stream
_fast = None                # the C++ marshalling, or None where it was not built
_f4 = _e8 = None            # the 4-bit form's dtypes, None where torch lacks one of them


def linear_symbols():
    """The functions of pipe_linear.h."""
    return list(_LINEAR_SIGS)


def _setup():
    """Loads the library once and binds the functions; torch is imported with
    the first call, as everywhere in this package."""
    global _fns, _torch, _current_stream, _fast, _f4, _e8
    with _lock:
        if _fns is None:
            L = _pt.lib()

            class Fns:
                pass

            fns = Fns()
            for name, args in _LINEAR_SIGS.items():
                fn = getattr(L, name)
                fn.restype = _I
                fn.argtypes = args
                setattr(fns, name, fn)
            import torch
            _codes.update({torch.bfloat16: PIPE_BF16, torch.float16: PIPE_FP16,
                           torch.float32: PIPE_FP32, torch.float8_e4m3fn: PIPE_E4M3})
            form = [getattr(torch, name, None) for name in _FORM]
            if None not in form:
                _f4, _e8 = form
                _codes[_f4] = PIPE_MXFP4
            # The address alone, without the Stream object around it (1 us a call).
            _current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
                lambda device: torch.cuda.current_stream(device).cuda_stream)
            _torch = torch
            try:
                from . import _linear as fast
            except ImportError:     # not built, or for another Python
                fast = None
            if fast is not None:
                at = [_c.cast(getattr(fns, n), _V).value for n in _LINEAR_SIGS]
                fast.bind(_current_stream, *at[:_FIRST])
                fast.bind_layer(*at[_FIRST:])
            _fast = fast
            _fns = fns
    return _fns


def _matrix(t, name, dtype, device, shape=None):
    """(rows, cols, pitch) of a 2-D row-major device tensor of the dtype on
    the device; the shape, where one is given, must match. The calls here are
    as long as a small kernel, so the common case asks little."""
    try:
        if (t.dtype is dtype and t.get_device() == device and device >= 0
                and (shape is None or t.shape == shape) and t.is_contiguous()):
            rows, cols = t.shape
            return rows, cols, cols
    except (AttributeError, ValueError):    # no tensor, or not two axes
        pass
    _tensor(t, name)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if device < 0:
        raise ValueError(f"{name} must be a device tensor")
    if t.get_device() != device:
        raise ValueError(f"{name} must be a tensor on device cuda:{device}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    return _pt.matrix_geometry(t.shape, t.stride(), name)


def _vector(t, name, dtype, device, n):
    """Address of a contiguous vector of n elements."""
    _tensor(t, name)
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be a tensor on device cuda:{device}")
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of {n} elements")
    return t.data_ptr()


def _dtype16(t, name):
    dtype = _tensor(t, name).dtype
    if _codes.get(dtype, PIPE_FP32) > PIPE_FP16:
        raise TypeError(f"{name} must be bfloat16 or float16, not {dtype}")
    return dtype


def _tensor(t, name):
    if not isinstance(t, _torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    return t


def _check_given(stream, workspace=None):
    """The types of arguments whose attributes are used further on."""
    if stream is not None and not isinstance(stream, _torch.cuda.Stream):
        raise TypeError("stream must be a torch.cuda.Stream")
    if workspace is not None:
        _tensor(workspace, "workspace")


def _make(made, stream, like, shape, dtype):
    """A tensor for work on `stream`, noted in `made`."""
    if stream is None:
        t = like.new_empty(shape, dtype=dtype)
    else:
        with _pt._allocating_for(stream):
            t = like.new_empty(shape, dtype=dtype)
    made.append(t)
    return t


def _call(fn, name, device, stream, made, *args):
    """The C call with the tensors' device current, on the given stream or the
    device's current one, which goes last; `made`: the tensors allocated here."""
    if stream is None:
        raw = _current_stream(device)
    else:
        if stream.device.index != device:
            raise ValueError(f"stream of {stream.device} for tensors on cuda:{device}")
        raw = stream.cuda_stream
    if _torch.cuda.current_device() == device:
        st = fn(*args, raw)
    else:
        with _torch.cuda.device(device):
            st = fn(*args, raw)
    if st:
        raise _pt.PipeError(st, name)
    if stream is not None:
        _pt._hold_for(stream, device, *made)


def pipe_rmsnorm(x, weight, residual=None, eps=1e-6, out_dtype=None, y=None, y_scales=None, h=None,
                 stream=None):
    """RMS norm of each row, the residual added first where one is given:
    h = x + residual (rounded to x's type), y = h * rsqrt(mean(h^2) + eps) * weight.

    x, residual: (M, N) bfloat16 or float16; weight: (N). out_dtype: x's type
    (the default), or torch.float8_e4m3fn, whose rows are scaled by
    scales[m] = max|y[m]| / 448 (y = values * scales). Returns y; with e4m3
    y, scales; with a residual the new stream h last: (y, h) or (y, scales, h).
    h may be x or residual itself to update the stream in place."""
    fns = _fns or _setup()
    if _fast and stream is None and y is None and h is None and y_scales is None:
        out = _fast.rmsnorm(x, weight, residual, eps, out_dtype)
        if out is not NotImplemented:
            return out
    _check_given(stream)
    eps = float(eps)
    dtype = _dtype16(x, "x")
    dev = x.get_device()
    M, N, ld_x = _matrix(x, "x", dtype, dev)
    out_dtype = out_dtype or (dtype if y is None else _tensor(y, "y").dtype)
    if out_dtype is not dtype and out_dtype is not _torch.float8_e4m3fn:
        raise TypeError(f"out_dtype must be {dtype} or float8_e4m3fn, not {out_dtype}")
    w = _vector(weight, "weight", dtype, dev, N)
    made = []
    if y is None:
        y = _make(made, stream, x, (M, N), out_dtype)
        ld_y = N
    else:
        ld_y = _matrix(y, "y", out_dtype, dev, (M, N))[2]
    q8 = out_dtype is not dtype
    scales = 0
    if q8:
        if y_scales is None:
            y_scales = _make(made, stream, x, (M,), _torch.float32)
            scales = y_scales.data_ptr()
        else:
            scales = _vector(y_scales, "y_scales", _torch.float32, dev, M)
    elif y_scales is not None:
        raise ValueError("y_scales go with an e4m3 output")
    r_ptr = h_ptr = ld_r = ld_h = 0
    if residual is not None:
        ld_r = _matrix(residual, "residual", dtype, dev, (M, N))[2]
        r_ptr = residual.data_ptr()
        if h is None:
            h = _make(made, stream, x, (M, N), dtype)
            ld_h = N
        else:
            ld_h = _matrix(h, "h", dtype, dev, (M, N))[2]
        h_ptr = h.data_ptr()
    elif h is not None:
        raise ValueError("h goes with a residual")
    _call(fns.pipe_rmsnorm, "pipe_rmsnorm", dev, stream, made, x.data_ptr(), r_ptr, w, y.data_ptr(),
          scales, h_ptr, M, N, ld_x, ld_r, ld_y, ld_h, eps, _codes[dtype], _codes[out_dtype])
    _pt._use_on(stream, x, weight, residual, y, y_scales, h)
    if residual is None:
        return (y, y_scales) if q8 else y
    return (y, y_scales, h) if q8 else (y, h)


def pipe_rmsnorm_backward(dy, x, weight, dh=None, eps=1e-6, dx=None, dweight=None, workspace=None,
                          stream=None):
    """Gradient of pipe_rmsnorm's y for its normalised input x (its h where a
    residual was added): dx (x's type) and dweight (float32). dh: the gradient
    that reaches h along the residual stream, added to dx before its rounding;
    dx is then the gradient of both addends."""
    fns = _fns or _setup()
    if _fast and stream is None and dx is None and dweight is None and workspace is None:
        out = _fast.rmsnorm_backward(dy, x, weight, dh, eps)
        if out is not NotImplemented:
            return out
    _check_given(stream, workspace)
    eps = float(eps)
    dtype = _dtype16(x, "x")
    dev = x.get_device()
    M, N, ld_x = _matrix(x, "x", dtype, dev)
    ld_dy = _matrix(dy, "dy", dtype, dev, (M, N))[2]
    w = _vector(weight, "weight", dtype, dev, N)
    dh_ptr = ld_dh = 0
    if dh is not None:
        ld_dh = _matrix(dh, "dh", dtype, dev, (M, N))[2]
        dh_ptr = dh.data_ptr()
    made = []
    if dx is None:
        dx = _make(made, stream, x, (M, N), dtype)
        ld_dx = N
    else:
        ld_dx = _matrix(dx, "dx", dtype, dev, (M, N))[2]
    if dweight is None:
        dweight = _make(made, stream, x, (N,), _torch.float32)
    else:
        _vector(dweight, "dweight", _torch.float32, dev, N)
    ws, ws_bytes = _workspace(fns.pipe_rmsnorm_backward_workspace_bytes,
                              "pipe_rmsnorm_backward_workspace_bytes", (M, N), workspace, x, made, stream)
    _call(fns.pipe_rmsnorm_backward, "pipe_rmsnorm_backward", dev, stream, made, dy.data_ptr(),
          x.data_ptr(), w, dh_ptr, dx.data_ptr(), dweight.data_ptr(), M, N, ld_dy, ld_x, ld_dh,
          ld_dx, eps, _codes[dtype], ws, ws_bytes)
    _pt._use_on(stream, dy, x, weight, dh, dx, dweight, workspace)
    return dx, dweight


def _workspace(fn, name, shape, given, like, made, stream):
    """(address, bytes) of a call's workspace: the given tensor, or one made here."""
    if given is not None:
        if not given.is_contiguous() or given.get_device() != like.get_device():
            raise ValueError("workspace must be a contiguous tensor on the operands' device")
        return given.data_ptr(), given.numel() * given.element_size()
    need = _Z(0)
    st = fn(*shape, ctypes.byref(need))
    if st:
        raise _pt.PipeError(st, name)
    size = need.value
    if size == 0:
        return 0, 0
    return _make(made, stream, like, (size,), _torch.uint8).data_ptr(), size


def pipe_rmsnorm_backward_workspace_bytes(M, N) -> int:
    need = _Z(0)
    st = (_fns or _setup()).pipe_rmsnorm_backward_workspace_bytes(M, N, ctypes.byref(need))
    _pt._check(st, "pipe_rmsnorm_backward_workspace_bytes")
    return need.value


def pipe_gemm_fp8_workspace_bytes(M, N, K) -> int:
    need = _Z(0)
    st = (_fns or _setup()).pipe_gemm_fp8_workspace_bytes(M, N, K, ctypes.byref(need))
    _pt._check(st, "pipe_gemm_fp8_workspace_bytes")
    return need.value


def pipe_gemm_fp8(A, a_scales, B, b_scales, C=None, out_dtype=None, workspace=None, stream=None):
    """C = (A @ B) * a_scales[:, None] * b_scales[None, :].

    A: (M, K) float8_e4m3fn, row-major; B: (K, N) float8_e4m3fn with unit row
    stride (the transpose of a row-major (N, K) weight); scales: float32 of M
    and N elements. C: bfloat16 (the default), float16 or float32. The sums are
    fp32 sums; for bfloat16 C and five rows or more those of the 8-bit matrix
    instructions, which keep 13 bits below the largest of each eight products
    (1.5e-5 to 2e-4 of the result's norm) and run at twice the rate."""
    fns = _fns or _setup()
    if _fast and stream is None and C is None and workspace is None:
        out = _fast.gemm_fp8(A, a_scales, B, b_scales, out_dtype)
        if out is not NotImplemented:
            return out
    _check_given(stream, workspace)
    e4m3 = _torch.float8_e4m3fn
    dev = A.get_device() if isinstance(A, _torch.Tensor) else -1
    M, K, lda = _matrix(A, "A", e4m3, dev)
    if not isinstance(B, _torch.Tensor) or B.dim() != 2:
        raise TypeError("B must be a 2-D torch.Tensor")
    N, Kb, ldb = _matrix(B.t(), "B (its transpose)", e4m3, dev)
    if Kb != K:
        raise ValueError("inner dimensions differ")
    sa = _vector(a_scales, "a_scales", _torch.float32, dev, M)
    sb = _vector(b_scales, "b_scales", _torch.float32, dev, N)
    made = []
    if C is None:
        out_dtype = out_dtype or _torch.bfloat16
        if _codes.get(out_dtype, PIPE_E4M3) > PIPE_FP32:
            raise TypeError(f"out_dtype must be bfloat16, float16 or float32, not {out_dtype}")
        C = _make(made, stream, A, (M, N), out_dtype)
        ldc = N
    else:
        out_dtype = out_dtype or _tensor(C, "C").dtype
        if _codes.get(out_dtype, PIPE_E4M3) > PIPE_FP32:
            raise TypeError(f"C must be bfloat16, float16 or float32, not {out_dtype}")
        ldc = _matrix(C, "C", out_dtype, dev, (M, N))[2]
    ws, ws_bytes = _workspace(fns.pipe_gemm_fp8_workspace_bytes, "pipe_gemm_fp8_workspace_bytes",
                              (M, N, K), workspace, A, made, stream)
    _call(fns.pipe_gemm_fp8, "pipe_gemm_fp8", dev, stream, made, A.data_ptr(), sa, B.data_ptr(), sb,
          C.data_ptr(), M, N, K, lda, ldb, ldc, _codes[out_dtype], ws, ws_bytes)
    _pt._use_on(stream, A, a_scales, B, b_scales, C, workspace)
    return C


def pipe_gemm_w4_workspace_bytes(M, N, K) -> int:
    need = _Z(0)
    st = (_fns or _setup()).pipe_gemm_w4_workspace_bytes(M, N, K, ctypes.byref(need))
    _pt._check(st, "pipe_gemm_w4_workspace_bytes")
    return need.value


def pipe_gemm_w4(A, codes, scales, zeros=None, C=None, workspace=None, stream=None):
    """C = A @ W.T for 4-bit weights W[n][k] = (q[n][k] - z[n][k // group]) * scales[n][k // group].

    A: (M, K) bfloat16 or float16; codes: (N, K // 2) uint8, the code of an
    even k in the low half of its byte; scales: (N, K // group) of A's type;
    zeros: (N, K // group) uint8 of 0..15, None for 8 everywhere. The group
    size is K divided by the scales' columns: a power of two >= 32, or K."""
    fns = _fns or _setup()
    if _fast and stream is None and C is None and workspace is None:
        out = _fast.gemm_w4(A, codes, scales, zeros)
        if out is not NotImplemented:
            return out
    _check_given(stream, workspace)
    dtype = _dtype16(A, "A")
    dev = A.get_device()
    M, K, lda = _matrix(A, "A", dtype, dev)
    N, half, ld_codes = _matrix(codes, "codes", _torch.uint8, dev)
    if half * 2 != K:
        raise ValueError(f"codes hold {half * 2} weights a row, A {K} columns")
    Ns, groups, ld_scales = _matrix(scales, "scales", dtype, dev)
    if Ns != N or (K > 0 and (groups == 0 or K % groups != 0)):
        raise ValueError("scales must have a row for each row of codes and a column for each group")
    z_ptr = ld_zeros = 0
    if zeros is not None:
        ld_zeros = _matrix(zeros, "zeros", _torch.uint8, dev, (N, groups))[2]
        z_ptr = zeros.data_ptr()
    made = []
    if C is None:
        C = _make(made, stream, A, (M, N), dtype)
        ldc = N
    else:
        ldc = _matrix(C, "C", dtype, dev, (M, N))[2]
    ws, ws_bytes = _workspace(fns.pipe_gemm_w4_workspace_bytes, "pipe_gemm_w4_workspace_bytes",
                              (M, N, K), workspace, A, made, stream)
    _call(fns.pipe_gemm_w4, "pipe_gemm_w4", dev, stream, made, A.data_ptr(), codes.data_ptr(),
          scales.data_ptr(), z_ptr, C.data_ptr(), M, N, K, K // groups if groups else 0, lda,
          ld_codes, ld_scales, ld_zeros, ldc, _codes[dtype], ws, ws_bytes)
    _pt._use_on(stream, A, codes, scales, zeros, C, workspace)
    return C


def _padded(n):
    """The pitch of n bytes' rows that start at multiples of 16 bytes."""
    return -(-n // 16) * 16


def _make_scales(made, stream, like, rows, blocks):
    """e8m0 scales of rows that start at multiples of 16 bytes."""
    return _make(made, stream, like, (rows, _padded(blocks)), _e8)[:, :blocks]


def _scales(t, name, device, rows, blocks):
    """Pitch of a matrix of e8m0 scales. The kernels read its rows in groups of
    16 bytes, so the last row's group has to lie in the tensor's memory."""
    pitch = _matrix(t, name, _e8, device, (rows, blocks))[2]
    if rows <= 1:
        pitch = _padded(blocks)
    if rows and t.storage_offset() + (rows - 1) * pitch + _padded(blocks) > t.untyped_storage().nbytes():
        raise ValueError(f"{name}: the memory of the last row must reach a multiple of 16 bytes "
                         "(rows of scales are read in groups of 16)")
    return pitch


def pipe_layernorm(x, weight, bias=None, residual=None, eps=1e-5, out_dtype=None, y=None, y_scales=None,
                   h=None, stream=None):
    """Layer norm of each row, the residual added first where one is given:
    h = x + residual (rounded to x's type), m = mean(h),
    y = (h - m) * rsqrt(mean((h - m)^2) + eps) * weight + bias.

    x, residual: (M, N) bfloat16 or float16; weight, bias: (N). out_dtype: x's
    type (the default); torch.float8_e4m3fn, whose rows are scaled by scales[m] =
    max|y[m]| / 448; or torch.float4_e2m1fn_x2, the microscaled 4-bit form of
    pipe_quantize_mxfp4 (N a multiple of 32). Returns y; with e4m3 or 4 bits y,
    scales; with a residual the new stream h last: (y, h) or (y, scales, h).
    h may be x or residual itself to update the stream in place. Finite rows whose
    squared deviations add up past fp32's range (bf16's largest values) give the bias."""
    fns = _fns or _setup()
    if _fast and stream is None and y is None and h is None and y_scales is None:
        out = _fast.layernorm(x, weight, bias, residual, eps, out_dtype)
        if out is not NotImplemented:
            return out
    _check_given(stream)
    eps = float(eps)
    dtype = _dtype16(x, "x")
    dev = x.get_device()
    M, N, ld_x = _matrix(x, "x", dtype, dev)
    out_dtype = out_dtype or (dtype if y is None else _tensor(y, "y").dtype)
    q8, mx = out_dtype is _torch.float8_e4m3fn, out_dtype is _f4
    if out_dtype is not dtype and not q8 and not mx:
        raise TypeError(f"out_dtype must be {dtype}, float8_e4m3fn or float4_e2m1fn_x2, not {out_dtype}")
    if mx and N % 32:
        raise ValueError(f"rows of {N} columns have no 4-bit form: blocks are of 32")
    w = _vector(weight, "weight", dtype, dev, N)
    b = 0 if bias is None else _vector(bias, "bias", dtype, dev, N)
    made = []
    shape = (M, N // 2) if mx else (M, N)
    if y is None:
        y = _make(made, stream, x, shape, out_dtype)
        ld_y = shape[1]
    else:
        ld_y = _matrix(y, "y", out_dtype, dev, shape)[2]
    scales = ld_s = 0
    if mx:
        if y_scales is None:
            y_scales = _make_scales(made, stream, x, M, N // 32)
        ld_s = _scales(y_scales, "y_scales", dev, M, N // 32)
        scales = y_scales.data_ptr()
    elif q8:
        if y_scales is None:
            y_scales = _make(made, stream, x, (M,), _torch.float32)
            scales = y_scales.data_ptr()
        else:
            scales = _vector(y_scales, "y_scales", _torch.float32, dev, M)
    elif y_scales is not None:
        raise ValueError("y_scales go with an e4m3 or a 4-bit output")
    r_ptr = h_ptr = ld_r = ld_h = 0
    if residual is not None:
        ld_r = _matrix(residual, "residual", dtype, dev, (M, N))[2]
        r_ptr = residual.data_ptr()
        if h is None:
            h = _make(made, stream, x, (M, N), dtype)
            ld_h = N
        else:
            ld_h = _matrix(h, "h", dtype, dev, (M, N))[2]
        h_ptr = h.data_ptr()
    elif h is not None:
        raise ValueError("h goes with a residual")
    _call(fns.pipe_layernorm, "pipe_layernorm", dev, stream, made, x.data_ptr(), r_ptr, w, b, y.data_ptr(),
          scales, h_ptr, M, N, ld_x, ld_r, ld_y, ld_s, ld_h, eps, _codes[dtype], _codes[out_dtype])
    _pt._use_on(stream, x, weight, bias, residual, y, y_scales, h)
    out = (y, y_scales) if q8 or mx else (y,)
    if residual is not None:
        out += (h,)
    return out if len(out) > 1 else y


def pipe_layernorm_backward_workspace_bytes(M, N) -> int:
    need = _Z(0)
    st = (_fns or _setup()).pipe_layernorm_backward_workspace_bytes(M, N, ctypes.byref(need))
    _pt._check(st, "pipe_layernorm_backward_workspace_bytes")
    return need.value


def pipe_layernorm_backward(dy, x, weight, dh=None, eps=1e-5, dx=None, dweight=None, dbias=None,
                            workspace=None, stream=None):
    """Gradient of pipe_layernorm's y for its normalised input x (its h where a
    residual was added): dx (x's type), dweight and dbias (float32). dh: the
    gradient that reaches h along the residual stream, added to dx before its
    rounding; dx is then the gradient of both addends."""
    fns = _fns or _setup()
    if _fast and stream is None and dx is None and dweight is None and dbias is None and workspace is None:
        out = _fast.layernorm_backward(dy, x, weight, dh, eps)
        if out is not NotImplemented:
            return out
    _check_given(stream, workspace)
    eps = float(eps)
    dtype = _dtype16(x, "x")
    dev = x.get_device()
    M, N, ld_x = _matrix(x, "x", dtype, dev)
    ld_dy = _matrix(dy, "dy", dtype, dev, (M, N))[2]
    w = _vector(weight, "weight", dtype, dev, N)
    dh_ptr = ld_dh = 0
    if dh is not None:
        ld_dh = _matrix(dh, "dh", dtype, dev, (M, N))[2]
        dh_ptr = dh.data_ptr()
    made = []
    if dx is None:
        dx = _make(made, stream, x, (M, N), dtype)
        ld_dx = N
    else:
        ld_dx = _matrix(dx, "dx", dtype, dev, (M, N))[2]
    sums = []
    for t, name in ((dweight, "dweight"), (dbias, "dbias")):
        if t is None:
            t = _make(made, stream, x, (N,), _torch.float32)
        else:
            _vector(t, name, _torch.float32, dev, N)
        sums.append(t)
    dweight, dbias = sums
    ws, ws_bytes = _workspace(fns.pipe_layernorm_backward_workspace_bytes,
                              "pipe_layernorm_backward_workspace_bytes", (M, N), workspace, x, made, stream)
    _call(fns.pipe_layernorm_backward, "pipe_layernorm_backward", dev, stream, made, dy.data_ptr(),
          x.data_ptr(), w, dh_ptr, dx.data_ptr(), dweight.data_ptr(), dbias.data_ptr(), M, N, ld_dy, ld_x,
          ld_dh, ld_dx, eps, _codes[dtype], ws, ws_bytes)
    _pt._use_on(stream, dy, x, weight, dh, dx, dweight, dbias, workspace)
    return dx, dweight, dbias
