"""The microscaled 4-bit form (``include/pipe_linear.h``) and its product:

    pipe_quantize_mxfp4(x, ...)                       -> codes, scales
    pipe_dequantize_mxfp4(codes, scales, ...)         -> x
    pipe_gemm_mxfp4(A, a_scales, W, w_scales, ...)    -> C

A matrix of M rows and K columns, K a multiple of 32, is held as

    codes   (M, K // 2) float4_e2m1fn_x2: two values a byte, the even column's in
            the low four bits, each 0, 0.5, 1, 1.5, 2, 3, 4, 6 or a negative of these;
    scales  (M, K // 32) float8_e8m0fnu: the power of two that 32 neighbours of a
            row are multiplied by, as its exponent plus 127 (255: all 32 are NaN).

They need a PyTorch that has these types; the library's other operators do not.
Bytes that come from elsewhere take them by ``.view(dtype)``. Rows of codes
and of scales start at multiples of 16 bytes, and the memory of a row of scales
reaches the next such multiple: the scales made here are views of wider rows where
K // 32 is no multiple of 16.

As in ``linear.py``, these functions only marshal arguments.
"""
from __future__ import annotations

import ctypes

import async_stage_tile_amd as _pt

from . import linear as _l


def _setup():
    fns = _l._fns or _l._setup()
    if _l._f4 is None:
        raise RuntimeError("the 4-bit form needs a PyTorch with " + " and ".join(f"torch.{n}" for n in _l._FORM))
    return fns


def _wide_dtype(dtype, name):
    """A type that has the 4-bit form: 16 or 32 bits."""
    if _l._codes.get(dtype, _l.PIPE_E4M3) > _l.PIPE_FP32:
        raise TypeError(f"{name} must be bfloat16, float16 or float32, not {dtype}")
    return dtype


def _form(codes, scales, names, device):
    """(rows, columns, pitch of codes, pitch of scales) of a matrix in the form."""
    M, half, ld = _l._matrix(codes, names[0], _l._f4, device)
    if half % 16:
        raise ValueError(f"{names[0]} hold {2 * half} values a row, no multiple of 32")
    return M, 2 * half, ld, _l._scales(scales, names[1], device, M, half // 16)


def _device(t, name):
    return _l._tensor(t, name).get_device()


def pipe_quantize_mxfp4(x, codes=None, scales=None, stream=None):
    """x, (M, K) bfloat16, float16 or float32, in the microscaled 4-bit form: codes
    and scales as above. A block's power of two is the largest one not above its
    largest magnitude, divided by 4; the values divided by it are rounded to nearest,
    ties to the even code, and what passes 6 becomes 6. A block with a NaN or an
    infinity has a NaN scale."""
    fns = _setup()
    if _l._fast and stream is None and codes is None and scales is None:
        made = _l._fast.quantize_mxfp4(x)
        if made is not NotImplemented:
            return made
    _l._check_given(stream)
    dev = _device(x, "x")
    dtype = _wide_dtype(x.dtype, "x")
    M, K, ld_x = _l._matrix(x, "x", dtype, dev)
    if K % 32:
        raise ValueError(f"rows of {K} columns have no 4-bit form: blocks are of 32")
    made = []
    if codes is None:
        codes = _l._make(made, stream, x, (M, K // 2), _l._f4)
        ld_codes = K // 2
    else:
        ld_codes = _l._matrix(codes, "codes", _l._f4, dev, (M, K // 2))[2]
    if scales is None:
        scales = _l._make_scales(made, stream, x, M, K // 32)
    ld_scales = _l._scales(scales, "scales", dev, M, K // 32)
    _l._call(fns.pipe_quantize_mxfp4, "pipe_quantize_mxfp4", dev, stream, made, x.data_ptr(), codes.data_ptr(),
             scales.data_ptr(), M, K, ld_x, ld_codes, ld_scales, _l._codes[dtype])
    _pt._use_on(stream, x, codes, scales)
    return codes, scales


def pipe_dequantize_mxfp4(codes, scales, out_dtype=None, out=None, stream=None):
    """The values that the form stands for, (M, K) in out_dtype: bfloat16 (the
    default), float16 or float32. fp16 rounds what it cannot hold; bf16 and fp32
    hold every value below 2^128, and so all that pipe_quantize_mxfp4 makes."""
    fns = _setup()
    if _l._fast and stream is None and out is None:
        made = _l._fast.dequantize_mxfp4(codes, scales, out_dtype)
        if made is not NotImplemented:
            return made
    _l._check_given(stream)
    dev = _device(codes, "codes")
    M, K, ld_codes, ld_scales = _form(codes, scales, ("codes", "scales"), dev)
    made = []
    if out is None:
        out_dtype = _wide_dtype(out_dtype or _l._torch.bfloat16, "out_dtype")
        out = _l._make(made, stream, codes, (M, K), out_dtype)
        ld_out = K
    else:
        out_dtype = _wide_dtype(out_dtype or _l._tensor(out, "out").dtype, "out")
        ld_out = _l._matrix(out, "out", out_dtype, dev, (M, K))[2]
    _l._call(fns.pipe_dequantize_mxfp4, "pipe_dequantize_mxfp4", dev, stream, made, codes.data_ptr(),
             scales.data_ptr(), out.data_ptr(), M, K, ld_codes, ld_scales, ld_out, _l._codes[out_dtype])
    _pt._use_on(stream, codes, scales, out)
    return out


def pipe_gemm_mxfp4_workspace_bytes(M, N, K) -> int:
    need = _l._Z(0)
    st = (_l._fns or _l._setup()).pipe_gemm_mxfp4_workspace_bytes(M, N, K, ctypes.byref(need))
    _pt._check(st, "pipe_gemm_mxfp4_workspace_bytes")
    return need.value


def pipe_gemm_mxfp4(A, a_scales, W, w_scales, C=None, out_dtype=None, workspace=None, stream=None):
    """C = A @ W.T of M rows A and N rows W (a weight) in the microscaled 4-bit form,
    K columns each. C: (M, N) bfloat16 (the default), float16 or float32. The 32
    products of two blocks add up exactly, the blocks in fp32. What pipe_quantize_mxfp4
    and pipe_layernorm give goes in as it is."""
    fns = _setup()
    if _l._fast and stream is None and C is None and workspace is None:
        made = _l._fast.gemm_mxfp4(A, a_scales, W, w_scales, out_dtype)
        if made is not NotImplemented:
            return made
    _l._check_given(stream, workspace)
    dev = _device(A, "A")
    M, K, lda, ld_as = _form(A, a_scales, ("A", "a_scales"), dev)
    N, Kw, ldw, ld_ws = _form(W, w_scales, ("W", "w_scales"), dev)
    if Kw != K:
        raise ValueError("inner dimensions differ")
    made = []
    if C is None:
        out_dtype = _wide_dtype(out_dtype or _l._torch.bfloat16, "out_dtype")
        C = _l._make(made, stream, A, (M, N), out_dtype)
        ldc = N
    else:
        out_dtype = _wide_dtype(out_dtype or _l._tensor(C, "C").dtype, "C")
        ldc = _l._matrix(C, "C", out_dtype, dev, (M, N))[2]
    ws, ws_bytes = _l._workspace(fns.pipe_gemm_mxfp4_workspace_bytes, "pipe_gemm_mxfp4_workspace_bytes",
                                 (M, N, K), workspace, A, made, stream)
    _l._call(fns.pipe_gemm_mxfp4, "pipe_gemm_mxfp4", dev, stream, made, A.data_ptr(), a_scales.data_ptr(),
             W.data_ptr(), w_scales.data_ptr(), C.data_ptr(), M, N, K, lda, ld_as, ldw, ld_ws, ldc,
             _l._codes[out_dtype], ws, ws_bytes)
    _pt._use_on(stream, A, a_scales, W, w_scales, C, workspace)
    return C
