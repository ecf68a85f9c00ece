"""FP8 (e4m3) operands with an fp32 scale per block of 128: quantisation and the grouped
matrix product of ``include/moe_fp8.h``.

    q, s = fp8.quantize(x)                    # rows [R, K] -> e4m3 [R, K], fp32 [R, ceil(K/128)]
    wq, ws = fp8.quantize_weights(w)          # stacks [E, N, K] -> e4m3, fp32 [E, ceil(N/128), ceil(K/128)]
    y = fp8.matmul(q, s, wq, ws, counts)      # rows in group order, counts [E] on the device -> bf16 [R, N]

The same operands as expert weights of the layer: ``w_dtype="fp8"`` with wq / ws as
``gate_up`` / ``gate_up_scales`` (``fp8.quantize_gate_up``) and ``down`` / ``down_scales``.
Argument marshalling only: the work runs in the CUDA library, on the current stream of
the tensors' device unless one is given (a torch.cuda.Stream, which the caller orders: inputs
ready on it, and kept, until the call has run; outputs read behind it).  Nothing here is
recorded by autograd: outputs of inputs that require a gradient have none.
"""
from __future__ import annotations

import contextlib
import ctypes as C

import torch

import mixture_experts_ffn_10_b200 as _m

EXPORTED = ("moe_fp8_quantize", "moe_fp8_quantize_weights", "moe_fp8_matmul_workspace_size", "moe_fp8_matmul")
BLOCK = 128

_lib = None


def _library():
    """The CUDA library with the entry points of moe_fp8.h declared."""
    global _lib
    if _lib is None:
        _m.moe_version()  # loads it
        lib = _m._lib
        i64, ptr = C.c_int64, C.c_void_p
        lib.moe_fp8_quantize.argtypes = [C.c_int, i64, i64, ptr, i64, ptr, ptr, ptr]
        lib.moe_fp8_quantize_weights.argtypes = [C.c_int, i64, i64, i64, ptr, ptr, ptr, ptr]
        lib.moe_fp8_matmul_workspace_size.argtypes = [i64, i64, i64, i64]
        lib.moe_fp8_matmul_workspace_size.restype = C.c_size_t
        lib.moe_fp8_matmul.argtypes = [i64, i64, i64, i64, ptr, ptr, ptr, ptr, ptr, ptr, ptr, C.c_size_t, ptr]
        _lib = lib
    return _lib


_NOTHING = contextlib.nullcontext()


def _on(device, stream=None):
    """The package's _on, without its call in the usual case."""
    if stream is None and device.type == "cuda" and device.index == torch.cuda.current_device():
        return _NOTHING
    return _m._on(device, stream)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # current_stream without its object: 2 us less


def _stream(stream, device):
    if stream is None and _raw_stream is not None:
        return _raw_stream(device.index)
    return (stream if stream is not None else torch.cuda.current_stream(device)).cuda_stream


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return _m.MOE_BF16
    if t.dtype == torch.float32:
        return _m.MOE_F32
    raise ValueError(f"expected bfloat16 or float32, got {t.dtype}")


def _cdiv(a, b):
    return -(-a // b)


def quantize(x, stream=None):
    """Rows of activations x [R, K] (bf16 or fp32; rows may be pitched, columns contiguous) ->
    (q [R, K] float8_e4m3fn, scales [R, ceil(K/128)] fp32)."""
    if x.dim() != 2 or (x.stride(1) != 1 and x.shape[1] > 1):
        raise ValueError("x must be [R, K] with contiguous columns")
    R, K = x.shape
    pitch = x.stride(0) if R > 1 else K
    if pitch < K:
        raise ValueError("the rows of x overlap")
    with _on(x.device, stream):
        q = torch.empty_like(x, dtype=torch.float8_e4m3fn, memory_format=torch.contiguous_format)
        s = x.new_empty((R, _cdiv(K, BLOCK)), dtype=torch.float32)
        _m._check(_library().moe_fp8_quantize(_dtype_code(x), R, K, x.data_ptr(), pitch, q.data_ptr(), s.data_ptr(),
                                              _stream(stream, x.device)))
    if stream is not None:
        _m._handed(x.device, stream, q, s)
    return q, s


def quantize_weights(w, stream=None):
    """Weight stacks w [E, N, K] (or one matrix [N, K]; bf16 or fp32, contiguous) ->
    (q like w float8_e4m3fn, scales [E, ceil(N/128), ceil(K/128)] fp32)."""
    if w.dim() not in (2, 3) or not w.is_contiguous():
        raise ValueError("w must be a contiguous [E, N, K] or [N, K]")
    *lead, N, K = w.shape
    E = lead[0] if lead else 1
    with _on(w.device, stream):
        q = torch.empty(w.shape, dtype=torch.float8_e4m3fn, device=w.device)
        s = torch.empty((*lead, _cdiv(N, BLOCK), _cdiv(K, BLOCK)), dtype=torch.float32, device=w.device)
        _m._check(_library().moe_fp8_quantize_weights(_dtype_code(w), E, N, K, w.data_ptr(), q.data_ptr(), s.data_ptr(),
                                                      _stream(stream, w.device)))
    if stream is not None:
        _m._handed(w.device, stream, q, s)
    return q, s


def quantize_gate_up(w, stream=None):
    """A concat gate||up stack [E, 2F, d] as the layer takes it: the gate rows and the up rows
    of an expert have blocks of their own -> (q [E, 2F, d], scales [E, 2 ceil(F/128), ceil(d/128)])."""
    E, F2, d = w.shape
    if F2 % 2:
        raise ValueError("a gate||up stack has an even number of rows")
    with _on(w.device, stream):  # (a stack that is not contiguous is copied)
        halves = w.reshape(2 * E, F2 // 2, d)
    q, s = quantize_weights(halves, stream)
    return q.view(E, F2, d), s.view(E, -1, s.shape[2])


def _operand(name, t, dtype, shape, device):
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous {dtype} {list(shape)} on {device}, got {t.dtype} {list(t.shape)} "
                         f"on {t.device}")


def matmul(xq, xs, wq, ws, counts=None, y=None, workspace=None, stream=None):
    """Grouped product of quantised rows xq [R, K], xs and weights wq [E, N, K], ws -> y [R, N] bf16:
    the first counts[0] rows by wq[0], the next counts[1] by wq[1], ... (counts [E] int32 on the
    device; None with one matrix: every row).  wq may be one matrix [N, K].  Rows past the sum of
    the counts are not written (a y allocated here holds anything there).  workspace: a Workspace
    of at least moe_fp8_matmul_workspace_size bytes, for callers that keep one."""
    if xq.dim() != 2 or wq.dim() not in (2, 3):
        raise ValueError("xq must be [R, K] and wq [E, N, K] or [N, K]")
    R, K = xq.shape
    lead, N = tuple(wq.shape[:-2]), wq.shape[-2]
    E = lead[0] if lead else 1
    dev, nbk = xq.device, _cdiv(K, BLOCK)
    _operand("xq", xq, torch.float8_e4m3fn, (R, K), dev)
    _operand("xs", xs, torch.float32, (R, nbk), dev)
    _operand("wq", wq, torch.float8_e4m3fn, (*lead, N, K), dev)
    _operand("ws", ws, torch.float32, (*lead, _cdiv(N, BLOCK), nbk), dev)
    if counts is not None:
        _operand("counts", counts, torch.int32, (E,), dev)
    if y is not None:
        _operand("y", y, torch.bfloat16, (R, N), dev)
    made = y is None
    with _on(dev, stream):
        lib = _library()
        if made:
            y = torch.empty((R, N), dtype=torch.bfloat16, device=dev)
        if workspace is None:
            workspace = _m.Workspace(lib.moe_fp8_matmul_workspace_size(R, E, N, K), dev)
        _m._check(lib.moe_fp8_matmul(R, E, N, K, xq.data_ptr(), xs.data_ptr(), wq.data_ptr(), ws.data_ptr(),
                                     None if counts is None else counts.data_ptr(), y.data_ptr(), workspace.ptr,
                                     workspace.nbytes, _stream(stream, dev)))
    if made and stream is not None:
        _m._handed(dev, stream, y)
    return y
