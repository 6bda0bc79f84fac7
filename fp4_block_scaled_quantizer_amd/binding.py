"""ctypes binding of ``libfp4q.so`` with the C ABI's entry-point names.

Argument marshalling only: every step of the quantizers, GEMMs and row-wise
operators runs in the library's HIP kernels.  PyTorch supplies device memory (``data_ptr()``) and the
stream (``torch.cuda.current_stream()``, or the one a call names with
``stream``, whose memory the outputs made for it then are).  If the library has
not been built this module raises -- there is no fallback path.  No call
records itself for autograd: an input may require grad, the outputs never do,
and the gradients are calls of their own.
"""
from __future__ import annotations

import ctypes
import math
import os
import re
from typing import NamedTuple, Optional, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp4q.so")
ROW_CALLS_PATH = os.path.join(_HERE, "_row_calls.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "fp4q.h")

# enums of include/fp4q.h
OK, EINVAL, ESHAPE, EALIGN, ELAUNCH, EUNSUPPORTED = 0, 1, 2, 3, 4, 5
ALONG_ROWS, ALONG_COLS = 0, 1
RNE, SR = 0, 1
NV_GLOBAL, NV_TILE128 = 0, 1
LAYOUT_LINEAR, LAYOUT_TILED = 0, 1
OUT_F32, OUT_BF16 = 0, 1
NORM_LAYER, NORM_RMS = 0, 1
ROTARY_HALF, ROTARY_INTERLEAVED = 0, 1

_lib = None


class Fp4qError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed with status {status}: {status_str(status)}")
        self.status = status


def declared_functions():
    """Names of the functions include/fp4q.h declares."""
    with open(HEADER) as f:
        text = f.read()
    return re.findall(r"^FP4Q_API\s+[\w\s\*]*?\b(\w+)\s*\(", text, flags=re.MULTILINE)


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise FileNotFoundError(
            f"{LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'` "
            "(hipcc, gfx950); libfp4q has no CPU fallback")
    L = ctypes.CDLL(LIB_PATH)
    vp, i64, u64, u32, i32, f32 = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint64, ctypes.c_uint32,
                                   ctypes.c_int, ctypes.c_float)
    L.fp4_quantize_mx.argtypes = [vp, i64, i64, i64, i32, i32, u64, u32, vp, vp, i32, vp]
    L.fp4_hadamard32_quantize.argtypes = [vp, i64, i64, i64, i32, u32, i32, u64, u32, vp, vp, i32, vp]
    L.fp4_quantize_mx_dual.argtypes = [vp, i64, i64, i64, i32, u32, vp, vp, i32, u32, i32, u32, vp, vp, u64, i32,
                                       vp]
    L.fp4q_nv_workspace_bytes.argtypes = [i64, i64, i32, i32]
    L.fp4q_nv_workspace_bytes.restype = ctypes.c_size_t
    L.fp4_quantize_nv.argtypes = [vp, i64, i64, i64, i32, i32, u64, u32, i32, vp, vp, vp, vp, ctypes.c_size_t,
                                  i32, vp]
    L.fp4_gemm_mx.argtypes = [vp, vp, vp, vp, i64, i64, i64, f32, i32, vp, i32, i64, vp]
    L.fp4_gemm_nv.argtypes = [vp, vp, vp, vp, vp, vp, i32, i64, i64, i64, f32, i32, vp, i32, i64, vp]
    L.fp4_gemm_mx_amax.argtypes = [vp, vp, vp, vp, i64, i64, i64, f32, i32, vp, i32, i64, vp, vp]
    L.fp4_gemm_mx_quant.argtypes = [vp, vp, vp, vp, i64, i64, i64, f32, i32, vp, vp, i32, vp]
    L.fp4_gemm_mx_swiglu_quant.argtypes = [vp, vp, vp, vp, i64, i64, i64, f32, i32, vp, vp, i32, vp]
    L.fp4_swiglu_bf16.argtypes = [vp, i64, i64, i64, i64, vp, i64, vp]
    L.fp4_gemm_nv_amax.argtypes = [vp, vp, vp, vp, vp, vp, i32, i64, i64, i64, f32, i32, vp, i32, i64, vp, vp]
    L.fp4_quantize_nv_amax.argtypes = [vp, i64, i64, i64, i32, u64, u32, vp, vp, vp, vp, vp]
    L.fp4_quantize_nv_noalloc.argtypes = [vp, i64, i64, i64, i32, i32, u64, u32, i32, vp, vp, vp, i32, vp]
    L.fp4_hadamard32_quantize_nv.argtypes = [vp, i64, i64, i64, i32, u32, i32, u64, u32, i32, vp, vp, vp, vp,
                                             ctypes.c_size_t, i32, vp]
    L.fp4_dropout.argtypes = [vp, i64, i64, i64, i32, vp, i64, f32, u64, u32, vp, i64, vp]
    L.fp4_norm.argtypes = [vp, i64, i64, i64, i32, vp, i64, f32, u64, u32, vp, i64, i32, vp, vp, i32, f32, vp, i64, vp,
                           vp, vp, vp, i32, vp]
    L.fp4q_norm_grad_workspace_bytes.argtypes = [i64, i64]
    L.fp4q_norm_grad_workspace_bytes.restype = ctypes.c_size_t
    L.fp4_norm_grad.argtypes = [vp, i64, i64, i64, i32, vp, i64, vp, i64, i32, vp, i32, vp, vp, f32, u64, u32, vp, i64,
                                vp, i64, vp, vp, vp, ctypes.c_size_t, vp]
    L.fp4_swiglu_grad_bf16.argtypes = [vp, i64, vp, i64, i64, i64, i64, vp, i64, vp, i64, vp]
    L.fp4_rotary.argtypes = [vp, i64, i64, i64, i64, i64, i32, vp, i32, vp, i64, i32, i32, f32, vp, i64, i64, vp]
    for fn in ("fp4_dropout", "fp4_norm", "fp4_norm_grad", "fp4_swiglu_grad_bf16", "fp4_rotary"):
        getattr(L, fn).restype = i32
    for fn in ("fp4_quantize_mx", "fp4_hadamard32_quantize", "fp4_quantize_mx_dual", "fp4_quantize_nv",
               "fp4_quantize_nv_noalloc",
               "fp4_quantize_nv_amax", "fp4_hadamard32_quantize_nv", "fp4_gemm_mx", "fp4_gemm_nv",
               "fp4_gemm_mx_amax", "fp4_gemm_nv_amax", "fp4_gemm_mx_quant"):
        getattr(L, fn).restype = i32
    L.fp4q_status_str.argtypes = [i32]
    L.fp4q_status_str.restype = ctypes.c_char_p
    L.fp4q_abi_version.argtypes = []
    L.fp4q_abi_version.restype = i32
    _lib = L
    return L


def status_str(status: int) -> str:
    return lib().fp4q_status_str(status).decode()


def abi_version() -> int:
    return lib().fp4q_abi_version()


def _check(fn: str, status: int):
    if status != OK:
        raise Fp4qError(fn, status)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _check_out(t: torch.Tensor, name: str, dtype, shape, device) -> torch.Tensor:
    """A caller-supplied output: the library cannot see buffer sizes, so a
    wrong one would be written past its end.  It must be a contiguous tensor
    of `dtype` on the input's device with exactly `shape`."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor")
    if t.device != torch.device(device):
        raise ValueError(f"{name} is on {t.device}, the input on {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _amax_ptr(t: torch.Tensor, device) -> int:
    if t.dtype != torch.float32 or t.numel() < 1 or t.device != torch.device(device):
        raise ValueError("c_amax must be a float32 tensor with at least one element on the operands' device")
    return t.data_ptr()


def _stream(stream) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _empty(shape, dtype, device, stream, *, returned: bool = True) -> torch.Tensor:
    """Memory made for a call on `stream` is that stream's: from the caller's
    current stream it could hold what kernels queued there still use, and be
    given out there while the call's kernels still write. What the call
    returns is recorded on the caller's stream too, where it is read next."""
    if stream is None or torch.device(device).type != "cuda":
        return torch.empty(shape, dtype=dtype, device=device)
    if not hasattr(stream, "stream_id"):  # a handle of another library's
        stream = torch.cuda.ExternalStream(stream.cuda_stream)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if returned:
        t.record_stream(torch.cuda.current_stream())
    return t


def _input(x: torch.Tensor, cols: Optional[int]):
    if x.dtype != torch.bfloat16 or x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be a 2-D bf16 tensor with unit column stride")
    rows = x.shape[0]
    cols = x.shape[1] if cols is None else cols
    ld = x.stride(0) if rows > 1 else x.shape[1]
    return rows, cols, ld


def _logical(rows: int, cols: int, axis: int):
    return (rows, cols) if axis == ALONG_ROWS else (cols, rows)


def mx_output_shapes(R: int, K: int, layout: int):
    """(codes shape, scales shape) of an MX operand [R x K] in `layout`."""
    if layout == LAYOUT_TILED:
        Rp = (R + 31) // 32 * 32
        return (Rp, K // 2), (K // 128, Rp, 4)
    return (R, K // 2), (R, K // 32)


def _mx_outputs(R, K, layout, codes, scales, device, stream):
    cshape, sshape = mx_output_shapes(R, K, layout)
    if codes is None:
        codes = _empty(cshape, torch.uint8, device, stream)
    if scales is None:
        scales = _empty(sshape, torch.uint8, device, stream)
    return (_check_out(codes, "codes", torch.uint8, cshape, device),
            _check_out(scales, "scales", torch.uint8, sshape, device))


def fp4_quantize_mx(x: torch.Tensor, *, cols: Optional[int] = None, axis: int = ALONG_ROWS, round: int = RNE,
                    seed: int = 0, stream_id: int = 0, layout: int = LAYOUT_LINEAR,
                    codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                    stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    rows, cols, ld = _input(x, cols)
    R, K = _logical(rows, cols, axis)
    codes, scales = _mx_outputs(R, K, layout, codes, scales, x.device, stream)
    _check("fp4_quantize_mx", lib().fp4_quantize_mx(x.data_ptr(), rows, cols, ld, axis, round, seed, stream_id,
                                                    codes.data_ptr(), scales.data_ptr(), layout, _stream(stream)))
    return codes, scales


def fp4_quantize_mx_dual(x: torch.Tensor, *, round_rows: int = RNE, stream_id_rows: int = 0,
                         hadamard_cols: bool = True, sign_mask: int = 0, round_cols: int = RNE,
                         stream_id_cols: int = 0, seed: int = 0, layout: int = LAYOUT_LINEAR,
                         codes_rows: Optional[torch.Tensor] = None, scales_rows: Optional[torch.Tensor] = None,
                         codes_cols: Optional[torch.Tensor] = None, scales_cols: Optional[torch.Tensor] = None,
                         stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """x along rows and x^T along columns (optionally Hadamard) from one read
    of x: (codes_rows, scales_rows, codes_cols, scales_cols)."""
    rows, cols, ld = _input(x, None)
    codes_rows, scales_rows = _mx_outputs(rows, cols, layout, codes_rows, scales_rows, x.device, stream)
    codes_cols, scales_cols = _mx_outputs(cols, rows, layout, codes_cols, scales_cols, x.device, stream)
    _check("fp4_quantize_mx_dual",
           lib().fp4_quantize_mx_dual(x.data_ptr(), rows, cols, ld, round_rows, stream_id_rows, codes_rows.data_ptr(),
                                      scales_rows.data_ptr(), int(bool(hadamard_cols)), sign_mask & 0xFFFFFFFF,
                                      round_cols, stream_id_cols, codes_cols.data_ptr(), scales_cols.data_ptr(),
                                      seed, layout, _stream(stream)))
    return codes_rows, scales_rows, codes_cols, scales_cols


def fp4_hadamard32_quantize(x: torch.Tensor, sign_mask: int, *, cols: Optional[int] = None, axis: int = ALONG_COLS,
                            round: int = RNE, seed: int = 0, stream_id: int = 0, layout: int = LAYOUT_LINEAR,
                            codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                            stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    rows, cols, ld = _input(x, cols)
    R, K = _logical(rows, cols, axis)
    codes, scales = _mx_outputs(R, K, layout, codes, scales, x.device, stream)
    _check("fp4_hadamard32_quantize",
           lib().fp4_hadamard32_quantize(x.data_ptr(), rows, cols, ld, axis, sign_mask & 0xFFFFFFFF, round, seed,
                                         stream_id, codes.data_ptr(), scales.data_ptr(), layout, _stream(stream)))
    return codes, scales


def fp4q_nv_workspace_bytes(rows: int, cols: int, axis: int, domain: int) -> int:
    return lib().fp4q_nv_workspace_bytes(rows, cols, axis, domain)


def nv_tensor_scale_shape(R: int, K: int, domain: int):
    return (1,) if domain == NV_GLOBAL else ((R + 127) // 128, (K + 127) // 128)


def nv_output_shapes(R: int, K: int, layout: int = LAYOUT_LINEAR):
    """(codes shape, scales shape) of an NV operand [R x K] in `layout`: the
    tiled layout stores Rp = 32 ceil(R/32) rows (same bytes per row)."""
    Rs = (R + 31) // 32 * 32 if layout == LAYOUT_TILED else R
    return (Rs, K // 2), (Rs, K // 16)


def fp4_quantize_nv(x: torch.Tensor, domain: int = NV_GLOBAL, *, cols: Optional[int] = None, axis: int = ALONG_ROWS,
                    round: int = RNE, seed: int = 0, stream_id: int = 0, codes: Optional[torch.Tensor] = None,
                    scales: Optional[torch.Tensor] = None, tensor_scale: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, amax: Optional[torch.Tensor] = None,
                    hadamard_mask: Optional[int] = None, layout: int = LAYOUT_LINEAR, stream=None):
    """NVFP4; with `amax` (a device float32 tensor holding max |x|, global
    domain only) the producer runs in one pass (fp4_quantize_nv_amax); with
    `hadamard_mask` the fixed-sign Hadamard-32 runs first
    (fp4_hadamard32_quantize_nv, along columns)."""
    rows, cols, ld = _input(x, cols)
    R, K = _logical(rows, cols, axis)
    cshape, sshape = nv_output_shapes(R, K, layout)
    if codes is None:
        codes = _empty(cshape, torch.uint8, x.device, stream)
    if scales is None:
        scales = _empty(sshape, torch.uint8, x.device, stream)
    if tensor_scale is None:
        tensor_scale = _empty(nv_tensor_scale_shape(R, K, domain), torch.float32, x.device, stream)
    _check_out(codes, "codes", torch.uint8, cshape, x.device)
    _check_out(scales, "scales", torch.uint8, sshape, x.device)
    _check_out(tensor_scale, "tensor_scale", torch.float32, nv_tensor_scale_shape(R, K, domain), x.device)
    if amax is not None:
        if (domain != NV_GLOBAL or axis != ALONG_ROWS or amax.dtype != torch.float32 or amax.device != x.device
                or layout != LAYOUT_LINEAR):
            raise ValueError("a given amax is a float32 tensor on x's device, for the global domain along rows, "
                             "linear layout")
        _check("fp4_quantize_nv_amax",
               lib().fp4_quantize_nv_amax(x.data_ptr(), rows, cols, ld, round, seed, stream_id, amax.data_ptr(),
                                          codes.data_ptr(), scales.data_ptr(), tensor_scale.data_ptr(),
                                          _stream(stream)))
        return codes, scales, tensor_scale
    need = fp4q_nv_workspace_bytes(rows, cols, axis, domain)
    if workspace is None and need > 0:
        workspace = _empty((need,), torch.uint8, x.device, stream, returned=False)
    if workspace is not None and (workspace.device != x.device or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous tensor on x's device")
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if hadamard_mask is not None:
        _check("fp4_hadamard32_quantize_nv",
               lib().fp4_hadamard32_quantize_nv(x.data_ptr(), rows, cols, ld, axis, hadamard_mask & 0xFFFFFFFF, round,
                                                seed, stream_id, domain, codes.data_ptr(), scales.data_ptr(),
                                                tensor_scale.data_ptr(), _ptr(workspace), wbytes, layout,
                                                _stream(stream)))
        return codes, scales, tensor_scale
    _check("fp4_quantize_nv",
           lib().fp4_quantize_nv(x.data_ptr(), rows, cols, ld, axis, round, seed, stream_id, domain,
                                 codes.data_ptr(), scales.data_ptr(), tensor_scale.data_ptr(), _ptr(workspace),
                                 wbytes, layout, _stream(stream)))
    return codes, scales, tensor_scale


def fp4_quantize_nv_noalloc(x: torch.Tensor, domain: int = NV_GLOBAL, *, cols: Optional[int] = None,
                            axis: int = ALONG_ROWS, round: int = RNE, seed: int = 0, stream_id: int = 0,
                            codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                            tensor_scale: Optional[torch.Tensor] = None, layout: int = LAYOUT_LINEAR, stream=None):
    """fp4_quantize_nv with the library's own workspace: the call allocates
    no device memory (pass every output to allocate none here either)."""
    rows, cols, ld = _input(x, cols)
    R, K = _logical(rows, cols, axis)
    cshape, sshape = nv_output_shapes(R, K, layout)
    if codes is None:
        codes = _empty(cshape, torch.uint8, x.device, stream)
    if scales is None:
        scales = _empty(sshape, torch.uint8, x.device, stream)
    if tensor_scale is None:
        tensor_scale = _empty(nv_tensor_scale_shape(R, K, domain), torch.float32, x.device, stream)
    _check_out(codes, "codes", torch.uint8, cshape, x.device)
    _check_out(scales, "scales", torch.uint8, sshape, x.device)
    _check_out(tensor_scale, "tensor_scale", torch.float32, nv_tensor_scale_shape(R, K, domain), x.device)
    _check("fp4_quantize_nv_noalloc",
           lib().fp4_quantize_nv_noalloc(x.data_ptr(), rows, cols, ld, axis, round, seed, stream_id, domain,
                                         codes.data_ptr(), scales.data_ptr(), tensor_scale.data_ptr(), layout,
                                         _stream(stream)))
    return codes, scales, tensor_scale


def _gemm_out(M: int, N: int, out_dtype, device, c: Optional[torch.Tensor], stream):
    if c is None:
        c = _empty((M, N), out_dtype, device, stream)
    if c.dtype not in (torch.float32, torch.bfloat16) or c.dim() != 2 or c.stride(1) != 1:
        raise ValueError("c must be a 2-D fp32 or bf16 tensor with unit column stride")
    if tuple(c.shape) != (M, N) or c.device != torch.device(device):
        raise ValueError(f"c must be a [{M} x {N}] tensor on {device}, not {tuple(c.shape)} on {c.device}")
    if M > 1 and c.stride(0) < N:
        raise ValueError("c's rows overlap (row stride below N)")
    ldc = c.stride(0) if M > 1 else N
    return c, (OUT_F32 if c.dtype == torch.float32 else OUT_BF16), ldc


def fp4_gemm_mx(a_codes: torch.Tensor, a_scales: torch.Tensor, b_codes: torch.Tensor, b_scales: torch.Tensor, *,
                alpha: float = 1.0, out_dtype=torch.float32, c: Optional[torch.Tensor] = None,
                layout: int = LAYOUT_LINEAR, m: Optional[int] = None, n: Optional[int] = None,
                c_amax: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """C = alpha * A B^T.  In the tiled layout the code tensors carry rows
    padded to a multiple of 32, so pass the logical m and n.  With `c_amax`
    (a device float32 tensor) max |C| is folded into it (fp4_gemm_mx_amax)."""
    M = a_codes.shape[0] if m is None else m
    N = b_codes.shape[0] if n is None else n
    K = a_codes.shape[1] * 2
    if b_codes.shape[1] * 2 != K:
        raise ValueError("A and B must have the same K")
    c, ctype, ldc = _gemm_out(M, N, out_dtype, a_codes.device, c, stream)
    if c_amax is not None:
        _check("fp4_gemm_mx_amax",
               lib().fp4_gemm_mx_amax(a_codes.data_ptr(), a_scales.data_ptr(), b_codes.data_ptr(), b_scales.data_ptr(),
                                      M, N, K, float(alpha), layout, c.data_ptr(), ctype, ldc, _amax_ptr(c_amax, a_codes.device),
                                      _stream(stream)))
        return c
    _check("fp4_gemm_mx", lib().fp4_gemm_mx(a_codes.data_ptr(), a_scales.data_ptr(), b_codes.data_ptr(),
                                            b_scales.data_ptr(), M, N, K, float(alpha), layout,
                                            c.data_ptr(), ctype, ldc, _stream(stream)))
    return c


def fp4_gemm_mx_quant(a_codes: torch.Tensor, a_scales: torch.Tensor, b_codes: torch.Tensor, b_scales: torch.Tensor,
                      *, alpha: float = 1.0, layout: int = LAYOUT_LINEAR, m: Optional[int] = None,
                      n: Optional[int] = None, c_layout: int = LAYOUT_LINEAR, codes: Optional[torch.Tensor] = None,
                      scales: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """C = alpha * A B^T written as an MXFP4 operand along rows (RNE of the
    bf16 C) in c_layout: returns (codes, scales)."""
    M = a_codes.shape[0] if m is None else m
    N = b_codes.shape[0] if n is None else n
    K = a_codes.shape[1] * 2
    if b_codes.shape[1] * 2 != K:
        raise ValueError("A and B must have the same K")
    codes, scales = _mx_outputs(M, N, c_layout, codes, scales, a_codes.device, stream)
    _check("fp4_gemm_mx_quant",
           lib().fp4_gemm_mx_quant(a_codes.data_ptr(), a_scales.data_ptr(), b_codes.data_ptr(), b_scales.data_ptr(),
                                   M, N, K, float(alpha), layout, codes.data_ptr(), scales.data_ptr(), c_layout,
                                   _stream(stream)))
    return codes, scales


def fp4_gemm_mx_swiglu_quant(a_codes: torch.Tensor, a_scales: torch.Tensor, b_codes: torch.Tensor,
                             b_scales: torch.Tensor, *, alpha: float = 1.0, layout: int = LAYOUT_LINEAR,
                             m: Optional[int] = None, n: Optional[int] = None, h_layout: int = LAYOUT_LINEAR,
                             codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                             stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """H = SwiGLU(alpha * A B^T) written as an MXFP4 operand along rows in
    h_layout; B's n = 2F rows interleave gate and up rows in groups of 32
    (pair_gate_up).  Returns (codes, scales) of H [m x F]."""
    M = a_codes.shape[0] if m is None else m
    N = b_codes.shape[0] if n is None else n
    K = a_codes.shape[1] * 2
    if b_codes.shape[1] * 2 != K:
        raise ValueError("A and B must have the same K")
    codes, scales = _mx_outputs(M, N // 2, h_layout, codes, scales, a_codes.device, stream)
    _check("fp4_gemm_mx_swiglu_quant",
           lib().fp4_gemm_mx_swiglu_quant(a_codes.data_ptr(), a_scales.data_ptr(), b_codes.data_ptr(),
                                          b_scales.data_ptr(), M, N, K, float(alpha), layout, codes.data_ptr(),
                                          scales.data_ptr(), h_layout, _stream(stream)))
    return codes, scales


def fp4_swiglu_bf16(c: torch.Tensor, f: int, *, pair: int = 32, h: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """h = bf16(SiLU(gate) * up) from a bf16 C [M x >= 2f] whose columns
    interleave gate and up in groups of `pair` columns."""
    if c.dtype != torch.bfloat16 or c.dim() != 2 or c.stride(1) != 1:
        raise ValueError("c must be a 2-D bf16 tensor with contiguous rows")
    M = c.shape[0]
    if h is None:
        h = _empty((M, f), torch.bfloat16, c.device, stream)
    if (h.dtype != torch.bfloat16 or h.dim() != 2 or h.stride(1) != 1 or tuple(h.shape) != (M, f)
            or h.device != c.device or (M > 1 and h.stride(0) < f)):
        raise ValueError(f"h must be a [{M} x {f}] bf16 tensor on {c.device} with unit column stride")
    _check("fp4_swiglu_bf16", lib().fp4_swiglu_bf16(c.data_ptr(), M, f, c.stride(0), pair, h.data_ptr(),
                                                    h.stride(0), _stream(stream)))
    return h


def pair_gate_up(w_gate: torch.Tensor, w_up: torch.Tensor, pair: int = 32) -> torch.Tensor:
    """The gate/up weight in the row order fp4_gemm_mx_swiglu_quant takes:
    rows 2 pair b .. + pair-1 = gate rows pair b .., the next pair rows the
    up rows of the same units (a one-time layout of the weight, like the
    tiled operand layout)."""
    F, K = w_gate.shape
    if w_up.shape != (F, K) or F % pair != 0:
        raise ValueError("gate and up must have the same [F x K] shape, F a multiple of pair")
    return torch.stack([w_gate.reshape(F // pair, pair, K), w_up.reshape(F // pair, pair, K)], dim=1).reshape(2 * F, K)


def fp4_gemm_nv(a_codes: torch.Tensor, a_scales: torch.Tensor, a_tensor_scale: torch.Tensor, b_codes: torch.Tensor,
                b_scales: torch.Tensor, b_tensor_scale: torch.Tensor, domain: int = NV_GLOBAL, *, alpha: float = 1.0,
                out_dtype=torch.float32, c: Optional[torch.Tensor] = None, c_amax: Optional[torch.Tensor] = None,
                layout: int = LAYOUT_LINEAR, m: Optional[int] = None, n: Optional[int] = None,
                stream=None) -> torch.Tensor:
    """With `c_amax` (a device float32 tensor) max |C| is folded into it
    (fp4_gemm_nv_amax).  In the tiled layout the code tensors carry rows
    padded to a multiple of 32, so pass the logical m and n."""
    M = a_codes.shape[0] if m is None else m
    N = b_codes.shape[0] if n is None else n
    K = a_codes.shape[1] * 2
    if b_codes.shape[1] * 2 != K:
        raise ValueError("A and B must have the same K")
    c, ctype, ldc = _gemm_out(M, N, out_dtype, a_codes.device, c, stream)
    if c_amax is not None:
        _check("fp4_gemm_nv_amax",
               lib().fp4_gemm_nv_amax(a_codes.data_ptr(), a_scales.data_ptr(), a_tensor_scale.data_ptr(),
                                      b_codes.data_ptr(), b_scales.data_ptr(), b_tensor_scale.data_ptr(), domain, M, N,
                                      K, float(alpha), layout, c.data_ptr(), ctype, ldc, _amax_ptr(c_amax, a_codes.device),
                                      _stream(stream)))
        return c
    _check("fp4_gemm_nv", lib().fp4_gemm_nv(a_codes.data_ptr(), a_scales.data_ptr(), a_tensor_scale.data_ptr(),
                                            b_codes.data_ptr(), b_scales.data_ptr(), b_tensor_scale.data_ptr(),
                                            domain, M, N, K, float(alpha), layout, c.data_ptr(), ctype, ldc,
                                            _stream(stream)))
    return c


# ---- the row-wise operators between the GEMMs
#
# A decoding step makes these calls on a few kilobytes each, where reading
# tensors' attributes from Python would cost more than the launch: their
# arguments are checked and marshalled in csrc/row_calls.cpp.

_row_calls = None
_row_lib = None  # the library whose addresses _row_calls holds
_new = tuple.__new__  # of a NamedTuple, at a third of its own constructor's time


def _rows():
    global _row_calls, _row_lib
    if _lib is None or _row_lib is not _lib:
        L = lib()
        try:
            from fp4_block_scaled_quantizer_amd import _row_calls as calls
        except ImportError as e:
            raise FileNotFoundError(
                f"{ROW_CALLS_PATH} cannot be loaded ({e}): build it with "
                "`python -c 'import __graft_entry__ as g; g.build()'`") from e
        at = [ctypes.cast(getattr(L, f), ctypes.c_void_p).value for f in
              ("fp4_dropout", "fp4_norm", "fp4q_norm_grad_workspace_bytes", "fp4_norm_grad", "fp4_swiglu_grad_bf16",
               "fp4_rotary")]
        calls.bind(*at, Fp4qError, torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream, torch.cuda.ExternalStream)
        _row_calls, _row_lib = calls, L
    return _row_calls


def fp4_dropout(x: torch.Tensor, p: float, *, seed: int, stream_id: int = 0, residual: Optional[torch.Tensor] = None,
                y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """[residual +] dropout(x): each element is kept with probability 1 - p
    (from 16 random bits of (seed, stream_id, row, column)) and scaled. The
    gradient is the same call on the gradient. seed is a number of the host's:
    a captured graph draws the same mask at every replay. y may be x or
    residual."""
    return _rows().dropout(x, p, seed, stream_id, residual, y, stream)


class Norm(NamedTuple):
    """fp4_norm's outputs; those not asked for are None."""
    y: Optional[torch.Tensor]
    h: Optional[torch.Tensor]
    mean: Optional[torch.Tensor]
    rstd: Optional[torch.Tensor]
    codes: Optional[torch.Tensor]
    scales: Optional[torch.Tensor]


def fp4_norm(x: torch.Tensor, gamma: Optional[torch.Tensor] = None, beta: Optional[torch.Tensor] = None, *,
             kind: int = NORM_LAYER, eps: float = 1e-5, residual: Optional[torch.Tensor] = None, p: float = 0.0,
             seed: int = 0, stream_id: int = 0, save: bool = False, want_y: bool = True, mx: bool = False,
             layout: int = LAYOUT_LINEAR, y: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None,
             mean: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None,
             codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None, stream=None) -> Norm:
    """h = [residual +] dropout(x); y = norm(h) * gamma + beta, with kind
    NORM_LAYER or NORM_RMS. h comes out where there is a residual or dropout
    (else it is x); `save` asks for the row statistics that fp4_norm_grad
    takes; `mx` for the MXFP4 operand of a bf16 y in `layout` (with want_y
    False, instead of y). h and y may each be x or residual."""
    if mx or codes is not None or scales is not None:
        if not isinstance(x, torch.Tensor):
            raise ValueError("x must be a tensor")
        if x.dim() != 2:
            raise ValueError("x must be a 2-D fp32 or bf16 tensor")
        codes, scales = _mx_outputs(x.shape[0], x.shape[1], layout, codes, scales, x.device, stream)
    y, h, mean, rstd = _rows().norm(x, gamma, beta, kind, eps, residual, p, seed, stream_id, save, want_y, layout, y, h,
                                    mean, rstd, codes, scales, stream)
    return _new(Norm, (y, h, mean, rstd, codes, scales))


class NormGrad(NamedTuple):
    """fp4_norm_grad's outputs; those not asked for are None."""
    dh: torch.Tensor
    dx: Optional[torch.Tensor]
    dgamma: Optional[torch.Tensor]
    dbeta: Optional[torch.Tensor]


def fp4_norm_grad(dy: torch.Tensor, h: torch.Tensor, gamma: Optional[torch.Tensor] = None, *, rstd: torch.Tensor,
                  mean: Optional[torch.Tensor] = None, kind: int = NORM_LAYER, dres: Optional[torch.Tensor] = None,
                  p: float = 0.0, seed: int = 0, stream_id: int = 0, weights: bool = True,
                  dh: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                  dgamma: Optional[torch.Tensor] = None, dbeta: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, stream=None) -> NormGrad:
    """The gradient of fp4_norm: dh of the normed rows (plus `dres`, what
    reaches them along the residual stream), dx of fp4_norm's x where p > 0
    (dx equals dh otherwise and is None), and with `weights` dgamma and, for
    NORM_LAYER, dbeta in fp32. dh and dx may each be dy, h or dres."""
    return _new(NormGrad, _rows().norm_grad(dy, h, gamma, kind, mean, rstd, dres, p, seed, stream_id, weights, dh, dx,
                                            dgamma, dbeta, workspace, stream))


def fp4_swiglu_grad_bf16(dh: torch.Tensor, c: torch.Tensor, *, pair: int = 32, want_h: bool = False,
                         dc: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None,
                         stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """The gradient of fp4_swiglu_bf16: (dc, h) from dh [M x F] and the bf16
    C [M x >= 2F] whose columns interleave gate and up in groups of `pair`;
    h (with `want_h`) is the forward's output again. dc may be c, h may be dh."""
    return _rows().swiglu_grad(dh, c, pair, want_h, dc, h, stream)


def fp4_rotary(x: torch.Tensor, positions: torch.Tensor, inv_freq: torch.Tensor, *, style: int = ROTARY_HALF,
               scale: float = 1.0, inverse: bool = False, y: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """Rotary positions of x [tokens, heads, dim] (tokens of whole heads, so a
    slice of a fused QKV output serves, or heads of whole tokens, such as
    `t.transpose(0, 1)` of an attention's [heads, tokens, dim]): pair i of each head
    turns by positions[t] * inv_freq[i], the first 2 len(inv_freq) elements
    of the head taking part. `inverse` turns back: the gradient. y may be x."""
    return _rows().rotary(x, positions, inv_freq, style, scale, inverse, y, stream)


def rotary_frequencies(rot: int, base: float = 10000.0, *, factor: float = 1.0, method: str = "none",
                       original_length: int = 8192, slow_turns: float = 1.0, fast_turns: float = 32.0,
                       device=None) -> Tuple[torch.Tensor, float]:
    """(inv_freq, scale) for fp4_rotary: rot / 2 frequencies base^(-2i/rot),
    stretched for a context `factor` times the trained `original_length`:
      "linear"  every frequency divided by factor (positions interpolated);
      "base"    the base raised to base * factor^(rot / (rot - 2)), so that the
                lowest frequency is divided by factor and the highest kept;
      "turns"   by the turns a pair makes over the trained length: below
                slow_turns divided by factor, above fast_turns kept, linear in
                the turns between; scale = 1 + 0.1 ln factor.
    A layout of constants made once, like pair_gate_up."""
    if (rot < 2 or rot % 2 or not factor >= 1 or not fast_turns > slow_turns
            or method not in ("none", "linear", "base", "turns")):
        raise ValueError("rot must be even and >= 2, factor >= 1, fast_turns > slow_turns, "
                         "method none, linear, base or turns")
    if method == "base" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    freq = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    scale = 1.0
    if method == "linear":
        freq = freq / factor
    elif method == "turns":
        turns = freq * original_length / (2 * math.pi)
        keep = ((turns - slow_turns) / (fast_turns - slow_turns)).clamp(0, 1)
        freq = freq * (keep + (1 - keep) / factor)
        scale = 1 + 0.1 * math.log(factor)
    return freq.to(torch.float32).to("cpu" if device is None else device), scale
