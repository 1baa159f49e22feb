"""ctypes binding of libjscan (argument marshalling only)."""
from __future__ import annotations

import ctypes
import os
import types

import torch
from torch.autograd import forward_ad

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libjscan.so")

D_STATE = 16
JSCAN_F32, JSCAN_BF16 = 0, 1
_DTYPES = {torch.float32: JSCAN_F32, torch.bfloat16: JSCAN_BF16}
_lib = None


class JScanError(RuntimeError):
    """A libjscan call returned an error status."""

    def __init__(self, status: int, msg: str, hip_error: int = 0):
        super().__init__(f"libjscan: {msg} (status {status}" + (f", hipError {hip_error})" if hip_error else ")"))
        self.status = status
        self.hip_error = hip_error


def library_path() -> str:
    return _LIB_PATH


def library():
    """Load libjscan.so (building it first if it is missing) and declare its signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        from . import build

        build.build()
    lib = ctypes.CDLL(_LIB_PATH)
    vp, fp, i64, i32 = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.jscan_prefill.argtypes = [vp, vp, fp, vp, vp, vp, fp, i64, i64, i64, i64, i32, vp]
    lib.jscan_prefill_resume.argtypes = [vp, vp, fp, vp, vp, fp, vp, fp, i64, i64, i64, i64, i32, vp]
    lib.jscan_step.argtypes = [fp, vp, vp, fp, vp, vp, vp, i64, i64, i64, i64, i64, i64, i32, vp]
    lib.jscan_prefill_chunked.argtypes = [vp, vp, fp, vp, vp, fp, vp, fp, i64, i64, i64, i64, i64, vp, i64, i32, vp]
    lib.jscan_prefill_chunked_workspace.argtypes = [i64, i64, i64, i64, i64]
    lib.jscan_prefill_chunked_noalloc.argtypes = [vp, vp, fp, vp, vp, fp, vp, fp, i64, i64, i64, i64, i64, i32, vp]
    lib.jscan_prefill_chunked_noalloc.restype = i32
    lib.jscan_ssm_inputs.argtypes = [vp, vp, fp, fp, fp, vp, fp, vp, vp, vp, vp, i64, i64, i64, i64, ctypes.c_float, i32,
                                     vp]
    lib.jscan_ssm_inputs.restype = i32
    lib.jscan_prefill_fused.argtypes = [vp, vp, vp, fp, fp, vp, vp, fp, vp, fp, i64, i64, i64, i64, i64, i32, vp]
    lib.jscan_prefill_fused.restype = i32
    lib.jscan_prefill_scalar_a.argtypes = [vp, vp, fp, vp, vp, fp, vp, fp, i64, i64, i64, i64, i32, vp]
    lib.jscan_step_scalar_a.argtypes = [fp, vp, vp, fp, vp, vp, vp, i64, i64, i64, i64, i64, i64, i32, vp]
    lib.jscan_prefill_complex.argtypes = [vp, vp, fp, vp, vp, fp, vp, fp, i64, i64, i64, i64, i32, vp]
    lib.jscan_step_complex.argtypes = [fp, vp, vp, fp, vp, vp, vp, i64, i64, i64, i64, i64, i64, i32, vp]
    lib.jscan_prefill_trapezoid.argtypes = [vp, vp, vp, fp, vp, vp, fp, vp, vp, vp, fp, i64, i64, i64, i64, i32, i32, vp]
    lib.jscan_step_trapezoid.argtypes = [fp, vp, vp, vp, vp, vp, fp, vp, vp, vp, i64, i64, i64, i64, i64, i64, i32, i32,
                                         vp]
    lib.jscan_prefill_mimo.argtypes = [vp, vp, fp, vp, vp, fp, vp, fp, i64, i64, i64, i64, i64, i32, i32, vp]
    lib.jscan_step_mimo.argtypes = [fp, vp, vp, fp, vp, vp, vp, i64, i64, i64, i64, i64, i64, i64, i64, i32, i32, vp]
    lib.jscan_prefill_mimo_trapezoid.argtypes = [vp, vp, vp, fp, vp, vp, fp, vp, vp, vp, fp, i64, i64, i64, i64, i64,
                                                 i32, i32, vp]
    lib.jscan_step_mimo_trapezoid.argtypes = [fp, vp, vp, vp, vp, vp, fp, vp, vp, vp, i64, i64, i64, i64, i64, i64, i64,
                                              i64, i32, i32, vp]
    lib.jscan_gated_scan.argtypes = [vp, vp, fp, vp, vp, fp, i64, i64, i64, i64, i64, i64, vp, i64, i32, i32, vp]
    lib.jscan_gated_scan_backward.argtypes = [vp, vp, vp, vp, fp, fp, vp, vp, vp, fp, i64, i64, i64, i64, i64, i64, i64,
                                              i64, i64, vp, i64, i32, i32, vp]
    lib.jscan_gated_scan_save.argtypes = [vp, vp, fp, vp, vp, fp, fp, i64, i64, i64, i64, i64, i64, vp, i64, i32, i32, vp]
    lib.jscan_gated_scan_backward_saved.argtypes = [vp, vp, fp, vp, fp, vp, vp, vp, fp, i64, i64, i64, i64, i64, i64, i64,
                                                    i64, vp, i64, i32, i32, vp]
    lib.jscan_gated_scan_states.argtypes = [i64, i64, i64]
    lib.jscan_gated_scan_states.restype = i64
    lib.jscan_gated_step.argtypes = [fp, vp, vp, vp, i64, i64, i64, i64, i64, i32, i32, vp]
    lib.jscan_gated_scan_workspace.argtypes = [i64, i64, i64]
    lib.jscan_gated_scan_workspace.restype = i64
    lib.jscan_quantize_rows.argtypes = [vp, vp, fp, i64, i64, i64, i32, vp]
    lib.jscan_matmul_i8.argtypes = [vp, fp, vp, fp, fp, vp, i64, i64, i64, i64, i32, vp]
    lib.jscan_causal_conv.argtypes = [vp, vp, fp, fp, vp, vp, vp, i64, i64, i64, i64, i64, i64, i32, i32, vp]
    lib.jscan_causal_conv_backward.argtypes = [vp, vp, fp, fp, vp, vp, vp, vp, vp, fp, fp, i64, i64, i64, i64, i64, i64,
                                               i64, vp, i64, i32, i32, vp]
    lib.jscan_causal_conv_step.argtypes = [vp, vp, fp, fp, vp, i64, i64, i64, i64, i64, i32, i32, vp]
    lib.jscan_causal_conv_backward_workspace.argtypes = [i64, i64, i64, i64]
    lib.jscan_causal_conv_backward_workspace.restype = i64
    f32 = ctypes.c_float
    lib.jscan_matmul_i8_epilogue.argtypes = [vp, fp, vp, fp, fp, vp, vp, i64, i64, i64, i64, i64, i32, i32, vp]
    lib.jscan_rms_norm.argtypes = [vp, vp, fp, vp, vp, i64, i64, i64, i64, i64, i64, f32, i32, vp]
    lib.jscan_rms_norm_quantize.argtypes = [vp, vp, fp, vp, fp, vp, i64, i64, i64, i64, i64, f32, i32, vp]
    lib.jscan_rms_norm_backward.argtypes = [vp, fp, vp, vp, vp, fp, i64, i64, i64, i64, i64, i64, vp, i64, f32, i32, vp]
    lib.jscan_rms_norm_backward_workspace.argtypes = [i64, i64]
    lib.jscan_rms_norm_backward_workspace.restype = i64
    lib.jscan_prefill_gate.argtypes = [vp, vp, fp, vp, vp, fp, fp, vp, vp, fp, i64, i64, i64, i64, i64, i64, vp, i64, i32,
                                       i32, vp]
    lib.jscan_prefill_gate_workspace.argtypes = [i64, i64, i64, i64, i64]
    lib.jscan_prefill_gate_workspace.restype = i64
    lib.jscan_step_gate.argtypes = [fp, vp, vp, fp, vp, vp, fp, vp, vp, i64, i64, i64, i64, i64, i64, i64, i32, i32, vp]
    lib.jscan_prefill_chunked_workspace.restype = i64
    for f in (lib.jscan_prefill, lib.jscan_prefill_resume, lib.jscan_step, lib.jscan_prefill_chunked,
              lib.jscan_prefill_scalar_a, lib.jscan_step_scalar_a, lib.jscan_prefill_complex, lib.jscan_step_complex,
              lib.jscan_prefill_trapezoid, lib.jscan_step_trapezoid, lib.jscan_prefill_mimo, lib.jscan_step_mimo,
              lib.jscan_prefill_mimo_trapezoid, lib.jscan_step_mimo_trapezoid, lib.jscan_gated_scan,
              lib.jscan_gated_scan_backward, lib.jscan_gated_scan_save, lib.jscan_gated_scan_backward_saved,
              lib.jscan_gated_step, lib.jscan_quantize_rows, lib.jscan_matmul_i8, lib.jscan_causal_conv,
              lib.jscan_causal_conv_backward, lib.jscan_causal_conv_step, lib.jscan_prefill_gate, lib.jscan_step_gate,
              lib.jscan_matmul_i8_epilogue, lib.jscan_rms_norm, lib.jscan_rms_norm_quantize, lib.jscan_rms_norm_backward):
        f.restype = i32
    lib.jscan_status_string.argtypes = [i32]
    lib.jscan_status_string.restype = ctypes.c_char_p
    lib.jscan_last_hip_error.restype = i32
    lib.jscan_version.restype = i32
    _lib = lib
    return lib


def _check(status: int):
    if status != 0:
        lib = library()
        raise JScanError(status, lib.jscan_status_string(status).decode(), lib.jscan_last_hip_error())


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(dev: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _require(cond: bool, msg: str):
    if not cond:
        raise ValueError(msg)


def _check_prefill_args(x, delta, A, B, C, h0, scalar_a=False):
    _require(x.is_cuda, "inputs must be CUDA (HIP) tensors")
    _require(x.dtype in _DTYPES, "x must be bfloat16 or float32")
    _require(x.dim() == 3, "x must be [batch, L, D]")
    batch, L, D = x.shape
    a_shape = (D,) if scalar_a else (D, D_STATE)
    for name, t, shape, dt in (("delta", delta, (batch, L, D), x.dtype), ("A", A, a_shape, torch.float32),
                               ("B", B, (batch, L, D_STATE), x.dtype), ("C", C, (batch, L, D_STATE), x.dtype)):
        _require(tuple(t.shape) == shape, f"{name} must have shape {shape}, got {tuple(t.shape)}")
        _require(t.dtype == dt, f"{name} must be {dt}")
        _require(t.device == x.device, f"{name} is on another device")
        _require(t.is_contiguous(), f"{name} must be contiguous")
    _require(x.is_contiguous(), "x must be contiguous")
    if h0 is not None:
        _require(tuple(h0.shape) == (batch, D, D_STATE) and h0.dtype == torch.float32 and h0.is_contiguous()
                 and h0.device == x.device, "h0 must be a contiguous fp32 [batch, D, 16] tensor on x's device")
    return batch, L, D


def prefill(x, delta, A, B, C, h0=None, y=None, h_final=None):
    """Scan ``L`` tokens.  x, delta ``[batch, L, D]``, B, C ``[batch, L, 16]`` (bf16 or fp32, one
    dtype), A ``[D, 16]`` fp32, optional h0 ``[batch, D, 16]`` fp32 to resume from.
    Returns ``(y [batch, L, D] in the input dtype, h_final [batch, D, 16] fp32)``.
    ``h_final`` may be passed as ``h0`` itself to update a state in place."""
    batch, L, D = _check_prefill_args(x, delta, A, B, C, h0)
    if y is None:
        y = torch.empty_like(x)
    if h_final is None:
        h_final = torch.empty((batch, D, D_STATE), dtype=torch.float32, device=x.device)
    lib = library()
    args_tail = (ctypes.c_void_p(y.data_ptr()), ctypes.c_void_p(h_final.data_ptr()), batch, L, D, D_STATE,
                 _DTYPES[x.dtype], _stream(x.device))
    with torch.cuda.device(x.device):
        if h0 is None:
            st = lib.jscan_prefill(_ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), *args_tail)
        else:
            st = lib.jscan_prefill_resume(_ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(h0), *args_tail)
    _check(st)
    return y, h_final


def prefill_scalar_a(x, delta, a, B, C, h0=None, y=None, h_final=None):
    """Prefill with a scaled-identity A (``jscan_prefill_scalar_a``): ``a`` ``[D]`` fp32 stands
    for ``A[d, n] = a[d]``.  Bit-identical to :func:`prefill` on that expanded A, and faster
    (one decay per token and channel).  Other arguments and results as for :func:`prefill`."""
    batch, L, D = _check_prefill_args(x, delta, a, B, C, h0, scalar_a=True)
    if y is None:
        y = torch.empty_like(x)
    if h_final is None:
        h_final = torch.empty((batch, D, D_STATE), dtype=torch.float32, device=x.device)
    lib = library()
    with torch.cuda.device(x.device):
        st = lib.jscan_prefill_scalar_a(_ptr(x), _ptr(delta), _ptr(a), _ptr(B), _ptr(C), _ptr(h0), _ptr(y),
                                        _ptr(h_final), batch, L, D, D_STATE, _DTYPES[x.dtype], _stream(x.device))
    _check(st)
    return y, h_final


def prefill_complex(x, delta, A, B, C, h0=None, y=None, h_final=None):
    """Prefill with the complex-valued state (``jscan_prefill_complex``): states 2k, 2k+1 of a
    channel are one complex state and ``A[d, 2k], A[d, 2k+1]`` the real and imaginary parts of
    its diagonal entry.  Arguments and results as for :func:`prefill`."""
    batch, L, D = _check_prefill_args(x, delta, A, B, C, h0)
    if y is None:
        y = torch.empty_like(x)
    if h_final is None:
        h_final = torch.empty((batch, D, D_STATE), dtype=torch.float32, device=x.device)
    lib = library()
    with torch.cuda.device(x.device):
        st = lib.jscan_prefill_complex(_ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(h0), _ptr(y),
                                       _ptr(h_final), batch, L, D, D_STATE, _DTYPES[x.dtype], _stream(x.device))
    _check(st)
    return y, h_final


def chunked_workspace_bytes(batch: int, L: int, D: int, chunk: int = 0) -> int:
    """Bytes of workspace ``prefill_chunked`` needs (0 when it runs as one segment)."""
    n = library().jscan_prefill_chunked_workspace(batch, L, D, D_STATE, chunk)
    if n < 0:
        raise ValueError(f"invalid shape or chunk: batch={batch} L={L} D={D} chunk={chunk}")
    return n


def prefill_chunked(x, delta, A, B, C, h0=None, y=None, h_final=None, chunk=0, workspace=None):
    """Time-parallel prefill (``jscan_prefill_chunked``): the same result as :func:`prefill` up
    to fp32 rounding of the segment composition, for shapes with too few channels to fill
    the GPU.  ``chunk`` is the segment length in tokens (0 = automatic).  ``workspace`` is a
    CUDA tensor of at least :func:`chunked_workspace_bytes` bytes; one is allocated if None."""
    batch, L, D = _check_prefill_args(x, delta, A, B, C, h0)
    need = chunked_workspace_bytes(batch, L, D, chunk)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if y is None:
        y = torch.empty_like(x)
    if h_final is None:
        h_final = torch.empty((batch, D, D_STATE), dtype=torch.float32, device=x.device)
    lib = library()
    with torch.cuda.device(x.device):
        st = lib.jscan_prefill_chunked(_ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(h0), _ptr(y),
                                       _ptr(h_final), batch, L, D, D_STATE, chunk, _ptr(workspace), ws_bytes,
                                       _DTYPES[x.dtype], _stream(x.device))
    _check(st)
    return y, h_final


NOALLOC_SCRATCH_BYTES = 24 * 1024 * 1024   # JSCAN_NOALLOC_SCRATCH_BYTES


def prefill_chunked_noalloc(x, delta, A, B, C, h0=None, y=None, h_final=None, chunk=0):
    """:func:`prefill_chunked` through ``jscan_prefill_chunked_noalloc``: the library's own
    scratch array instead of a workspace (calls on one GPU must not overlap in time).  Pass
    ``y`` and ``h_final`` to allocate nothing here either."""
    batch, L, D = _check_prefill_args(x, delta, A, B, C, h0)
    if y is None:
        y = torch.empty_like(x)
    if h_final is None:
        h_final = torch.empty((batch, D, D_STATE), dtype=torch.float32, device=x.device)
    lib = library()
    with torch.cuda.device(x.device):
        st = lib.jscan_prefill_chunked_noalloc(_ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(h0), _ptr(y),
                                               _ptr(h_final), batch, L, D, D_STATE, chunk, _DTYPES[x.dtype],
                                               _stream(x.device))
    _check(st)
    return y, h_final


def ssm_inputs(x, w_x, g_delta, g_B, g_C, w_dt, b_dt, eps=1e-6, delta=None, B=None, C=None, delta_low=None,
               skip_delta=False):
    """Producer side (``jscan_ssm_inputs``): delta, B and C of the scan computed from x.
    x ``[..., D]`` bf16; w_x ``[R + 32, D]`` bf16; gains fp32 ``[R]``, ``[16]``, ``[16]``;
    w_dt ``[D, R]`` bf16; b_dt ``[D]`` fp32.  Returns ``(delta [..., D], B [..., 16], C [..., 16],
    delta_low [..., R])``, all bf16, with x's leading shape.  ``skip_delta`` runs only the first
    product (delta is then None): the input of :func:`prefill_fused`."""
    _require(x.is_cuda and x.dtype == torch.bfloat16 and x.is_contiguous(), "x must be a contiguous bf16 CUDA tensor")
    D = x.shape[-1]
    lead = tuple(x.shape[:-1])
    M = x.numel() // D if D else 0
    R = w_dt.shape[1] if w_dt.dim() == 2 else -1
    for name, t, shape, dt in (("w_x", w_x, (R + 2 * D_STATE, D), torch.bfloat16),
                               ("g_delta", g_delta, (R,), torch.float32), ("g_B", g_B, (D_STATE,), torch.float32),
                               ("g_C", g_C, (D_STATE,), torch.float32), ("w_dt", w_dt, (D, R), torch.bfloat16),
                               ("b_dt", b_dt, (D,), torch.float32)):
        _require(tuple(t.shape) == shape, f"{name} must have shape {shape}, got {tuple(t.shape)}")
        _require(t.dtype == dt and t.is_contiguous() and t.device == x.device, f"{name} must be contiguous {dt} on x's device")
    dev = x.device
    if skip_delta:
        delta = None
    elif delta is None:
        delta = torch.empty(lead + (D,), dtype=torch.bfloat16, device=dev)
    B = torch.empty(lead + (D_STATE,), dtype=torch.bfloat16, device=dev) if B is None else B
    C = torch.empty(lead + (D_STATE,), dtype=torch.bfloat16, device=dev) if C is None else C
    delta_low = torch.empty(lead + (R,), dtype=torch.bfloat16, device=dev) if delta_low is None else delta_low
    lib = library()
    with torch.cuda.device(dev):
        st = lib.jscan_ssm_inputs(_ptr(x), _ptr(w_x), _ptr(g_delta), _ptr(g_B), _ptr(g_C), _ptr(w_dt), _ptr(b_dt),
                                  _ptr(delta_low), _ptr(delta), _ptr(B), _ptr(C), M, D, R, D_STATE, float(eps),
                                  JSCAN_BF16, _stream(dev))
    _check(st)
    return delta, B, C, delta_low


def prefill_fused(x, delta_low, w_dt, b_dt, A, B, C, h0=None, y=None, h_final=None):
    """Prefill with delta computed inside the scan from delta_low (``jscan_prefill_fused``):
    bit-identical to ``ssm_inputs`` then ``prefill``.  bf16, rank 256, long-sequence shapes."""
    _require(x.is_cuda and x.dtype == torch.bfloat16 and x.dim() == 3 and x.is_contiguous(),
             "x must be a contiguous bf16 [batch, L, D] CUDA tensor")
    batch, L, D = x.shape
    R = delta_low.shape[-1]
    for name, t, shape, dt in (("delta_low", delta_low, (batch, L, R), torch.bfloat16),
                               ("w_dt", w_dt, (D, R), torch.bfloat16), ("b_dt", b_dt, (D,), torch.float32),
                               ("A", A, (D, D_STATE), torch.float32), ("B", B, (batch, L, D_STATE), torch.bfloat16),
                               ("C", C, (batch, L, D_STATE), torch.bfloat16)):
        _require(tuple(t.shape) == shape, f"{name} must have shape {shape}, got {tuple(t.shape)}")
        _require(t.dtype == dt and t.is_contiguous() and t.device == x.device, f"{name} must be contiguous {dt}")
    if h0 is not None:
        _require(tuple(h0.shape) == (batch, D, D_STATE) and h0.dtype == torch.float32 and h0.is_contiguous(),
                 "h0 must be a contiguous fp32 [batch, D, 16] tensor")
    y = torch.empty_like(x) if y is None else y
    h_final = torch.empty((batch, D, D_STATE), dtype=torch.float32, device=x.device) if h_final is None else h_final
    lib = library()
    with torch.cuda.device(x.device):
        st = lib.jscan_prefill_fused(_ptr(x), _ptr(delta_low), _ptr(w_dt), _ptr(b_dt), _ptr(A), _ptr(B), _ptr(C),
                                     _ptr(h0), _ptr(y), _ptr(h_final), batch, L, D, D_STATE, R, JSCAN_BF16,
                                     _stream(x.device))
    _check(st)
    return y, h_final


def _step_output(y_t, shape, dtype, device):
    """The output of a decode step and its row stride in elements: a new contiguous tensor, or
    the caller's ``y_t`` of that shape and dtype whose rows are contiguous (the row stride of a
    strided view, e.g. ``y[:, t]``, is passed to the library, which checks it)."""
    if y_t is None:
        y_t = torch.empty(shape, dtype=dtype, device=device)
    _require(tuple(y_t.shape) == tuple(shape) and y_t.dtype == dtype and y_t.device == device,
             f"y_t must be {tuple(shape)} of dtype {dtype} on {device}")
    row = 1
    for k in range(len(shape) - 1, 0, -1):
        _require(y_t.stride(k) == row, "y_t rows must be contiguous")
        row *= shape[k]
    return y_t, (y_t.stride(0) if shape[0] > 1 else row)


def step_raw(h, x_t, delta_t, A, B_t, C_t, y_t, batch, D, ld_xd, ld_bc, dtype, scalar_a=False, complex_a=False,
             ld_y=None):
    """Direct call of ``jscan_step`` (``jscan_step_scalar_a`` with ``scalar_a``,
    ``jscan_step_complex`` with ``complex_a``) on raw tensors/pointers with explicit row strides
    (no checks beyond the library's own; ``ld_y`` defaults to ``ld_xd``).  ``x_t`` etc. may be
    tensors or integer device addresses."""
    lib = library()

    def p(v):
        return ctypes.c_void_p(v if isinstance(v, int) else v.data_ptr())

    dev = h.device if hasattr(h, "device") else torch.device("cuda")
    fn = lib.jscan_step_scalar_a if scalar_a else lib.jscan_step_complex if complex_a else lib.jscan_step
    st = fn(p(h), p(x_t), p(delta_t), p(A), p(B_t), p(C_t), p(y_t), batch, D, D_STATE, ld_xd, ld_bc,
            ld_xd if ld_y is None else ld_y, _DTYPES[dtype], _stream(dev))
    _check(st)


def step_scalar_a(h, x_t, delta_t, a, B_t, C_t, y_t=None):
    """:func:`step` with a scaled-identity A, ``a`` ``[D]`` fp32 (``jscan_step_scalar_a``)."""
    return step(h, x_t, delta_t, a, B_t, C_t, y_t, _scalar_a=True)


def step_complex(h, x_t, delta_t, A, B_t, C_t, y_t=None):
    """:func:`step` with the complex-valued state (``jscan_step_complex``)."""
    return step(h, x_t, delta_t, A, B_t, C_t, y_t, _complex_a=True)


def step(h, x_t, delta_t, A, B_t, C_t, y_t=None, _scalar_a=False, _complex_a=False):
    """One decode token for a batch: h ``[batch, D, 16]`` fp32 is updated in place; x_t, delta_t
    ``[batch, D]`` and B_t, C_t ``[batch, 16]`` (rows may be strided views of prefill tensors,
    e.g. ``x[:, t]``).  Returns y_t ``[batch, D]``: a new contiguous tensor, or the given ``y_t``,
    whose rows may be strided too (for example ``y[:, t]`` of a ``[batch, L, D]`` output)."""
    _require(h.is_cuda and h.dtype == torch.float32 and h.dim() == 3 and h.shape[2] == D_STATE and h.is_contiguous(),
             "h must be a contiguous fp32 [batch, D, 16] CUDA tensor")
    batch, D, _ = h.shape
    _require(x_t.dtype in _DTYPES, "x_t must be bfloat16 or float32")
    for name, t, shape in (("x_t", x_t, (batch, D)), ("delta_t", delta_t, (batch, D)),
                           ("B_t", B_t, (batch, D_STATE)), ("C_t", C_t, (batch, D_STATE))):
        _require(tuple(t.shape) == shape, f"{name} must have shape {shape}")
        _require(t.dtype == x_t.dtype, f"{name} must be {x_t.dtype}")
        _require(t.stride(1) == 1, f"{name} rows must be contiguous")
        _require(t.device == h.device, f"{name} is on another device")
    a_shape = (D,) if _scalar_a else (D, D_STATE)
    _require(A.dtype == torch.float32 and tuple(A.shape) == a_shape and A.is_contiguous(),
             f"A must be a contiguous fp32 tensor of shape {a_shape}")
    ld_xd = x_t.stride(0) if batch > 1 else D
    _require(batch <= 1 or delta_t.stride(0) == ld_xd, "x_t and delta_t must share a row stride")
    ld_bc = B_t.stride(0) if batch > 1 else D_STATE
    _require(batch <= 1 or C_t.stride(0) == ld_bc, "B_t and C_t must share a row stride")
    y_t, ld_y = _step_output(y_t, (batch, D), x_t.dtype, h.device)
    with torch.cuda.device(h.device):
        step_raw(h, x_t, delta_t, A, B_t, C_t, y_t, batch, D, ld_xd, ld_bc, x_t.dtype, scalar_a=_scalar_a,
                 complex_a=_complex_a, ld_y=ld_y)
    return y_t


# ---- exponential-trapezoidal rule ----------------------------------------------------------
# jscan_a_form values: the form of A that the trapezoidal entry points take.
A_FORMS = {"diagonal": 0, "scalar": 1, "complex": 2}


def prefill_trapezoid(x, delta, lam, A, B, C, h0=None, x_prev=None, B_prev=None, form="diagonal", y=None,
                      h_final=None):
    """Prefill with the exponential-trapezoidal rule (``jscan_prefill_trapezoid``).  ``lam``
    ``[batch, L, D]`` (x's dtype) weights each step's right end; the left end, the previous
    token's input, gets ``1 - lam`` and decays over the step.  ``x_prev [batch, D]`` and
    ``B_prev [batch, 16]`` are the token before the first (omit both for a fresh sequence).
    ``form``: "diagonal" (A ``[D, 16]``), "scalar" (a ``[D]``) or "complex" (A ``[D, 16]`` as
    (real, imaginary) pairs).  Other arguments and results as for :func:`prefill`."""
    _require(form in A_FORMS, f"form must be one of {tuple(A_FORMS)}")
    batch, L, D = _check_prefill_args(x, delta, A, B, C, h0, scalar_a=form == "scalar")
    _require(tuple(lam.shape) == (batch, L, D) and lam.dtype == x.dtype and lam.is_contiguous()
             and lam.device == x.device, "lam must be a contiguous [batch, L, D] tensor like x")
    _require((x_prev is None) == (B_prev is None), "x_prev and B_prev go together")
    if x_prev is not None:
        for name, t, shape in (("x_prev", x_prev, (batch, D)), ("B_prev", B_prev, (batch, D_STATE))):
            _require(tuple(t.shape) == shape and t.dtype == x.dtype and t.is_contiguous() and t.device == x.device,
                     f"{name} must be a contiguous {shape} tensor like x")
    if y is None:
        y = torch.empty_like(x)
    if h_final is None:
        h_final = torch.empty((batch, D, D_STATE), dtype=torch.float32, device=x.device)
    lib = library()
    with torch.cuda.device(x.device):
        st = lib.jscan_prefill_trapezoid(_ptr(x), _ptr(delta), _ptr(lam), _ptr(A), _ptr(B), _ptr(C), _ptr(h0),
                                         _ptr(x_prev), _ptr(B_prev), _ptr(y), _ptr(h_final), batch, L, D, D_STATE,
                                         A_FORMS[form], _DTYPES[x.dtype], _stream(x.device))
    _check(st)
    return y, h_final


def step_trapezoid(h, x_prev, B_prev, x_t, delta_t, lam_t, A, B_t, C_t, form="diagonal", y_t=None):
    """One decode token with the exponential-trapezoidal rule (``jscan_step_trapezoid``): as
    :func:`step`, plus the previous token's ``x_prev [batch, D]`` and ``B_prev [batch, 16]``
    (zeros before a sequence's first token) and this token's ``lam_t [batch, D]``.  x_prev and
    lam_t share x_t's row stride, B_prev shares B_t's."""
    _require(form in A_FORMS, f"form must be one of {tuple(A_FORMS)}")
    _require(h.is_cuda and h.dtype == torch.float32 and h.dim() == 3 and h.shape[2] == D_STATE and h.is_contiguous(),
             "h must be a contiguous fp32 [batch, D, 16] CUDA tensor")
    batch, D, _ = h.shape
    _require(x_t.dtype in _DTYPES, "x_t must be bfloat16 or float32")
    ld_xd = x_t.stride(0) if batch > 1 else D
    ld_bc = B_t.stride(0) if batch > 1 else D_STATE
    for name, t, shape, ld in (("x_t", x_t, (batch, D), ld_xd), ("delta_t", delta_t, (batch, D), ld_xd),
                               ("lam_t", lam_t, (batch, D), ld_xd), ("x_prev", x_prev, (batch, D), ld_xd),
                               ("B_t", B_t, (batch, D_STATE), ld_bc), ("C_t", C_t, (batch, D_STATE), ld_bc),
                               ("B_prev", B_prev, (batch, D_STATE), ld_bc)):
        _require(tuple(t.shape) == shape, f"{name} must have shape {shape}")
        _require(t.dtype == x_t.dtype, f"{name} must be {x_t.dtype}")
        _require(t.stride(1) == 1 and (batch <= 1 or t.stride(0) == ld), f"{name} rows must be contiguous with "
                 f"the row stride of {'x_t' if ld is ld_xd else 'B_t'}")
        _require(t.device == h.device, f"{name} is on another device")
    a_shape = (D,) if form == "scalar" else (D, D_STATE)
    _require(A.dtype == torch.float32 and tuple(A.shape) == a_shape and A.is_contiguous(),
             f"A must be a contiguous fp32 tensor of shape {a_shape}")
    y_t, ld_y = _step_output(y_t, (batch, D), x_t.dtype, h.device)
    lib = library()
    with torch.cuda.device(h.device):
        st = lib.jscan_step_trapezoid(_ptr(h), _ptr(x_prev), _ptr(B_prev), _ptr(x_t), _ptr(delta_t), _ptr(lam_t),
                                      _ptr(A), _ptr(B_t), _ptr(C_t), _ptr(y_t), batch, D, D_STATE, ld_xd, ld_bc,
                                      ld_y, A_FORMS[form], _DTYPES[x_t.dtype], _stream(h.device))
    _check(st)
    return y_t


# ---- multi-input, multi-output (MIMO) --------------------------------------------------------

def prefill_mimo(x, delta, A, B, C, h0=None, form="diagonal", y=None, h_final=None):
    """MIMO prefill (``jscan_prefill_mimo``): each channel takes R inputs and gives R outputs.
    x ``[batch, L, D, R]``, delta ``[batch, L, D]``, B, C ``[batch, L, 16, R]`` (one dtype),
    A as for ``form`` ("diagonal" ``[D, 16]``, "scalar" ``[D]``, "complex" ``[D, 16]``), optional
    h0 ``[batch, D, 16]``; R is 1, 2, 4 or 8.  Returns ``(y [batch, L, D, R], h_final)``."""
    batch, L, D, R = _check_mimo_args(x, delta, A, B, C, h0, form)
    if y is None:
        y = torch.empty_like(x)
    if h_final is None:
        h_final = torch.empty((batch, D, D_STATE), dtype=torch.float32, device=x.device)
    lib = library()
    with torch.cuda.device(x.device):
        st = lib.jscan_prefill_mimo(_ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(h0), _ptr(y), _ptr(h_final),
                                    batch, L, D, D_STATE, R, A_FORMS[form], _DTYPES[x.dtype], _stream(x.device))
    _check(st)
    return y, h_final


def _check_mimo_args(x, delta, A, B, C, h0, form):
    _require(form in A_FORMS, f"form must be one of {tuple(A_FORMS)}")
    _require(x.is_cuda and x.dtype in _DTYPES and x.dim() == 4 and x.is_contiguous(),
             "x must be a contiguous [batch, L, D, R] CUDA tensor (bfloat16 or float32)")
    batch, L, D, R = x.shape
    a_shape = (D,) if form == "scalar" else (D, D_STATE)
    for name, t, shape, dt in (("delta", delta, (batch, L, D), x.dtype), ("A", A, a_shape, torch.float32),
                               ("B", B, (batch, L, D_STATE, R), x.dtype), ("C", C, (batch, L, D_STATE, R), x.dtype)):
        _require(tuple(t.shape) == shape, f"{name} must have shape {shape}, got {tuple(t.shape)}")
        _require(t.dtype == dt and t.is_contiguous() and t.device == x.device, f"{name} must be a contiguous {dt} "
                 "tensor on x's device")
    if h0 is not None:
        _require(tuple(h0.shape) == (batch, D, D_STATE) and h0.dtype == torch.float32 and h0.is_contiguous()
                 and h0.device == x.device, "h0 must be a contiguous fp32 [batch, D, 16] tensor on x's device")
    return batch, L, D, R


def prefill_mimo_trapezoid(x, delta, lam, A, B, C, h0=None, x_prev=None, B_prev=None, form="diagonal", y=None,
                           h_final=None):
    """MIMO prefill with the exponential-trapezoidal rule (``jscan_prefill_mimo_trapezoid``): as
    :func:`prefill_mimo`, plus ``lam`` ``[batch, L, D]`` (the right-end weight, x's dtype) and the
    token before the first, ``x_prev [batch, D, R]`` and ``B_prev [batch, 16, R]`` (omit both for a
    fresh sequence)."""
    batch, L, D, R = _check_mimo_args(x, delta, A, B, C, h0, form)
    _require(tuple(lam.shape) == (batch, L, D) and lam.dtype == x.dtype and lam.is_contiguous()
             and lam.device == x.device, "lam must be a contiguous [batch, L, D] tensor like x")
    _require((x_prev is None) == (B_prev is None), "x_prev and B_prev go together")
    if x_prev is not None:
        for name, t, shape in (("x_prev", x_prev, (batch, D, R)), ("B_prev", B_prev, (batch, D_STATE, R))):
            _require(tuple(t.shape) == shape and t.dtype == x.dtype and t.is_contiguous() and t.device == x.device,
                     f"{name} must be a contiguous {shape} tensor like x")
    if y is None:
        y = torch.empty_like(x)
    if h_final is None:
        h_final = torch.empty((batch, D, D_STATE), dtype=torch.float32, device=x.device)
    lib = library()
    with torch.cuda.device(x.device):
        st = lib.jscan_prefill_mimo_trapezoid(_ptr(x), _ptr(delta), _ptr(lam), _ptr(A), _ptr(B), _ptr(C), _ptr(h0),
                                              _ptr(x_prev), _ptr(B_prev), _ptr(y), _ptr(h_final), batch, L, D, D_STATE,
                                              R, A_FORMS[form], _DTYPES[x.dtype], _stream(x.device))
    _check(st)
    return y, h_final


def step_mimo_trapezoid(h, x_prev, B_prev, x_t, delta_t, lam_t, A, B_t, C_t, form="diagonal", y_t=None):
    """One MIMO decode token with the exponential-trapezoidal rule (``jscan_step_mimo_trapezoid``):
    as :func:`step_mimo`, plus the previous token's ``x_prev [batch, D, R]`` (x_t's row stride) and
    ``B_prev [batch, 16, R]`` (B_t's) and this token's ``lam_t [batch, D]`` (delta_t's)."""
    return step_mimo(h, x_t, delta_t, A, B_t, C_t, form=form, y_t=y_t, _trap=(x_prev, B_prev, lam_t))


def step_mimo(h, x_t, delta_t, A, B_t, C_t, form="diagonal", y_t=None, _trap=None):
    """One MIMO decode token (``jscan_step_mimo``): h ``[batch, D, 16]`` fp32 in place; x_t
    ``[batch, D, R]``, delta_t ``[batch, D]``, B_t, C_t ``[batch, 16, R]`` (each row contiguous;
    rows may be strided views of prefill tensors, e.g. ``x[:, t]``).  Returns y_t ``[batch, D, R]``."""
    _require(form in A_FORMS, f"form must be one of {tuple(A_FORMS)}")
    _require(h.is_cuda and h.dtype == torch.float32 and h.dim() == 3 and h.shape[2] == D_STATE and h.is_contiguous(),
             "h must be a contiguous fp32 [batch, D, 16] CUDA tensor")
    batch, D, _ = h.shape
    _require(x_t.dim() == 3 and x_t.shape[:2] == (batch, D) and x_t.dtype in _DTYPES, "x_t must be [batch, D, R]")
    R = x_t.shape[2]
    _require(x_t.stride(2) == 1 and x_t.stride(1) == R, "x_t rows must be contiguous")
    _require(tuple(delta_t.shape) == (batch, D) and delta_t.stride(1) == 1 and delta_t.dtype == x_t.dtype,
             "delta_t must be [batch, D] with contiguous rows, x_t's dtype")
    for name, t in (("B_t", B_t), ("C_t", C_t)):
        _require(tuple(t.shape) == (batch, D_STATE, R) and t.dtype == x_t.dtype and t.stride(2) == 1
                 and t.stride(1) == R, f"{name} must be [batch, 16, R] with contiguous rows, x_t's dtype")
    a_shape = (D,) if form == "scalar" else (D, D_STATE)
    _require(A.dtype == torch.float32 and tuple(A.shape) == a_shape and A.is_contiguous(),
             f"A must be a contiguous fp32 tensor of shape {a_shape}")
    ld_x = x_t.stride(0) if batch > 1 else D * R
    ld_d = delta_t.stride(0) if batch > 1 else D
    ld_bc = B_t.stride(0) if batch > 1 else D_STATE * R
    _require(batch <= 1 or C_t.stride(0) == ld_bc, "B_t and C_t must share a row stride")
    if _trap is not None:
        x_prev, B_prev, lam_t = _trap
        for name, t, shape, ld in (("x_prev", x_prev, (batch, D, R), ld_x), ("B_prev", B_prev, (batch, D_STATE, R), ld_bc),
                                   ("lam_t", lam_t, (batch, D), ld_d)):
            _require(tuple(t.shape) == shape and t.dtype == x_t.dtype and t.device == h.device
                     and t.stride(-1) == 1 and (t.dim() == 2 or t.stride(1) == R) and (batch <= 1 or t.stride(0) == ld),
                     f"{name} must be {shape} with contiguous rows and the row stride of the matching input")
    y_t, ld_y = _step_output(y_t, (batch, D, R), x_t.dtype, h.device)
    lib = library()
    with torch.cuda.device(h.device):
        if _trap is None:
            st = lib.jscan_step_mimo(_ptr(h), _ptr(x_t), _ptr(delta_t), _ptr(A), _ptr(B_t), _ptr(C_t), _ptr(y_t), batch,
                                     D, D_STATE, R, ld_x, ld_d, ld_bc, ld_y, A_FORMS[form], _DTYPES[x_t.dtype],
                                     _stream(h.device))
        else:
            st = lib.jscan_step_mimo_trapezoid(_ptr(h), _ptr(_trap[0]), _ptr(_trap[1]), _ptr(x_t), _ptr(delta_t),
                                               _ptr(_trap[2]), _ptr(A), _ptr(B_t), _ptr(C_t), _ptr(y_t), batch, D,
                                               D_STATE, R, ld_x, ld_d, ld_bc, ld_y, A_FORMS[form],
                                               _DTYPES[x_t.dtype], _stream(h.device))
    _check(st)
    return y_t


# ---- gated recurrence ------------------------------------------------------------------------
# jscan_gate_form values: how the gate makes the decay.
GATE_FORMS = {"decay": 0, "sigmoid": 1}

# A decode token's kernels take a few microseconds, as much as a handful of Python calls: the checks below
# build their messages only when they fail, and a launch asks for the raw stream and changes the current
# device only where it has to.  New tensors take their sizes one by one (a torch.Size costs torch.empty 0.8 us
# more of its 2.1).
_F32, _I8, _I32 = torch.float32, torch.int8, torch.int32
# Its private accessors where torch has them; the public ones build a Stream object and check the device's state.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
# The level of forward-mode differentiation (-1 outside of it), where torch shows it; unpack_dual finds it by itself.
_dual = forward_ad if hasattr(forward_ad, "_current_level") else types.SimpleNamespace(_current_level=0)
_forward_mode = getattr(torch._C, "_is_fwd_grad_enabled", None) or (lambda: True)


def _launch(name, dev, *args):
    """Library function `name` on args and dev's current stream, with dev current; raises on an error status."""
    fn = getattr(_lib or library(), name)
    index = dev.index
    if index == _current_device():
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status:
        _check(status)


def _addr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _bad(msg: str):
    raise ValueError(msg)


def _refuse_grad():
    """For calls on tensors that require gradients, which autograd would lose without a word where it records."""
    if torch.is_grad_enabled():
        _bad("autograd does not record this call: make it under torch.no_grad(), on detached tensors, or inside a "
             "torch.autograd.Function whose backward gives its gradients (gated_scan_backward for gated_scan, and so on)")


def _refuse_tangents(*tensors):
    """The same for forward mode: its tensors carry a tangent and do not require gradients, and no_grad does not stop it."""
    if _forward_mode() and any(t is not None and forward_ad.unpack_dual(t).tangent is not None for t in tensors):
        _bad("forward-mode differentiation does not pass through this call: make it on detached tensors, or inside a "
             "torch.autograd.Function whose jvp gives the tangent")


def _check_like(name, t, shape, dtype, dev):
    if t.shape != shape or t.dtype != dtype or t.device != dev:
        _bad(f"{name} must have shape {tuple(shape)} and be {dtype} on {dev}, got {tuple(t.shape)}, {t.dtype}, {t.device}")


def _matrix(name, t, shape, dtype, dev):
    """The strides of a matrix of this shape."""
    if t.shape != shape or t.dtype != dtype or t.device != dev:
        _check_like(name, t, shape, dtype, dev)
    return t.stride()


def _check_flat(name, t, shape, dtype, dev):
    """t is None or a contiguous tensor of this shape and dtype on dev."""
    if t is not None and (t.shape != shape or t.dtype != dtype or t.device != dev or not t.is_contiguous()):
        _check_like(name, t, shape, dtype, dev)
        _bad(f"{name} must be contiguous")


def _token_rows(name, t, like, shape):
    """The token stride in elements of a [batch, L, D] tensor whose rows are contiguous and evenly
    spaced (contiguous, or a slice of a wider last dimension)."""
    if t is not like and (t.shape != shape or t.dtype != like.dtype or t.device != like.device):
        _check_like(name, t, shape, like.dtype, like.device)
    batch, L, D = shape
    s_b, s_t, s_d = t.stride()
    if s_d != 1 and D > 1:
        _bad(f"{name} rows must be contiguous")
    if L > 1:
        if batch > 1 and s_b != L * s_t:
            _bad(f"{name}: sequences must follow each other at the token stride")
        return s_t
    return s_b if batch > 1 else D


def _check_gated(g, form, lengths):
    if form not in GATE_FORMS:
        _bad(f"form must be one of {tuple(GATE_FORMS)}")
    if not g.is_cuda:
        _bad("inputs must be CUDA (HIP) tensors")
    if g.dtype not in _DTYPES:
        _bad("g must be bfloat16 or float32")
    if g.dim() != 3:
        _bad("g must be [batch, L, D]")
    _check_flat("lengths", lengths, g.shape[:1], _I32, g.device)


def gated_scan_workspace_bytes(batch: int, L: int, D: int) -> int:
    """Bytes of workspace ``gated_scan`` and ``gated_scan_backward`` need (0 for most shapes)."""
    n = library().jscan_gated_scan_workspace(batch, L, D)
    if n < 0:
        raise ValueError(f"invalid shape: batch={batch} L={L} D={D}")
    return n


def _gated_workspace(workspace, batch, L, D, dev):
    return _workspace(workspace, gated_scan_workspace_bytes(batch, L, D), dev)


def _workspace(workspace, need, dev):
    """The caller's workspace, or a new one of `need` bytes (None for 0), and its size."""
    if workspace is None:
        return (torch.empty(need, dtype=torch.uint8, device=dev), need) if need > 0 else (None, 0)
    if workspace.device != dev or not workspace.is_contiguous():
        _bad(f"workspace must be contiguous and on {dev}")
    return workspace, workspace.numel() * workspace.element_size()


def gated_scan_states(g):
    """A new tensor for the states that :func:`gated_scan` of g ``[batch, L, D]`` bf16 keeps for its backward pass:
    ``[batch, ceil(L / 8), D]`` fp32, the state before every eighth token.  None for fp32, where y holds them."""
    if g.dtype not in _DTYPES or g.dim() != 3:
        _bad("g must be a bfloat16 or float32 [batch, L, D]")
    batch, L, D = g.shape
    return torch.empty(batch, (L + 7) // 8, D, dtype=_F32, device=g.device) if g.dtype != _F32 else None


def _check_states(states, g):
    if g.dtype == _F32:
        _bad("states are for bfloat16 tensors: with float32, y holds them")
    batch, L, D = g.shape
    _check_flat("states", states, (batch, (L + 7) // 8, D), _F32, g.device)


def gated_scan(g, u, h0=None, lengths=None, form="decay", y=None, h_final=None, workspace=None, states=None):
    """Gated recurrence over whole sequences (``jscan_gated_scan``).  g, u ``[batch, L, D]`` (bf16 or
    fp32; rows may be slices of a wider projection): ``h_t = a h_{t-1} + u_t`` with ``a = exp(g_t)``
    (form "decay"), or ``h_t = a h_{t-1} + (1 - a) u_t`` with ``a = sigmoid(g_t)`` (form "sigmoid").  h0
    ``[batch, D]`` fp32; ``lengths`` int32 ``[batch]`` for padded sequences (y is zero in the padding).
    Returns ``(y [batch, L, D] in g's dtype, h_final [batch, D] fp32)``; ``h_final`` may be ``h0``.  For training
    in bf16, ``states`` from :func:`gated_scan_states` keeps fp32 states for the backward pass.

    ``g = -inf`` drops a finite state (a reset inside a row); an infinity or a NaN stays in its channel to the
    end of its sequence.  Decays above one (g > 0 in the decay form) have to multiply to a finite fp32 number over
    any run of tokens: runs are composed before they meet their starting state.  Autograd does not record the
    call: tensors that require gradients are refused where it would (:func:`gated_scan_backward` has them)."""
    if g.requires_grad or u.requires_grad or (h0 is not None and h0.requires_grad):
        _refuse_grad()
    if _dual._current_level >= 0:
        _refuse_tangents(g, u, h0)
    _check_gated(g, form, lengths)
    shape, dev = g.shape, g.device
    batch, L, D = shape
    ld_g, ld_u = _token_rows("g", g, g, shape), _token_rows("u", u, g, shape)
    state = (batch, D)
    _check_flat("h0", h0, state, _F32, dev)
    if y is None:
        y, ld_y = torch.empty(batch, L, D, dtype=g.dtype, device=dev), D
    else:
        ld_y = _token_rows("y", y, g, shape)
    if h_final is None:
        h_final = torch.empty(batch, D, dtype=_F32, device=dev)
    else:
        _check_flat("h_final", h_final, state, _F32, dev)
    workspace, ws_bytes = _gated_workspace(workspace, batch, L, D, dev)
    if states is None:
        _launch("jscan_gated_scan", dev, g.data_ptr(), u.data_ptr(), _addr(h0), _addr(lengths), y.data_ptr(),
                h_final.data_ptr(), batch, L, D, ld_g, ld_u, ld_y, _addr(workspace), ws_bytes, GATE_FORMS[form],
                _DTYPES[g.dtype])
    else:
        _check_states(states, g)
        _launch("jscan_gated_scan_save", dev, g.data_ptr(), u.data_ptr(), _addr(h0), _addr(lengths), y.data_ptr(),
                h_final.data_ptr(), states.data_ptr(), batch, L, D, ld_g, ld_u, ld_y, _addr(workspace), ws_bytes,
                GATE_FORMS[form], _DTYPES[g.dtype])
    return y, h_final


def gated_scan_backward(g, u, y, dy, h0=None, dh_final=None, lengths=None, form="decay", dg=None, du=None, dh0=None,
                        workspace=None, states=None):
    """Gradients of :func:`gated_scan` (``jscan_gated_scan_backward``): g, u, h0, lengths and form as given
    to it, y as it returned, dy ``[batch, L, D]`` and optionally dh_final ``[batch, D]`` fp32 the gradients of
    its results.  The decay form does not read u (it may be None).  Returns ``(dg, du, dh0)``; dg and du
    may be given as the halves of one wider gradient.

    The state before each token is read from y.  In bf16 that is its rounded value, and dg is off by up to
    ``2**-8 * |c * h|`` (sigmoid: ``2**-8 * |c * (1 - a) * h|``, which may be a large part of it where states and
    inputs are close).  With the ``states`` that the scan kept, h is in fp32 throughout; u is then needed
    in both forms, and y and h0 are not read (they may be None)."""
    if g.requires_grad or dy.requires_grad or any(t is not None and t.requires_grad for t in (u, y, h0, dh_final)):
        _refuse_grad()
    if _dual._current_level >= 0:
        _refuse_tangents(g, u, y, dy, h0, dh_final)
    _check_gated(g, form, lengths)
    shape, dev = g.shape, g.device
    batch, L, D = shape
    if u is None and (form != "decay" or states is not None):
        _bad("u is needed by the sigmoid form and with states")
    ld_g, ld_dy = _token_rows("g", g, g, shape), _token_rows("dy", dy, g, shape)
    ld_u = D if u is None else _token_rows("u", u, g, shape)
    state = (batch, D)
    if states is None:
        if y is None:
            _bad("y is needed without states")
        ld_y = _token_rows("y", y, g, shape)
        _check_flat("h0", h0, state, _F32, dev)
    else:
        _check_states(states, g)
    _check_flat("dh_final", dh_final, state, _F32, dev)
    if dg is None:
        dg, ld_dg = torch.empty(batch, L, D, dtype=g.dtype, device=dev), D
    else:
        ld_dg = _token_rows("dg", dg, g, shape)
    if du is None:
        du, ld_du = torch.empty(batch, L, D, dtype=g.dtype, device=dev), D
    else:
        ld_du = _token_rows("du", du, g, shape)
    if dh0 is None:
        dh0 = torch.empty(batch, D, dtype=_F32, device=dev)
    else:
        _check_flat("dh0", dh0, state, _F32, dev)
    workspace, ws_bytes = _gated_workspace(workspace, batch, L, D, dev)
    if states is None:
        _launch("jscan_gated_scan_backward", dev, g.data_ptr(), _addr(u), y.data_ptr(), dy.data_ptr(), _addr(h0),
                _addr(dh_final), _addr(lengths), dg.data_ptr(), du.data_ptr(), dh0.data_ptr(), batch, L, D, ld_g, ld_u,
                ld_y, ld_dy, ld_dg, ld_du, _addr(workspace), ws_bytes, GATE_FORMS[form], _DTYPES[g.dtype])
    else:
        _launch("jscan_gated_scan_backward_saved", dev, g.data_ptr(), u.data_ptr(), states.data_ptr(), dy.data_ptr(),
                _addr(dh_final), _addr(lengths), dg.data_ptr(), du.data_ptr(), dh0.data_ptr(), batch, L, D, ld_g, ld_u,
                ld_dy, ld_dg, ld_du, _addr(workspace), ws_bytes, GATE_FORMS[form], _DTYPES[g.dtype])
    return dg, du, dh0


def gated_step(h, g_t, u_t, y_t=None, form="decay"):
    """One decode token of the gated recurrence (``jscan_gated_step``): h ``[batch, D]`` fp32 is updated in
    place; g_t, u_t ``[batch, D]`` may be strided views, e.g. ``g[:, t]``.  Returns y_t ``[batch, D]``: a new
    contiguous tensor, or the given ``y_t``, whose rows may be strided too."""
    if h.requires_grad or g_t.requires_grad or u_t.requires_grad:
        _refuse_grad()
    if _dual._current_level >= 0:
        _refuse_tangents(h, g_t, u_t)
    code = GATE_FORMS.get(form)
    if code is None:
        _bad(f"form must be one of {tuple(GATE_FORMS)}")
    if not h.is_cuda or h.dtype != _F32 or h.dim() != 2 or not h.is_contiguous():
        _bad("h must be a contiguous fp32 [batch, D] CUDA tensor")
    shape, dev, dtype = h.shape, h.device, g_t.dtype
    if dtype not in _DTYPES:
        _bad("g_t must be bfloat16 or float32")
    batch, D = shape
    ld_g, one_g = _matrix("g_t", g_t, shape, dtype, dev)
    ld_u, one_u = _matrix("u_t", u_t, shape, dtype, dev)
    if y_t is None:
        y_t, ld_y, one_y = torch.empty(batch, D, dtype=dtype, device=dev), D, 1
    else:
        ld_y, one_y = _matrix("y_t", y_t, shape, dtype, dev)
    if D > 1 and not one_g == one_u == one_y == 1:
        _bad("the rows of g_t, u_t and y_t must be contiguous")
    if batch <= 1:
        ld_g = ld_u = ld_y = D
    _launch("jscan_gated_step", dev, h.data_ptr(), g_t.data_ptr(), u_t.data_ptr(), y_t.data_ptr(), batch, D, ld_g, ld_u, ld_y,
            code, _DTYPES[dtype])
    return y_t


# ---- int8 projection -------------------------------------------------------------------------
# jscan_activation values.
ACTIVATIONS = {"none": 0, "silu": 1, "gelu_tanh": 2}


def _row_stride(name, t):
    """The stride in elements of the rows of ``[..., K]``: contiguous rows, evenly spaced over all leading
    dimensions (contiguous, or a slice of a wider last dimension)."""
    K = t.shape[-1]
    if t.is_contiguous():
        return K
    if K > 1 and t.stride(-1) != 1:
        _bad(f"{name} rows must be contiguous")
    lead = [(n, s) for n, s in zip(t.shape[:-1], t.stride()[:-1]) if n != 1]
    for (_, outer), (n, inner) in zip(lead, lead[1:]):
        if outer != n * inner:
            _bad(f"{name} rows must be evenly spaced")
    return lead[-1][1] if lead else K


def quantize_rows(x, q=None, scale=None):
    """Rows of x ``[..., K]`` (bf16 or fp32, K a multiple of 16; a slice of a wider tensor too) to int8, each
    with a scale of its own (``jscan_quantize_rows``).  Returns ``(q [..., K] int8, scale [...] fp32)``: the
    first input of :func:`matmul_i8`."""
    if x.requires_grad:
        _refuse_grad()
    if _dual._current_level >= 0:
        _refuse_tangents(x)
    if not x.is_cuda or x.dtype not in _DTYPES:
        _bad("x must be a bfloat16 or float32 CUDA tensor")
    if x.dim() < 1:
        _bad("x must have a last dimension")
    shape, dev = x.shape, x.device
    K, lead = shape[-1], shape[:-1]
    ld_x = _row_stride("x", x)
    if q is None:
        q = torch.empty(*shape, dtype=_I8, device=dev)
    else:
        _check_flat("q", q, shape, _I8, dev)
    if scale is None:
        scale = torch.empty(*(lead or ((),)), dtype=_F32, device=dev)   # () is no list of sizes
    else:
        _check_flat("scale", scale, lead, _F32, dev)
    _launch("jscan_quantize_rows", dev, x.data_ptr(), q.data_ptr(), scale.data_ptr(), lead.numel(), K, ld_x,
            _DTYPES[x.dtype])
    return q, scale


def matmul_i8(q, q_scale, w, w_scale, bias=None, out=None, out_dtype=torch.bfloat16, activation="none", residual=None):
    """``out = (q @ w.T) * q_scale * w_scale + bias`` from int8 q ``[..., K]`` and w ``[N, K]`` with fp32 scales
    ``[...]`` (a token each) and ``[N]`` (an output channel each) and an optional fp32 bias ``[N]``
    (``jscan_matmul_i8``).  Returns out ``[..., N]`` in out_dtype; a given ``out`` may be a slice of a wider
    tensor.  An ``activation`` ("silu" or "gelu_tanh") and a ``residual`` ``[..., N]`` in out's dtype are applied before the
    one rounding, ``act(...) + residual`` (``jscan_matmul_i8_epilogue``); ``out`` may be the residual itself."""
    if q_scale.requires_grad or w_scale.requires_grad or (bias is not None and bias.requires_grad) or \
            (residual is not None and residual.requires_grad):
        _refuse_grad()
    if _dual._current_level >= 0:
        _refuse_tangents(q_scale, w_scale, bias, residual)
    code = ACTIVATIONS.get(activation)
    if code is None:
        _bad(f"activation must be one of {tuple(ACTIVATIONS)}")
    if not q.is_cuda or q.dtype != torch.int8 or q.dim() < 1 or not q.is_contiguous():
        _bad("q must be a contiguous int8 CUDA tensor")
    dev, K, lead = q.device, q.shape[-1], q.shape[:-1]
    if w.dim() != 2 or w.shape[1] != K:
        _bad(f"w must be [N, {K}], got {tuple(w.shape)}")
    N = w.shape[0]
    _check_flat("w", w, (N, K), _I8, dev)
    _check_flat("q_scale", q_scale, lead, _F32, dev)
    _check_flat("w_scale", w_scale, (N,), _F32, dev)
    _check_flat("bias", bias, (N,), _F32, dev)
    if out is None:
        if out_dtype not in _DTYPES:
            _bad("out_dtype must be bfloat16 or float32")
        out, ld_out = torch.empty(*lead, N, dtype=out_dtype, device=dev), N
    else:
        if out.dtype not in _DTYPES:
            _bad("out must be bfloat16 or float32")
        _check_like("out", out, (*lead, N), out.dtype, dev)
        ld_out = _row_stride("out", out)
    if code or residual is not None:
        ld_residual = N
        if residual is not None:
            _check_like("residual", residual, out.shape, out.dtype, dev)
            ld_residual = _row_stride("residual", residual)
        _launch("jscan_matmul_i8_epilogue", dev, q.data_ptr(), q_scale.data_ptr(), w.data_ptr(), w_scale.data_ptr(),
                _addr(bias), _addr(residual), out.data_ptr(), lead.numel(), N, K, ld_residual, ld_out, code,
                _DTYPES[out.dtype])
        return out
    _launch("jscan_matmul_i8", dev, q.data_ptr(), q_scale.data_ptr(), w.data_ptr(), w_scale.data_ptr(),
            _addr(bias), out.data_ptr(), lead.numel(), N, K, ld_out, _DTYPES[out.dtype])
    return out


# ---- scan with skip and output gate ----------------------------------------------------------


def prefill_gate_workspace_bytes(batch: int, L: int, D: int, chunk: int = 0) -> int:
    """Bytes of workspace ``prefill_gate`` needs (0 when it runs token by token)."""
    n = library().jscan_prefill_gate_workspace(batch, L, D, D_STATE, chunk)
    if n < 0:
        raise ValueError(f"invalid shape or chunk: batch={batch} L={L} D={D} chunk={chunk}")
    return n


def prefill_gate(x, delta, A, B, C, skip=None, z=None, h0=None, form="diagonal", chunk=None, y=None, h_final=None,
                 workspace=None):
    """Selective scan with its skip and output gate in one pass (``jscan_prefill_gate``):
    ``y = (scan(x) + skip * x) * silu(z)``, with ``skip`` ``[D]`` fp32 and z ``[batch, L, D]`` in x's dtype (rows may be a
    half of a wider projection); either may be None.  Other arguments and results as for :func:`prefill`, A as the
    ``form`` has it.  ``chunk`` None scans token by token (h_final is bit for bit :func:`prefill`'s), a segment length as
    :func:`prefill_chunked` does, and 0 whichever way is expected to be fastest (form "diagonal"; the others take 0 as None).
    The sum over the states is fp32, except that token by token in bf16 with D a multiple of 32 it is :func:`prefill`'s, which
    rounds each state to bf16 first: of the diagonal form with ``chunk=None``, of the others always.
    ``workspace`` of :func:`prefill_gate_workspace_bytes`, or one is allocated.  There are no lengths: in a padded batch
    ``delta`` has to be zero behind every sequence, which keeps its state.  Autograd does not record the call."""
    if x.requires_grad or delta.requires_grad or A.requires_grad or B.requires_grad or C.requires_grad or \
            any(t is not None and t.requires_grad for t in (skip, z, h0)):
        _refuse_grad()
    if _dual._current_level >= 0:
        _refuse_tangents(x, delta, A, B, C, skip, z, h0)
    code = A_FORMS.get(form)
    if code is None:
        _bad(f"form must be one of {tuple(A_FORMS)}")
    if not x.is_cuda or x.dtype not in _DTYPES or x.dim() != 3 or not x.is_contiguous():
        _bad("x must be a contiguous bfloat16 or float32 [batch, L, D] CUDA tensor")
    shape, dev, dtype = x.shape, x.device, x.dtype
    batch, L, D = shape
    pairs = (batch, L, D_STATE)
    _check_flat("delta", delta, shape, dtype, dev)
    _check_flat("A", A, (D,) if form == "scalar" else (D, D_STATE), _F32, dev)
    _check_flat("B", B, pairs, dtype, dev)
    _check_flat("C", C, pairs, dtype, dev)
    if skip is None and z is None:
        _bad("skip or z is needed (prefill has neither)")
    if chunk is not None and chunk < 0:
        _bad("chunk must be None, 0 or a segment length")
    _check_flat("skip", skip, (D,), _F32, dev)
    ld_z = D if z is None else _token_rows("z", z, x, shape)
    if y is None:
        y = torch.empty_like(x)
    else:
        _check_flat("y", y, shape, dtype, dev)
    state = (batch, D, D_STATE)
    _check_flat("h0", h0, state, _F32, dev)
    if h_final is None:
        h_final = torch.empty(batch, D, D_STATE, dtype=_F32, device=dev)
    else:
        _check_flat("h_final", h_final, state, _F32, dev)
    cut = chunk is not None and form == "diagonal"
    workspace, ws_bytes = _workspace(workspace, prefill_gate_workspace_bytes(batch, L, D, chunk) if cut else 0, dev)
    _launch("jscan_prefill_gate", dev, x.data_ptr(), delta.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(), _addr(h0),
            _addr(skip), _addr(z), y.data_ptr(), h_final.data_ptr(), batch, L, D, D_STATE, ld_z, -1 if chunk is None else chunk,
            _addr(workspace), ws_bytes, code, _DTYPES[dtype])
    return y, h_final


def step_gate(h, x_t, delta_t, A, B_t, C_t, skip=None, z_t=None, form="diagonal", y_t=None):
    """One decode token of :func:`prefill_gate` (``jscan_step_gate``): h ``[batch, D, 16]`` fp32 in place; x_t, delta_t
    and z_t ``[batch, D]``, B_t and C_t ``[batch, 16]`` (rows may be strided, x_t's and delta_t's alike and B_t's and C_t's
    alike).  Returns y_t ``[batch, D]``: a new contiguous tensor, or the given ``y_t``, whose rows may be strided too."""
    if h.requires_grad or x_t.requires_grad or delta_t.requires_grad or A.requires_grad or B_t.requires_grad or \
            C_t.requires_grad or (skip is not None and skip.requires_grad) or (z_t is not None and z_t.requires_grad):
        _refuse_grad()
    if _dual._current_level >= 0:
        _refuse_tangents(h, x_t, delta_t, A, B_t, C_t, skip, z_t)
    code = A_FORMS.get(form)
    if code is None:
        _bad(f"form must be one of {tuple(A_FORMS)}")
    if not h.is_cuda or h.dtype != _F32 or h.dim() != 3 or h.shape[2] != D_STATE or not h.is_contiguous():
        _bad("h must be a contiguous fp32 [batch, D, 16] CUDA tensor")
    dev, dtype = h.device, x_t.dtype
    if dtype not in _DTYPES:
        _bad("x_t must be bfloat16 or float32")
    if skip is None and z_t is None:
        _bad("skip or z_t is needed (step has neither)")
    batch, D, _ = h.shape
    shape, pair = (batch, D), (batch, D_STATE)
    _check_flat("A", A, (D,) if form == "scalar" else (D, D_STATE), _F32, dev)
    _check_flat("skip", skip, (D,), _F32, dev)
    ld_x, one_x = _matrix("x_t", x_t, shape, dtype, dev)
    ld_d, one_d = _matrix("delta_t", delta_t, shape, dtype, dev)
    ld_b, one_b = _matrix("B_t", B_t, pair, dtype, dev)
    ld_c, one_c = _matrix("C_t", C_t, pair, dtype, dev)
    ld_z, one_z = (D, 1) if z_t is None else _matrix("z_t", z_t, shape, dtype, dev)
    if y_t is None:
        y_t, ld_y, one_y = torch.empty(batch, D, dtype=dtype, device=dev), D, 1
    else:
        ld_y, one_y = _matrix("y_t", y_t, shape, dtype, dev)
    if not one_x == one_d == one_b == one_c == one_z == one_y == 1:
        _bad("the rows of x_t, delta_t, B_t, C_t, z_t and y_t must be contiguous")
    if batch <= 1:
        ld_x = ld_d = ld_z = ld_y = D
        ld_b = ld_c = D_STATE
    if ld_x != ld_d or ld_b != ld_c:
        _bad("x_t and delta_t must share a row stride, and so must B_t and C_t")
    _launch("jscan_step_gate", dev, h.data_ptr(), x_t.data_ptr(), delta_t.data_ptr(), A.data_ptr(), B_t.data_ptr(),
            C_t.data_ptr(), _addr(skip), _addr(z_t), y_t.data_ptr(), batch, D, D_STATE, ld_x, ld_b, ld_z, ld_y, code,
            _DTYPES[dtype])
    return y_t


# ---- short causal convolution ----------------------------------------------------------------


def _conv_activation(name):
    if name not in ("none", "silu"):
        _bad('activation must be "none" or "silu"')
    return ACTIVATIONS[name]


def _check_conv(x, w, bias, state, lengths):
    """The width W of the taps and the shape of the state."""
    if not x.is_cuda:
        _bad("inputs must be CUDA (HIP) tensors")
    if x.dtype not in _DTYPES:
        _bad("x must be bfloat16 or float32")
    if x.dim() != 3:
        _bad("x must be [batch, L, D]")
    dev = x.device
    batch, L, D = x.shape
    if w.dim() != 2 or not 2 <= w.shape[1] <= 4:
        _bad(f"w must be [D, W] with W = 2, 3 or 4, got {tuple(w.shape)}")
    W = w.shape[1]
    # the conditions of _check_flat, which says what is wrong: a call of it costs as much as they do
    if w.dtype != _F32 or w.shape[0] != D or w.device != dev or not w.is_contiguous():
        _check_flat("w", w, (D, W), _F32, dev)
    if bias is not None and (bias.dtype != _F32 or bias.shape != (D,) or bias.device != dev or not bias.is_contiguous()):
        _check_flat("bias", bias, (D,), _F32, dev)
    if state is not None and (state.dtype != x.dtype or state.shape != (batch, W - 1, D) or state.device != dev or
                              not state.is_contiguous()):
        _check_flat("state", state, (batch, W - 1, D), x.dtype, dev)
    if lengths is not None:
        _check_flat("lengths", lengths, (batch,), _I32, dev)
    return W


def causal_conv(x, w, bias=None, state=None, lengths=None, activation="silu", y=None, state_out=None):
    """Short causal convolution of every channel over its own last W tokens (``jscan_causal_conv``), as it stands before
    a scan: ``y_t = act(bias + sum_k w[:, k] x_{t - (W - 1) + k})``.  x ``[batch, L, D]`` (bf16 or fp32; rows may be
    slices of a wider projection), w ``[D, W]`` and bias ``[D]`` fp32 with W = 2, 3 or 4, ``activation`` "silu" or
    "none".  ``state`` ``[batch, W - 1, D]`` in x's dtype are the tokens before the first, oldest first (None: zeros);
    ``lengths`` int32 ``[batch]`` for padded sequences (y is zero in the padding; :func:`prefill_gate` behind it needs delta
    zero there).  Returns ``(y, state_out)``:
    ``state_out`` holds each sequence's last W - 1 tokens, for the next call or :func:`causal_conv_step`, and may be
    ``state`` itself.  Autograd does not record the call (:func:`causal_conv_backward` has its gradients)."""
    if x.requires_grad or w.requires_grad or (bias is not None and bias.requires_grad) or \
            (state is not None and state.requires_grad):
        _refuse_grad()
    if _dual._current_level >= 0:
        _refuse_tangents(x, w, bias, state)
    code = _conv_activation(activation)
    W = _check_conv(x, w, bias, state, lengths)
    shape, dev, dtype = x.shape, x.device, x.dtype
    batch, L, D = shape
    ld_x = _token_rows("x", x, x, shape)
    if y is None:
        y, ld_y = torch.empty(batch, L, D, dtype=dtype, device=dev), D
    else:
        ld_y = _token_rows("y", y, x, shape)
    if state_out is None:
        state_out = torch.empty(batch, W - 1, D, dtype=dtype, device=dev)
    else:
        _check_flat("state_out", state_out, (batch, W - 1, D), dtype, dev)
    _launch("jscan_causal_conv", dev, x.data_ptr(), _addr(state), w.data_ptr(), _addr(bias), _addr(lengths), y.data_ptr(),
            state_out.data_ptr(), batch, L, D, W, ld_x, ld_y, code, _DTYPES[dtype])
    return y, state_out


def causal_conv_workspace_bytes(batch: int, L: int, D: int, W: int) -> int:
    """Bytes of workspace ``causal_conv_backward`` needs."""
    n = library().jscan_causal_conv_backward_workspace(batch, L, D, W)
    if n < 0:
        raise ValueError(f"invalid shape: batch={batch} L={L} D={D} W={W}")
    return n


def causal_conv_backward(x, w, dy, bias=None, state=None, dstate_out=None, lengths=None, activation="silu", dx=None,
                         dw=None, dbias=None, dstate=None, workspace=None):
    """Gradients of :func:`causal_conv` (``jscan_causal_conv_backward``): x, w, bias, state, lengths and activation as
    given to it, dy ``[batch, L, D]`` and optionally dstate_out ``[batch, W - 1, D]`` (x's dtype) the gradients of its
    results.  Returns ``(dx, dw, dbias, dstate)``: dx and dstate in x's dtype, dw ``[D, W]`` and dbias ``[D]`` fp32
    sums over all tokens; dbias is None without a bias and dstate without a state.  dx may be given as a slice of a
    wider gradient."""
    if x.requires_grad or w.requires_grad or dy.requires_grad or (bias is not None and bias.requires_grad) or \
            (state is not None and state.requires_grad) or (dstate_out is not None and dstate_out.requires_grad):
        _refuse_grad()
    if _dual._current_level >= 0:
        _refuse_tangents(x, w, dy, bias, state, dstate_out)
    code = _conv_activation(activation)
    W = _check_conv(x, w, bias, state, lengths)
    shape, dev, dtype = x.shape, x.device, x.dtype
    batch, L, D = shape
    past = (batch, W - 1, D)
    ld_x, ld_dy = _token_rows("x", x, x, shape), _token_rows("dy", dy, x, shape)
    _check_flat("dstate_out", dstate_out, past, dtype, dev)
    if dx is None:
        dx, ld_dx = torch.empty(batch, L, D, dtype=dtype, device=dev), D
    else:
        ld_dx = _token_rows("dx", dx, x, shape)
    if dw is None:
        dw = torch.empty(D, W, dtype=_F32, device=dev)
    else:
        _check_flat("dw", dw, (D, W), _F32, dev)
    if bias is None:
        if dbias is not None:
            _bad("dbias goes with a bias")
    elif dbias is None:
        dbias = torch.empty(D, dtype=_F32, device=dev)
    else:
        _check_flat("dbias", dbias, (D,), _F32, dev)
    if state is None:
        if dstate is not None:
            _bad("dstate goes with a state")
    elif dstate is None:
        dstate = torch.empty(batch, W - 1, D, dtype=dtype, device=dev)
    else:
        _check_flat("dstate", dstate, past, dtype, dev)
    workspace, ws_bytes = _workspace(workspace, causal_conv_workspace_bytes(batch, L, D, W), dev)
    _launch("jscan_causal_conv_backward", dev, x.data_ptr(), _addr(state), w.data_ptr(), _addr(bias), _addr(lengths),
            dy.data_ptr(), _addr(dstate_out), dx.data_ptr(), _addr(dstate), dw.data_ptr(), _addr(dbias), batch, L, D, W,
            ld_x, ld_dy, ld_dx, _addr(workspace), ws_bytes, code, _DTYPES[dtype])
    return dx, dw, dbias, dstate


def causal_conv_step(state, x_t, w, bias=None, activation="silu", y_t=None):
    """One decode token of the convolution (``jscan_causal_conv_step``): state ``[batch, W - 1, D]`` in x_t's dtype is
    updated in place (x_t joins, the oldest token leaves); x_t ``[batch, D]`` may be a strided view, e.g. ``x[:, t]``.
    Returns y_t ``[batch, D]``: a new contiguous tensor, or the given ``y_t``, whose rows may be strided too."""
    if state.requires_grad or x_t.requires_grad or w.requires_grad or (bias is not None and bias.requires_grad):
        _refuse_grad()
    if _dual._current_level >= 0:
        _refuse_tangents(state, x_t, w, bias)
    code = _conv_activation(activation)
    if not state.is_cuda or state.dtype not in _DTYPES or state.dim() != 3 or not state.is_contiguous():
        _bad("state must be a contiguous bfloat16 or float32 [batch, W - 1, D] CUDA tensor")
    dev, dtype = state.device, state.dtype
    batch, past, D = state.shape
    if not 1 <= past <= 3:
        _bad(f"state must be [batch, W - 1, D] with W = 2, 3 or 4, got {tuple(state.shape)}")
    _check_flat("w", w, (D, past + 1), _F32, dev)
    _check_flat("bias", bias, (D,), _F32, dev)
    shape = (batch, D)
    ld_x, one_x = _matrix("x_t", x_t, shape, dtype, dev)
    if y_t is None:
        y_t, ld_y, one_y = torch.empty(batch, D, dtype=dtype, device=dev), D, 1
    else:
        ld_y, one_y = _matrix("y_t", y_t, shape, dtype, dev)
    if D > 1 and not one_x == one_y == 1:
        _bad("the rows of x_t and y_t must be contiguous")
    if batch <= 1:
        ld_x = ld_y = D
    _launch("jscan_causal_conv_step", dev, state.data_ptr(), x_t.data_ptr(), w.data_ptr(), _addr(bias), y_t.data_ptr(), batch,
            D, past + 1, ld_x, ld_y, code, _DTYPES[dtype])
    return y_t


# ---- norm ------------------------------------------------------------------------------------


def _check_norm(x, gain, name="x"):
    """The width and the number of x's rows."""
    if not x.is_cuda or x.dtype not in _DTYPES:
        _bad(f"{name} must be a bfloat16 or float32 CUDA tensor")
    shape = x.shape
    if not shape or shape[-1] < 1:
        _bad(f"{name} must have a last dimension")
    K = shape[-1]
    if gain.shape != (K,) or gain.dtype != _F32 or gain.device != x.device or not gain.is_contiguous():
        _check_flat("gain", gain, (K,), _F32, x.device)
    return K, x.numel() // K


def _new_rows(x):
    """A contiguous tensor of x's shape, dtype and device."""
    return torch.empty_like(x) if x.is_contiguous() else torch.empty(*x.shape, dtype=x.dtype, device=x.device)


def _norm_rows(name, t, like):
    """The row stride of a tensor that has x's shape, dtype and device."""
    if t is not like and (t.shape != like.shape or t.dtype != like.dtype or t.device != like.device):
        _check_like(name, t, like.shape, like.dtype, like.device)
    return like.shape[-1] if t.is_contiguous() else _row_stride(name, t)


def _norm_total(x, residual, total):
    """total's tensor and the row strides of residual and total."""
    if residual is None:
        if total is not None:
            _bad("total goes with a residual (without one it is x)")
        return None, 0, 0
    ld_residual = _norm_rows("residual", residual, x)
    if total is None:
        return _new_rows(x), ld_residual, x.shape[-1]
    return total, ld_residual, _norm_rows("total", total, x)


def rms_norm(x, gain, residual=None, eps=1e-6, y=None, total=None):
    """Root-mean-square norm with the residual's addition in front of it (``jscan_rms_norm``): ``total = x + residual``
    (rounded to x's dtype), ``y = total * gain / sqrt(mean(total ** 2) + eps)`` over the last dimension.  x and residual
    ``[..., K]`` (bf16 or fp32; slices of wider tensors too), gain ``[K]`` fp32.  Returns ``(y, total)``; without a
    residual ``total`` is x.  A given ``total`` may be x or residual itself.  A row with a NaN or an infinity, or whose squares
    overflow (or vanish, with ``eps`` 0), is NaN.  Autograd does not record the call
    (:func:`rms_norm_backward` has its gradients)."""
    if x.requires_grad or gain.requires_grad or (residual is not None and residual.requires_grad):
        _refuse_grad()
    if _dual._current_level >= 0:
        _refuse_tangents(x, gain, residual)
    K, M = _check_norm(x, gain)
    ld_x = K if x.is_contiguous() else _row_stride("x", x)
    total, ld_residual, ld_total = _norm_total(x, residual, total)
    if y is None:
        y, ld_y = _new_rows(x), K
    else:
        ld_y = _norm_rows("y", y, x)
    _launch("jscan_rms_norm", x.device, x.data_ptr(), _addr(residual), gain.data_ptr(), y.data_ptr(), _addr(total),
            M, K, ld_x, ld_residual, ld_y, ld_total, eps, _DTYPES[x.dtype])
    return y, x if total is None else total


def rms_norm_quantize(x, gain, residual=None, eps=1e-6, q=None, scale=None, total=None):
    """:func:`rms_norm` with its output in 8 bits (``jscan_rms_norm_quantize``): returns ``(q [..., K] int8, scale [...]
    fp32, total)``, q and scale the first inputs of :func:`matmul_i8`.  K a multiple of 16."""
    if x.requires_grad or gain.requires_grad or (residual is not None and residual.requires_grad):
        _refuse_grad()
    if _dual._current_level >= 0:
        _refuse_tangents(x, gain, residual)
    K, M = _check_norm(x, gain)
    dev, lead = x.device, x.shape[:-1]
    ld_x = _row_stride("x", x)
    total, ld_residual, ld_total = _norm_total(x, residual, total)
    if q is None:
        q = torch.empty(*x.shape, dtype=_I8, device=dev)
    else:
        _check_flat("q", q, x.shape, _I8, dev)
    if scale is None:
        scale = torch.empty(*(lead or ((),)), dtype=_F32, device=dev)   # () is no list of sizes
    else:
        _check_flat("scale", scale, lead, _F32, dev)
    _launch("jscan_rms_norm_quantize", dev, x.data_ptr(), _addr(residual), gain.data_ptr(), q.data_ptr(), scale.data_ptr(),
            _addr(total), M, K, ld_x, ld_residual, ld_total, eps, _DTYPES[x.dtype])
    return q, scale, x if total is None else total


def rms_norm_workspace_bytes(M: int, K: int) -> int:
    """Bytes of workspace ``rms_norm_backward`` of M rows of K values needs."""
    n = library().jscan_rms_norm_backward_workspace(M, K)
    if n < 0:
        raise ValueError(f"invalid shape: M={M} K={K}")
    return n


def rms_norm_backward(total, gain, dy, dtotal=None, eps=1e-6, dx=None, dgain=None, workspace=None):
    """Gradients of :func:`rms_norm` (``jscan_rms_norm_backward``) from its ``total`` (x where there was no residual): dy
    the gradient of y, dtotal that of total's other uses (None: zeros).  Returns ``(dx, dgain)``: dx the gradient of
    x and of residual alike, in their dtype; dgain ``[K]`` fp32.  A given ``dx`` may be dtotal itself.  A row that has no norm makes its dx
    and all of dgain NaN."""
    if total.requires_grad or gain.requires_grad or dy.requires_grad or (dtotal is not None and dtotal.requires_grad):
        _refuse_grad()
    if _dual._current_level >= 0:
        _refuse_tangents(total, gain, dy, dtotal)
    K, M = _check_norm(total, gain, "total")
    dev = total.device
    ld_total, ld_dy = _row_stride("total", total), _norm_rows("dy", dy, total)
    ld_dtotal = 0 if dtotal is None else _norm_rows("dtotal", dtotal, total)
    if dx is None:
        dx, ld_dx = _new_rows(total), K
    else:
        ld_dx = _norm_rows("dx", dx, total)
    if dgain is None:
        dgain = torch.empty(K, dtype=_F32, device=dev)
    else:
        _check_flat("dgain", dgain, (K,), _F32, dev)
    workspace, ws_bytes = _workspace(workspace, rms_norm_workspace_bytes(M, K), dev)
    _launch("jscan_rms_norm_backward", dev, total.data_ptr(), gain.data_ptr(), dy.data_ptr(), _addr(dtotal), dx.data_ptr(),
            dgain.data_ptr(), M, K, ld_total, ld_dy, ld_dtotal, ld_dx, _addr(workspace), ws_bytes, eps, _DTYPES[total.dtype])
    return dx, dgain
