"""Thin ctypes binding of libqmm.so (include/qmm.h).

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C ABI.  Tensors are torch tensors on the GPU; their
data_ptr() and the current torch stream are passed through.  If the library is
missing the binding raises: there is no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os
from ctypes import POINTER, Structure, c_double, c_float, c_int, c_int64, c_size_t, c_void_p

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libqmm.so")

QMM_F32, QMM_F16, QMM_BF16 = 0, 1, 2
QMM_E_BITS, QMM_E_BLOCK = -3, -4
QMM_ZP_NONE, QMM_ZP_PACKED, QMM_ZP_F16, QMM_ZP_UNIFORM = 0, 1, 2, 3
QMOE_FP, QMOE_INT8_ACT = 0, 1
STATUS = {0: "QMM_OK", -1: "QMM_E_NULL", -2: "QMM_E_DTYPE", -3: "QMM_E_BITS", -4: "QMM_E_BLOCK",
          -5: "QMM_E_SHAPE", -6: "QMM_E_ALIGN", -7: "QMM_E_WORKSPACE", -8: "QMM_E_MODE",
          -9: "QMM_E_DEVICE", -10: "QMM_E_PARAM"}
ENTRY_NBITS, ENTRY_CODEBOOK, ENTRY_QMOE_FC1, ENTRY_QMOE_FC2, ENTRY_QMOE_FUSED = 0, 1, 2, 3, 4


class QmmError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        name = STATUS.get(status, f"hipError {status}")
        super().__init__(f"{fn} failed: {name} ({status})")


class qmoe_weights(Structure):
    _fields_ = [("W", c_void_p), ("scales", c_void_p), ("zp", c_void_p), ("bias", c_void_p)]


class qmm_qparams(Structure):
    _fields_ = [("scale", c_float), ("zero_point", ctypes.c_int32)]


class qmm_nested_absmax(Structure):
    _fields_ = [("codes", c_void_p), ("table", c_void_p), ("scales", c_void_p), ("offset", c_float),
                ("group", c_int)]


class qmm_lora_weights(Structure):
    _fields_ = [("A", c_void_p), ("B", c_void_p), ("scale", c_void_p)]


_lib = None

_SIGS = {
    "qmm_nbits": (c_int, [c_void_p, c_int, c_int64, c_int64, c_int64, c_void_p, c_int, c_int,
                          c_void_p, c_void_p, c_int, c_float, c_void_p, c_void_p, c_int,
                          c_void_p, c_size_t, c_void_p]),
    "qmm_nbits_workspace_bytes": (c_size_t, [c_int64, c_int64, c_int64, c_int]),
    "qmm_validate_nbits": (c_int, [c_void_p, c_int, c_int64, c_int64, c_int64, c_void_p, c_int,
                                   c_int, c_void_p, c_void_p, c_int, c_void_p, c_void_p, c_int,
                                   c_void_p, c_size_t]),
    "qmm_codebook4": (c_int, [c_void_p, c_int, c_int64, c_int64, c_int64, c_void_p, c_int,
                              c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_void_p, c_size_t,
                              c_void_p]),
    "qmm_codebook4_workspace_bytes": (c_size_t, [c_int64, c_int64, c_int64, c_int]),
    "qmm_validate_codebook4": (c_int, [c_void_p, c_int, c_int64, c_int64, c_int64, c_void_p, c_int,
                                       c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_void_p,
                                       c_size_t]),
    "qmm_dequantize_absmax_nested": (c_int, [POINTER(qmm_nested_absmax), c_int64, c_void_p, c_void_p]),
    "qmm_codebook4_nested": (c_int, [c_void_p, c_int, c_int64, c_int64, c_int64, c_void_p, c_int,
                                     POINTER(qmm_nested_absmax), c_void_p, c_void_p, c_void_p, c_int, c_void_p,
                                     c_size_t, c_void_p]),
    "qmm_codebook4_nested_workspace_bytes": (c_size_t, [c_int64, c_int64, c_int64, c_int, c_int]),
    "qmm_fp16_uniform_value": (c_int, [c_void_p, c_int64, c_void_p, c_size_t, POINTER(c_int),
                                       POINTER(c_float), c_void_p]),
    "qmm_uniform_scratch_bytes": (c_size_t, []),
    "qmm_dequantize_nbits": (c_int, [c_void_p, c_int, c_int, c_void_p, c_void_p, c_int, c_float,
                                     c_int64, c_int64, c_void_p, c_int, c_void_p]),
    "qmm_dequantize_codebook4": (c_int, [c_void_p, c_int, c_void_p, c_void_p, c_int64, c_int64,
                                         c_void_p, c_int, c_void_p]),
    "qmoe_decode_fused": (c_int, [c_void_p, c_int64, c_int64, c_int64, c_int64, c_int, c_void_p,
                                  c_void_p, qmoe_weights, qmoe_weights, c_int, c_int, c_int,
                                  c_void_p, c_void_p, c_size_t, c_void_p]),
    "qmoe_decode_scratch_bytes": (c_size_t, [c_int64, c_int64, c_int64, c_int, c_int]),
    "qmoe_decode_status": (c_int, [c_void_p, c_size_t, c_int64, c_int64, c_int64, c_int, c_int,
                                   POINTER(c_int), c_void_p]),
    "qmoe_ragged_mm": (c_int, [c_void_p, c_int64, c_int64, c_int64, c_int64, c_void_p, qmoe_weights, c_int,
                               c_int, c_void_p, c_void_p]),
    "qmoe_decode_fused_noalloc": (c_int, [c_void_p, c_int64, c_int64, c_int64, c_int64, c_int, c_void_p,
                                          c_void_p, qmoe_weights, qmoe_weights, c_int, c_int, c_int,
                                          c_void_p, c_void_p]),
    "qmm_validate_qmoe": (c_int, [c_void_p, c_int64, c_int64, c_int64, c_int64, c_int, c_void_p,
                                  c_void_p, qmoe_weights, qmoe_weights, c_int, c_int, c_int,
                                  c_void_p, c_void_p, c_size_t]),
    "qmm_quantize_linear": (c_int, [c_void_p, c_int, c_int64, qmm_qparams, c_int, c_void_p, c_void_p]),
    "qmm_dequantize_linear": (c_int, [c_void_p, c_int64, qmm_qparams, c_int, c_void_p, c_int, c_void_p]),
    "qmm_fake_quantize": (c_int, [c_void_p, c_int, c_int64, qmm_qparams, c_int, c_void_p, c_void_p]),
    "qmm_qsigmoid": (c_int, [c_void_p, c_int64, qmm_qparams, qmm_qparams, c_int, c_void_p, c_void_p]),
    "qmm_qmul": (c_int, [c_void_p, qmm_qparams, c_void_p, qmm_qparams, c_int64, qmm_qparams, c_int,
                         c_void_p, c_void_p]),
    "qmm_qswiglu": (c_int, [c_void_p, c_void_p, c_int, c_int64, c_int, POINTER(qmm_qparams), c_void_p,
                            c_void_p]),
    "qmm_nbits_dgrad": (c_int, [c_void_p, c_int, c_int64, c_int64, c_int64, c_void_p, c_int, c_int, c_void_p, c_void_p,
                                c_int, c_float, c_void_p, c_int, c_void_p, c_size_t, c_void_p]),
    "qmm_codebook4_dgrad": (c_int, [c_void_p, c_int, c_int64, c_int64, c_int64, c_void_p, c_int, c_void_p, c_void_p,
                                    c_void_p, c_int, c_void_p, c_size_t, c_void_p]),
    "qmm_dgrad_workspace_bytes": (c_size_t, [c_int64, c_int64, c_int64]),
    "qmm_validate_nbits_dgrad": (c_int, [c_void_p, c_int, c_int64, c_int64, c_int64, c_void_p, c_int, c_int, c_void_p,
                                         c_void_p, c_int, c_void_p, c_int, c_void_p, c_size_t]),
    "qmm_validate_codebook4_dgrad": (c_int, [c_void_p, c_int, c_int64, c_int64, c_int64, c_void_p, c_int, c_void_p,
                                             c_void_p, c_void_p, c_int, c_void_p, c_size_t]),
    "qmm_nbits_dgrad_f32": (c_int, [c_void_p, c_int, c_int64, c_int64, c_int64, c_void_p, c_int, c_int, c_void_p,
                                    c_void_p, c_int, c_float, c_void_p, c_int, c_void_p, c_size_t, c_void_p]),
    "qmm_codebook4_dgrad_f32": (c_int, [c_void_p, c_int, c_int64, c_int64, c_int64, c_void_p, c_int, c_void_p,
                                        c_void_p, c_void_p, c_int, c_void_p, c_size_t, c_void_p]),
    "qmm_dgrad_f32_workspace_bytes": (c_size_t, [c_int, c_int64, c_int64, c_int64]),
    "qmm_validate_nbits_dgrad_f32": (c_int, [c_void_p, c_int, c_int64, c_int64, c_int64, c_void_p, c_int, c_int,
                                             c_void_p, c_void_p, c_int, c_void_p, c_int, c_void_p, c_size_t]),
    "qmm_validate_codebook4_dgrad_f32": (c_int, [c_void_p, c_int, c_int64, c_int64, c_int64, c_void_p, c_int,
                                                 c_void_p, c_void_p, c_void_p, c_int, c_void_p, c_size_t]),
    "qmoe_grouped_mm": (c_int, [c_void_p, c_int, c_int64, c_int64, c_int64, c_int64, c_void_p, c_void_p, c_void_p,
                                c_void_p, c_int, c_void_p]),
    "qmoe_grouped_mm_grad": (c_int, [c_void_p, c_void_p, c_int, c_int64, c_int64, c_int64, c_int64, c_void_p,
                                     c_void_p, c_void_p, c_int, c_void_p, c_void_p, c_int, c_void_p]),
    "qmm_validate_grouped_mm": (c_int, [c_void_p, c_int, c_int64, c_int64, c_int64, c_int64, c_void_p, c_void_p,
                                        c_void_p, c_void_p, c_int]),
    "qmm_validate_grouped_mm_grad": (c_int, [c_void_p, c_void_p, c_int, c_int64, c_int64, c_int64, c_int64, c_void_p,
                                             c_void_p, c_void_p, c_int, c_void_p, c_void_p, c_int]),
    "qmm_lora_add": (c_int, [c_void_p, c_int, c_int64, c_int64, c_int64, c_int, c_int64, c_void_p,
                             qmm_lora_weights, c_void_p, c_int, c_void_p, c_int, c_void_p, c_void_p, c_size_t,
                             c_void_p]),
    "qmm_lora_add_workspace_bytes": (c_size_t, [c_int64, c_int64, c_int64, c_int, c_int64]),
    "qmm_lora_grad": (c_int, [c_void_p, c_void_p, c_int, c_int64, c_int64, c_int64, c_int, c_int64, c_void_p,
                              qmm_lora_weights, c_void_p, c_void_p, c_int, c_void_p, c_int, c_void_p, c_void_p,
                              c_int, c_void_p, c_size_t, c_void_p]),
    "qmm_lora_grad_workspace_bytes": (c_size_t, [c_int64, c_int64, c_int64, c_int, c_int64]),
    "qmm_validate_lora_add": (c_int, [c_void_p, c_int, c_int64, c_int64, c_int64, c_int, c_int64, c_void_p,
                                      qmm_lora_weights, c_void_p, c_int, c_void_p, c_int, c_void_p, c_void_p,
                                      c_size_t]),
    "qmm_validate_lora_grad": (c_int, [c_void_p, c_void_p, c_int, c_int64, c_int64, c_int64, c_int, c_int64,
                                       c_void_p, qmm_lora_weights, c_void_p, c_void_p, c_int, c_void_p, c_int,
                                       c_void_p, c_void_p, c_int, c_void_p, c_size_t]),
    "qmm_hbm_read_probe": (c_int, [c_void_p, c_int64, c_void_p, c_int, c_void_p]),
    "qmm_launch_timing_begin": (c_int, [c_int]),
    "qmm_launch_timing_end": (c_int, [c_void_p, c_int, c_void_p]),
    "qmm_set_tuning": (c_int, [c_int, c_int]),
    "qmm_num_candidates": (c_int, [c_int]),
    "qmm_nbits_gemv_matrix_core_form": (c_int, [c_int64, c_int64, c_int64, c_int, c_int]),
    "qmm_tuned_choice": (c_int, [c_int]),
    "qmm_clear_tuning": (None, []),
    "qmm_tuner_pick": (c_int, [POINTER(c_double), c_int, c_int]),
    "qmm_tuner_pick_single_launch": (c_int, [POINTER(c_double), c_int, c_int]),
    "qmm_status_string": (ctypes.c_char_p, [c_int]),
}


def lib():
    """Load libqmm.so once (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: run __graft_entry__.build() first")
        # torch ships its own HIP runtime with the same soname as ROCm's; importing
        # torch first makes libqmm.so bind to that one runtime instead of a second copy
        import torch  # noqa: F401
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name, None)
            if fn is None:  # reported by the export test; calling it raises AttributeError
                continue
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(fn, status):
    if status != 0:
        raise QmmError(fn, status)


# ---------------------------------------------------------------------------
# torch marshalling
# ---------------------------------------------------------------------------

def _torch():
    import torch
    return torch


def dtype_code(t) -> int:
    torch = _torch()
    m = {torch.float32: QMM_F32, torch.float16: QMM_F16, torch.bfloat16: QMM_BF16}
    if t.dtype not in m:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return m[t.dtype]


def torch_dtype(code: int):
    torch = _torch()
    return {QMM_F32: torch.float32, QMM_F16: torch.float16, QMM_BF16: torch.bfloat16}[code]


def _ptr(t):
    return None if t is None else c_void_p(t.data_ptr())


def _stream(stream=None):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return c_void_p(s.cuda_stream)


def _contig(t, name):
    if t is not None and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


# Memory of a call on a given stream comes from that stream's part of the caching allocator: a block
# of the current stream's part may still be in use by work queued there, which the given stream does
# not wait for.

def _new(shape, dtype, like, stream):
    """An output of a call on `stream`, which the caller will use on the current stream: its memory is not
    handed out again before what is queued there by the time it is freed has run."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=like.device)
    t.record_stream(torch.cuda.current_stream(like.device))
    return t


def _temporary(nbytes, like, stream, zeroed=False):
    """Scratch memory that only a call on `stream` uses."""
    torch = _torch()
    make = torch.zeros if zeroed else torch.empty
    if stream is None:
        return make(nbytes, dtype=torch.uint8, device=like.device)
    with torch.cuda.stream(stream):
        return make(nbytes, dtype=torch.uint8, device=like.device)


def nblocks(K, block):
    return (K + block - 1) // block


def qmm_nbits(A, W, scales, K, bits, block, zp=None, zp_kind=QMM_ZP_NONE, uniform_zp=0.0,
              bias=None, out=None, out_dtype=None, workspace=None, stream=None):
    """C[M,N] = A[M,K] . dequant(W)^T (+ bias) through the C ABI."""
    torch = _torch()
    A = _contig(A, "A")
    M = A.shape[0]
    N = W.shape[0]
    ctype = dtype_code(A) if out_dtype is None else dtype_code(torch.empty(0, dtype=out_dtype))
    if out is None:
        out = _new((M, N), torch_dtype(ctype), A, stream)
    ws_bytes = lib().qmm_nbits_workspace_bytes(M, K, N, dtype_code(A))
    if ws_bytes and workspace is None:
        workspace = _temporary(ws_bytes, A, stream)
    st = lib().qmm_nbits(_ptr(A), dtype_code(A), M, K, N, _ptr(W), bits, block, _ptr(scales),
                         _ptr(zp), zp_kind, float(uniform_zp), _ptr(bias), _ptr(out),
                         dtype_code(out), _ptr(workspace),
                         0 if workspace is None else workspace.numel() * workspace.element_size(),
                         _stream(stream))
    _check("qmm_nbits", st)
    return out


def qmm_codebook4(A, W, absmax, codebook, K, block=64, bias=None, out=None, out_dtype=None,
                  workspace=None, stream=None):
    torch = _torch()
    A = _contig(A, "A")
    M = A.shape[0]
    N = W.shape[0]
    ctype = dtype_code(A) if out_dtype is None else dtype_code(torch.empty(0, dtype=out_dtype))
    if out is None:
        out = _new((M, N), torch_dtype(ctype), A, stream)
    ws_bytes = lib().qmm_codebook4_workspace_bytes(M, K, N, dtype_code(A))
    if ws_bytes and workspace is None:
        workspace = _temporary(ws_bytes, A, stream)
    st = lib().qmm_codebook4(_ptr(A), dtype_code(A), M, K, N, _ptr(W), block, _ptr(absmax),
                             _ptr(codebook), _ptr(bias), _ptr(out), dtype_code(out),
                             _ptr(workspace),
                             0 if workspace is None else workspace.numel() * workspace.element_size(),
                             _stream(stream))
    _check("qmm_codebook4", st)
    return out


def _nested(na):
    """na: dict of device tensors codes, table, scales and python offset, group."""
    return qmm_nested_absmax(na["codes"].data_ptr(), na["table"].data_ptr(), na["scales"].data_ptr(),
                             float(na["offset"]), int(na["group"]))


def qmm_dequantize_absmax_nested(na, count, stream=None):
    torch = _torch()
    out = _new(count, torch.float32, na["codes"], stream)
    desc = _nested(na)
    _check("qmm_dequantize_absmax_nested", lib().qmm_dequantize_absmax_nested(ctypes.byref(desc), count, _ptr(out),
                                                                              _stream(stream)))
    return out


def qmm_codebook4_nested(A, W, na, codebook, K, block=64, bias=None, out=None, out_dtype=None, workspace=None,
                         stream=None):
    torch = _torch()
    A = _contig(A, "A")
    M = A.shape[0]
    N = W.shape[0]
    ctype = dtype_code(A) if out_dtype is None else dtype_code(torch.empty(0, dtype=out_dtype))
    if out is None:
        out = _new((M, N), torch_dtype(ctype), A, stream)
    ws_bytes = lib().qmm_codebook4_nested_workspace_bytes(M, K, N, dtype_code(A), block)
    if ws_bytes and workspace is None:
        workspace = _temporary(ws_bytes, A, stream)
    desc = _nested(na)
    st = lib().qmm_codebook4_nested(_ptr(A), dtype_code(A), M, K, N, _ptr(W), block, ctypes.byref(desc),
                                    _ptr(codebook), _ptr(bias), _ptr(out), dtype_code(out), _ptr(workspace),
                                    0 if workspace is None else workspace.numel() * workspace.element_size(),
                                    _stream(stream))
    _check("qmm_codebook4_nested", st)
    return out


def qmm_fp16_uniform_value(zp, scratch=None, stream=None):
    """(is_uniform, value) of an fp16 zero-point tensor (synchronizes the stream)."""
    if scratch is None:
        scratch = _temporary(lib().qmm_uniform_scratch_bytes(), zp, stream)
    flag = c_int(0)
    val = c_float(0.0)
    st = lib().qmm_fp16_uniform_value(_ptr(zp), zp.numel(), _ptr(scratch), scratch.numel(),
                                      ctypes.byref(flag), ctypes.byref(val), _stream(stream))
    _check("qmm_fp16_uniform_value", st)
    return bool(flag.value), float(val.value)


def qmm_dequantize_nbits(W, scales, K, bits, block, zp=None, zp_kind=QMM_ZP_NONE, uniform_zp=0.0,
                         out_dtype=None, stream=None):
    torch = _torch()
    out_dtype = out_dtype or torch.float32
    N = W.shape[0]
    out = _new((N, K), out_dtype, W, stream)
    st = lib().qmm_dequantize_nbits(_ptr(W), bits, block, _ptr(scales), _ptr(zp), zp_kind,
                                    float(uniform_zp), N, K, _ptr(out), dtype_code(out),
                                    _stream(stream))
    _check("qmm_dequantize_nbits", st)
    return out


def qmm_dequantize_codebook4(W, absmax, codebook, K, block=64, out_dtype=None, stream=None):
    torch = _torch()
    out_dtype = out_dtype or torch.float32
    N = W.shape[0]
    out = _new((N, K), out_dtype, W, stream)
    st = lib().qmm_dequantize_codebook4(_ptr(W), block, _ptr(absmax), _ptr(codebook), N, K,
                                        _ptr(out), dtype_code(out), _stream(stream))
    _check("qmm_dequantize_codebook4", st)
    return out


def _qw(d):
    if d is None:
        return qmoe_weights(None, None, None, None)
    return qmoe_weights(d["W"].data_ptr(), d["scales"].data_ptr(),
                        None if d.get("zp") is None else d["zp"].data_ptr(),
                        None if d.get("bias") is None else d["bias"].data_ptr())


def qmoe_decode_scratch_bytes(T, H, I, k, mode=QMOE_FP):
    return lib().qmoe_decode_scratch_bytes(T, H, I, k, mode)


def qmoe_decode_fused(X, expert_ids, expert_w, fc1, fc2, H, I, E, block, mode=QMOE_FP, bits=4,
                      out=None, scratch=None, stream=None):
    """Y[T,H] fp16 = top-k MoE decode (fc1 -> SwiGLU -> fc2) through the C ABI.

    fc1 / fc2: dicts of device tensors {"W", "scales", "zp" (or None), "bias" (or None)}.
    """
    torch = _torch()
    X = _contig(X, "X")
    T = X.shape[0]
    k = expert_ids.shape[1]
    if out is None:
        out = _new((T, H), torch.float16, X, stream)
    sb = lib().qmoe_decode_scratch_bytes(T, H, I, k, mode)
    if scratch is None:
        # zeroed: the single-launch form's sync words must start at zero (calls leave them so)
        scratch = _temporary(max(sb, 1), X, stream, zeroed=True)
    st = lib().qmoe_decode_fused(_ptr(X), T, H, I, E, k, _ptr(expert_ids), _ptr(expert_w), _qw(fc1),
                                 _qw(fc2), bits, block, mode, _ptr(out), _ptr(scratch),
                                 scratch.numel() * scratch.element_size(), _stream(stream))
    _check("qmoe_decode_fused", st)
    return out


def qmoe_ragged_mm(X, row_offsets, w, N, E, block, bits=4, out=None, stream=None):
    """Y[R, N] fp16: rows of X grouped by expert (row_offsets [E+1] int32 on the device),
    each row times its expert's dequantized u4 weights (w: dict W, scales, zp, bias)."""
    torch = _torch()
    X = _contig(X, "X")
    R, K = X.shape
    if out is None:
        out = _new((R, N), torch.float16, X, stream)
    st = lib().qmoe_ragged_mm(_ptr(X), R, K, N, E, _ptr(row_offsets), _qw(w), bits, block, _ptr(out),
                              _stream(stream))
    _check("qmoe_ragged_mm", st)
    return out


QMOE_NOALLOC_SCRATCH_BYTES = 8 << 20


def qmoe_decode_fused_noalloc(X, expert_ids, expert_w, fc1, fc2, H, I, E, block, out, mode=QMOE_FP, bits=4,
                              stream=None):
    """The MoE decode on the library's static scratch: no allocation in the library
    (the caller passes the output)."""
    X = _contig(X, "X")
    T = X.shape[0]
    k = expert_ids.shape[1]
    st = lib().qmoe_decode_fused_noalloc(_ptr(X), T, H, I, E, k, _ptr(expert_ids), _ptr(expert_w), _qw(fc1),
                                         _qw(fc2), bits, block, mode, _ptr(out), _stream(stream))
    _check("qmoe_decode_fused_noalloc", st)
    return out


def qmoe_decode_status(scratch, T, H, I, k, mode=QMOE_FP, stream=None) -> bool:
    """True if a single-launch decode on `scratch` gave up its wait (clears the flag)."""
    flag = c_int(0)
    st = lib().qmoe_decode_status(_ptr(scratch), scratch.numel() * scratch.element_size(), T, H, I, k,
                                  mode, ctypes.byref(flag), _stream(stream))
    _check("qmoe_decode_status", st)
    return bool(flag.value)


# ---------------------------------------------------------------------------
# activation quantization ops
# ---------------------------------------------------------------------------

def _qp(q):
    s, z = q
    return qmm_qparams(float(s), int(z))


def _code_dtype(bits):
    torch = _torch()
    return torch.uint8 if bits == 8 else torch.uint16


def quantize_linear(x, q, bits, out=None, stream=None):
    """uint8 / uint16 codes of x under the per-tensor (scale, zero_point) q."""
    x = _contig(x, "x")
    if out is None:
        out = _new(x.shape, _code_dtype(bits), x, stream)
    _check("qmm_quantize_linear", lib().qmm_quantize_linear(_ptr(x), dtype_code(x), x.numel(), _qp(q), bits,
                                                            _ptr(out), _stream(stream)))
    return out


def dequantize_linear(codes, q, bits, out_dtype=None, out=None, stream=None):
    torch = _torch()
    codes = _contig(codes, "codes")
    if out is None:
        out = _new(codes.shape, out_dtype or torch.float32, codes, stream)
    _check("qmm_dequantize_linear", lib().qmm_dequantize_linear(_ptr(codes), codes.numel(), _qp(q), bits,
                                                                _ptr(out), dtype_code(out), _stream(stream)))
    return out


def fake_quantize(x, q, bits, out=None, stream=None):
    x = _contig(x, "x")
    if out is None:
        out = _new(x.shape, x.dtype, x, stream)
    _check("qmm_fake_quantize", lib().qmm_fake_quantize(_ptr(x), dtype_code(x), x.numel(), _qp(q), bits,
                                                        _ptr(out), _stream(stream)))
    return out


def qsigmoid(codes, q_in, q_out, bits, out=None, stream=None):
    codes = _contig(codes, "codes")
    if out is None:
        out = _new(codes.shape, codes.dtype, codes, stream)
    _check("qmm_qsigmoid", lib().qmm_qsigmoid(_ptr(codes), codes.numel(), _qp(q_in), _qp(q_out), bits, _ptr(out),
                                              _stream(stream)))
    return out


def qmul(a, qa, b, qb, qc, bits, out=None, stream=None):
    a, b = _contig(a, "a"), _contig(b, "b")
    if a.numel() != b.numel():
        raise ValueError("a and b differ in size")
    if out is None:
        out = _new(a.shape, a.dtype, a, stream)
    _check("qmm_qmul", lib().qmm_qmul(_ptr(a), _qp(qa), _ptr(b), _qp(qb), a.numel(), _qp(qc), bits, _ptr(out),
                                      _stream(stream)))
    return out


def qswiglu(gate, up, qparams, bits, out=None, stream=None):
    """Fused quantized SwiGLU chain; qparams: five (scale, zero_point) pairs
    (gate, sigmoid, silu, up, out)."""
    torch = _torch()
    gate, up = _contig(gate, "gate"), _contig(up, "up")
    if gate.numel() != up.numel() or gate.dtype != up.dtype:
        raise ValueError("gate and up differ in size or dtype")
    if out is None:
        out = _new(gate.shape, gate.dtype, gate, stream)
    arr = (qmm_qparams * 5)(*[_qp(q) for q in qparams])
    _check("qmm_qswiglu", lib().qmm_qswiglu(_ptr(gate), _ptr(up), dtype_code(gate), gate.numel(), bits, arr,
                                            _ptr(out), _stream(stream)))
    return out


# ---------------------------------------------------------------------------
# checks of the training and adapter operators' tensors (a decode step makes hundreds of these
# calls, so each check is one attribute read)
# ---------------------------------------------------------------------------

class _Types:
    """torch, its dtypes by element-type code, and the current stream's handle."""

    def __init__(self):
        torch = _torch()
        self.torch = torch
        self.any = {torch.float32: QMM_F32, torch.float16: QMM_F16, torch.bfloat16: QMM_BF16}
        self.half = {torch.float16: QMM_F16, torch.bfloat16: QMM_BF16}
        self.only = {d: {d: c} for d, c in self.any.items()}
        self.f32 = self.only[torch.float32]
        self.i32 = {torch.int32: 0}
        self.u8 = {torch.uint8: 0}
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        self.current = raw or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


_types_cache = None


def _types() -> _Types:
    global _types_cache
    if _types_cache is None:
        _types_cache = _Types()
    return _types_cache


def _expect(t, name, shape, codes, dev):
    """Checks a dense tensor of the given shape on device index `dev`; its element-type code."""
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    code = codes.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be one of {list(codes)}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the device of the call")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return code


def _optional(t, name, shape, codes, dev):
    """_expect of a tensor that may be None: its address (or None) and element-type code."""
    if t is None:
        return None, QMM_F32
    code = _expect(t, name, shape, codes, dev)
    return t.data_ptr(), code


def _device_of(t):
    """Index of the tensor's device, which has to be the current one (kernels launch there)."""
    dev = t.get_device()
    if dev < 0 or dev != _types().torch.cuda.current_device():
        raise ValueError("the tensors must be on the current device (torch.cuda.set_device)")
    return dev


def _handle(stream, dev):
    if stream is None:
        return _types().current(dev)
    if stream.device_index != dev:
        raise ValueError("the stream must be one of the tensors' device")
    return stream.cuda_stream


def _scratch(workspace, need, like, stream):
    """The workspace, allocated here when not given, its address and size."""
    if workspace is None:
        workspace = _temporary(need, like, stream)
        return workspace, workspace.data_ptr(), need
    if not workspace.is_contiguous() or workspace.get_device() != like.get_device():
        raise ValueError("workspace must be contiguous and on the device of the call")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


@functools.lru_cache(maxsize=4096)
def _bytes_of(query, *sizes):
    """Workspace bytes of a shape (a pure function of the sizes)."""
    return max(1, getattr(lib(), query)(*sizes))


# ---------------------------------------------------------------------------
# low-rank adapters
# ---------------------------------------------------------------------------

def _lora_shapes(X, A, B, ids, scale):
    ty = _types()
    if X.dim() != 2 or A.dim() != 3 or B.dim() != 3:
        raise ValueError("rows must be [M, K], A [L, r, K] and B [L, N, r]")
    code = ty.half.get(X.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {X.dtype}")
    dev = _device_of(X)
    M = X.shape[0]
    L, r, K = A.shape
    N = B.shape[1]
    same = ty.only[X.dtype]
    _expect(X, "X", (M, K), same, dev)
    _expect(A, "A", (L, r, K), same, dev)
    _expect(B, "B", (L, N, r), same, dev)
    _expect(ids, "ids", (M,), ty.i32, dev)
    s, _ = _optional(scale, "scale", (L,), ty.f32, dev)
    return ty, dev, code, M, K, N, r, L, qmm_lora_weights(A.data_ptr(), B.data_ptr(), s)


def qmm_lora_add(X, A, B, ids, scale=None, base=None, out=None, out_dtype=None, T=None, workspace=None,
                 stream=None):
    """Y[m] = base[m] + scale[a] * B[a] (A[a] X[m]), a = ids[m] (outside [0, L): Y[m] = base[m]).

    X [M, K], A [L, r, K], B [L, N, r] fp16 or bf16; ids int32 [M]; scale fp32 [L]; base [M, N],
    for instance the fp32 output of qmm_nbits.  T (fp32 [M, r]) receives A[a] X[m] for qmm_lora_grad."""
    ty, dev, code, M, K, N, r, L, w = _lora_shapes(X, A, B, ids, scale)
    base_p, base_t = _optional(base, "base", (M, N), ty.any, dev)
    T_p, _ = _optional(T, "T", (M, r), ty.f32, dev)
    if out is None:
        out = _new((M, N), out_dtype or X.dtype, X, stream)
    out_t = _expect(out, "out", (M, N), ty.any, dev)
    keep, ws, wsb = _scratch(workspace, _bytes_of("qmm_lora_add_workspace_bytes", M, K, N, r, L), X, stream)
    st = lib().qmm_lora_add(X.data_ptr(), code, M, K, N, r, L, ids.data_ptr(), w, base_p, base_t, out.data_ptr(),
                            out_t, T_p, ws, wsb, _handle(stream, dev))
    _check("qmm_lora_add", st)
    return out


def qmm_lora_grad(dY, X, A, B, ids, scale=None, T=None, base=None, dX=None, dA=None, dB=None, dx_dtype=None,
                  grad_dtype=None, need=(True, True, True), workspace=None, stream=None):
    """Gradients (dX, dA, dB) of qmm_lora_add; need: which of the three to compute (others None).

    dX[m] = base[m] + A[a]^T dT[m] with dT[m] = scale[a] B[a]^T dY[m]; dA[a] = sum dT[m] X[m]^T;
    dB[a] = scale[a] sum dY[m] T[m]^T.  T: kept from qmm_lora_add, or None (computed again).
    dX is of dx_dtype (default X's), dA and dB of grad_dtype (default fp32)."""
    ty, dev, code, M, K, N, r, L, w = _lora_shapes(X, A, B, ids, scale)
    _expect(dY, "dY", (M, N), ty.only[X.dtype], dev)
    T_p, _ = _optional(T, "T", (M, r), ty.f32, dev)
    base_p, base_t = _optional(base, "base", (M, K), ty.any, dev)
    if dX is None and need[0]:
        dX = _new((M, K), dx_dtype or X.dtype, X, stream)
    if dA is None and need[1]:
        dA = _new((L, r, K), grad_dtype or ty.torch.float32, X, stream)
    if dB is None and need[2]:
        dB = _new((L, N, r), grad_dtype or ty.torch.float32, X, stream)
    dX_p, dX_t = _optional(dX, "dX", (M, K), ty.any, dev)
    dA_p, dA_t = _optional(dA, "dA", (L, r, K), ty.any, dev)
    dB_p, dB_t = _optional(dB, "dB", (L, N, r), ty.any, dev)
    if dA is not None and dB is not None and dA_t != dB_t:
        raise TypeError("dA and dB differ in dtype")
    keep, ws, wsb = _scratch(workspace, _bytes_of("qmm_lora_grad_workspace_bytes", M, K, N, r, L), X, stream)
    st = lib().qmm_lora_grad(dY.data_ptr(), X.data_ptr(), code, M, K, N, r, L, ids.data_ptr(), w, T_p, base_p, base_t,
                             dX_p, dX_t, dA_p, dB_p, dB_t if dA is None else dA_t, ws, wsb, _handle(stream, dev))
    _check("qmm_lora_grad", st)
    return dX, dA, dB


# ---------------------------------------------------------------------------
# input gradients of low-bit projections
# ---------------------------------------------------------------------------

def _dgrad_shapes(name, dY, W, K, block, bits, out, out_dtype, stream):
    """Checks dY [M, N] and the packed weights W [N, nblk, block * bits / 8]."""
    ty = _types()
    # the format first, as the shapes are computed from it
    if bits not in (2, 3, 4, 8):
        raise QmmError(name, QMM_E_BITS)
    if block not in (16, 32, 64, 128, 256) or (bits == 3 and block == 16):
        raise QmmError(name, QMM_E_BLOCK)
    if dY.dim() != 2:
        raise ValueError("dY must be [M, N]")
    M, N = dY.shape
    dev = _device_of(dY)
    code = _expect(dY, "dY", (M, N), ty.any, dev)
    if W.shape[0] != N or W.numel() != N * nblocks(K, block) * (block * bits // 8):
        raise ValueError(f"W does not hold {N} rows of {K} codes of {bits} bits in blocks of {block}")
    _expect(W, "W", W.shape, ty.u8, dev)
    if out is None:
        out = _new((M, K), out_dtype or dY.dtype, dY, stream)
    return dev, code, M, N, out, _expect(out, "out", (M, K), ty.any, dev)


def _sized(t, name, count, size, dev):
    """Address of a dense tensor of at least `count` elements of `size` bytes on device `dev`."""
    if t.element_size() != size:
        raise TypeError(f"{name} must have elements of {size} bytes, got {t.dtype}")
    if t.numel() < count:
        raise ValueError(f"{name} must hold {count} elements, got {t.numel()}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the device of the call")
    return _contig(t, name).data_ptr()


def _dgrad_workspace(f32, workspace, code, M, K, N, dY, stream):
    if f32:
        need = _bytes_of("qmm_dgrad_f32_workspace_bytes", code, M, K, N)
    else:
        need = _bytes_of("qmm_dgrad_workspace_bytes", M, K, N)
    return _scratch(workspace, need, dY, stream)


def qmm_nbits_dgrad(dY, W, scales, K, bits, block, zp=None, zp_kind=QMM_ZP_NONE, uniform_zp=0.0, out=None,
                    out_dtype=None, workspace=None, stream=None, f32=False):
    """dX[M, K] = dY[M, N] . dequant(W): the input gradient of qmm_nbits, from the same weight buffers.

    f32: dY and the weights enter the products as they are (qmm_nbits_dgrad_f32), not rounded to fp16."""
    name = "qmm_nbits_dgrad_f32" if f32 else "qmm_nbits_dgrad"
    dev, code, M, N, out, out_t = _dgrad_shapes(name, dY, W, K, block, bits, out, out_dtype, stream)
    nblk = nblocks(K, block)
    s_p = _sized(scales, "scales", N * nblk, 2, dev)
    z_p = None
    if zp is not None and zp_kind == QMM_ZP_PACKED:
        z_p = _sized(zp, "zp", N * ((nblk * bits + 7) // 8), 1, dev)
    elif zp is not None and zp_kind == QMM_ZP_F16:
        z_p = _sized(zp, "zp", N * nblk, 2, dev)
    keep, ws, wsb = _dgrad_workspace(f32, workspace, code, M, K, N, dY, stream)
    st = getattr(lib(), name)(dY.data_ptr(), code, M, K, N, W.data_ptr(), bits, block, s_p, z_p, zp_kind,
                              float(uniform_zp), out.data_ptr(), out_t, ws, wsb, _handle(stream, dev))
    _check(name, st)
    return out


def qmm_codebook4_dgrad(dY, W, absmax, codebook, K, block=64, out=None, out_dtype=None, workspace=None, stream=None,
                        f32=False):
    """dX[M, K] = dY[M, N] . (codebook[q] * absmax): the input gradient of qmm_codebook4 (f32: as
    qmm_nbits_dgrad)."""
    name = "qmm_codebook4_dgrad_f32" if f32 else "qmm_codebook4_dgrad"
    dev, code, M, N, out, out_t = _dgrad_shapes(name, dY, W, K, block, 4, out, out_dtype, stream)
    a_p = _sized(absmax, "absmax", N * nblocks(K, block), 4, dev)
    c_p = _sized(codebook, "codebook", 16, 4, dev)
    keep, ws, wsb = _dgrad_workspace(f32, workspace, code, M, K, N, dY, stream)
    st = getattr(lib(), name)(dY.data_ptr(), code, M, K, N, W.data_ptr(), block, a_p, c_p, out.data_ptr(), out_t, ws,
                              wsb, _handle(stream, dev))
    _check(name, st)
    return out


# ---------------------------------------------------------------------------
# ragged products of 16-bit weights
# ---------------------------------------------------------------------------

def _grouped_shapes(X, W, row_offsets):
    ty = _types()
    if X.dim() != 2 or W.dim() != 3:
        raise ValueError("rows must be [R, K] and W [E, N, K]")
    code = ty.half.get(X.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {X.dtype}")
    dev = _device_of(X)
    R = X.shape[0]
    E, N, K = W.shape
    same = ty.only[X.dtype]
    _expect(X, "X", (R, K), same, dev)
    _expect(W, "W", (E, N, K), same, dev)
    _expect(row_offsets, "row_offsets", (E + 1,), ty.i32, dev)
    return ty, dev, code, R, K, N, E


def qmoe_grouped_mm(X, row_offsets, W, bias=None, out=None, out_dtype=None, stream=None):
    """Y[r] = X[r] W[e]^T (+ bias[e]) for the rows row_offsets[e] .. row_offsets[e+1] of expert e.

    X [R, K], W [E, N, K] fp16 or bf16; bias [E, N] of the output's dtype (default X's)."""
    ty, dev, code, R, K, N, E = _grouped_shapes(X, W, row_offsets)
    if out is None:
        out = _new((R, N), out_dtype or X.dtype, X, stream)
    out_t = _expect(out, "out", (R, N), ty.any, dev)
    b_p, _ = _optional(bias, "bias", (E, N), ty.only[out.dtype], dev)
    st = lib().qmoe_grouped_mm(X.data_ptr(), code, R, K, N, E, row_offsets.data_ptr(), W.data_ptr(), b_p,
                               out.data_ptr(), out_t, _handle(stream, dev))
    _check("qmoe_grouped_mm", st)
    return out


def qmoe_grouped_mm_grad(dY, X, row_offsets, W, dX=None, dW=None, dbias=None, dx_dtype=None, dw_dtype=None,
                         need=(True, True), need_dbias=False, stream=None):
    """Gradients (dX, dW, dbias) of qmoe_grouped_mm; need: whether dX and dW are computed.

    dX[r] = dY[r] W[e] of dx_dtype (default X's); dW[e] = sum dY[r]^T X[r] and dbias[e] = sum dY[r]
    over the rows of expert e, of dw_dtype (default X's)."""
    ty, dev, code, R, K, N, E = _grouped_shapes(X, W, row_offsets)
    _expect(dY, "dY", (R, N), ty.only[X.dtype], dev)
    if dX is None and need[0]:
        dX = _new((R, K), dx_dtype or X.dtype, X, stream)
    if dW is None and need[1]:
        dW = _new((E, N, K), dw_dtype or X.dtype, X, stream)
    if dbias is None and need_dbias:
        dbias = _new((E, N), dw_dtype or (X.dtype if dW is None else dW.dtype), X, stream)
    dX_p, dX_t = _optional(dX, "dX", (R, K), ty.any, dev)
    dW_p, dW_t = _optional(dW, "dW", (E, N, K), ty.any, dev)
    db_p, db_t = _optional(dbias, "dbias", (E, N), ty.any, dev)
    if dW is not None and dbias is not None and dW_t != db_t:
        raise TypeError("dW and dbias differ in dtype")
    st = lib().qmoe_grouped_mm_grad(dY.data_ptr(), X.data_ptr(), code, R, K, N, E, row_offsets.data_ptr(),
                                    W.data_ptr(), dX_p, dX_t, dW_p, db_p, db_t if dW is None else dW_t,
                                    _handle(stream, dev))
    _check("qmoe_grouped_mm_grad", st)
    return dX, dW, dbias


def hbm_read_probe(buf, sink, groups, stream=None):
    """Read every byte of `buf` once with 128-bit loads (measurement helper)."""
    _check("qmm_hbm_read_probe", lib().qmm_hbm_read_probe(_ptr(buf), buf.numel() * buf.element_size(), _ptr(sink),
                                                          groups, _stream(stream)))


def launch_timing_begin(n: int):
    """Time the next n kernel launches the library makes from this thread."""
    _check("qmm_launch_timing_begin", lib().qmm_launch_timing_begin(n))


def launch_timing_end(n_max: int = 65536):
    """Stop launch timing; the execution time in us of each timed launch, in order."""
    buf = (c_float * n_max)()
    count = c_int(0)
    _check("qmm_launch_timing_end", lib().qmm_launch_timing_end(buf, n_max, ctypes.byref(count)))
    return [float(buf[i]) for i in range(min(count.value, n_max))]


def set_tuning(mode: int, forced_index: int = 0):
    _check("qmm_set_tuning", lib().qmm_set_tuning(mode, forced_index))


def num_candidates(entry: int) -> int:
    return lib().qmm_num_candidates(entry)


def nbits_gemv_matrix_core_form(M: int, K: int, N: int, bits: int, block: int) -> bool:
    return bool(lib().qmm_nbits_gemv_matrix_core_form(M, K, N, bits, block))


def tuned_choice(entry: int) -> int:
    return lib().qmm_tuned_choice(entry)


def clear_tuning():
    lib().qmm_clear_tuning()


def tuner_pick(times_us, rounds, ncand):
    arr = (c_double * len(times_us))(*times_us)
    return lib().qmm_tuner_pick(arr, rounds, ncand)


def tuner_pick_single_launch(times_us, rounds, ncand):
    arr = (c_double * len(times_us))(*times_us)
    return lib().qmm_tuner_pick_single_launch(arr, rounds, ncand)
