"""Python binding of libhsq's C ABI (include/hsq.h).

Argument marshalling only: every step of the layer runs in the CUDA kernels of
``libhsq.so``.  Tensors are torch CUDA tensors (torch supplies device memory and
streams); their ``data_ptr()`` values are handed to the C functions of the
same names.  There is no CPU fallback: if the library is missing or a call
fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional

import torch

from . import build as _build

GROUP = 64

HSQ_OK = 0
HSQ_ERR_INVALID_ARG = 1
HSQ_ERR_ALIGNMENT = 2
HSQ_ERR_UNSUPPORTED = 3
HSQ_ERR_CUDA = 4
HSQ_ERR_TIMEOUT = 5
HSQ_ERR_SCRATCH_LIMIT = 6
HSQ_ERR_BAD_PAGE = 7
#: Size of the built-in scratch array of hsq_linear_forward_noalloc.
HSQ_NOALLOC_SCRATCH_BYTES = 16 << 20
HSQ_OUT_BF16 = 0
HSQ_OUT_F32 = 1
HSQ_BF16, HSQ_F32, HSQ_E4M3 = 0, 1, 2
HSQ_POS_I32, HSQ_POS_I64, HSQ_POS_F32 = 0, 1, 2
HSQ_ROPE_MAX_AXES = 4
#: Activations of the epilogue, by name (hsq_act).
ACTIVATIONS = {"none": 0, "relu": 1, "gelu_tanh": 2, "gelu_erf": 3, "silu": 4}

#: Every symbol that include/hsq.h declares.
EXPORTED = (
    "hsq_num_groups", "hsq_codes_bytes", "hsq_scales_ld", "hsq_scales_bytes",
    "hsq_workspace_bytes", "hsq_pack_weights", "hsq_quantize_act",
    "hsq_linear_forward", "hsq_status_string", "hsq_get_device_status",
    "hsq_debug_force_timeout", "hsq_linear_forward_noalloc", "hsq_linear_forward_fused", "hsq_fused_form",
    "hsq_weights_e4m3_bytes", "hsq_expand_weights", "hsq_workspace_bytes_pre", "hsq_linear_forward_pre",
    "hsq_workspace_bytes_x", "hsq_linear_forward_x",
    "hsq_lowrank_workspace_bytes", "hsq_lowrank_init",
    "hsq_fp4_codes_bytes", "hsq_fp4_scales_bytes", "hsq_fp4_pack_weights", "hsq_fp4_quantize_act",
    "hsq_fp4_linear_forward",
    "hsq_linear_forward_ep", "hsq_linear_forward_noalloc_ep", "hsq_linear_forward_x_ep", "hsq_linear_forward_fused_ep", "hsq_fp4_linear_forward_ep",
    "hsq_rope", "hsq_kv_append",
)


class HsqError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what} failed: {status_string(status)}")


class _CEpilogue(ctypes.Structure):
    _fields_ = [("act", ctypes.c_int), ("mul", ctypes.c_void_p), ("mul_dtype", ctypes.c_int),
                ("mul_rows", ctypes.c_int), ("mul_ld", ctypes.c_longlong), ("residual", ctypes.c_void_p),
                ("residual_dtype", ctypes.c_int), ("residual_ld", ctypes.c_longlong)]


class _CHeads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_longlong), ("head_stride", ctypes.c_longlong)]


class _CRotation(ctypes.Structure):
    _fields_ = [("freqs", ctypes.c_void_p), ("pair_axis", ctypes.c_char_p), ("pairs", ctypes.c_int),
                ("n_axes", ctypes.c_int), ("interleaved", ctypes.c_int), ("transpose", ctypes.c_int),
                ("scale", ctypes.c_float)]


class _CPositions(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("type", ctypes.c_int), ("rows", ctypes.c_int), ("ld", ctypes.c_longlong)]


class _CPagedCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("dtype", ctypes.c_int), ("pages", ctypes.c_int),
                ("page_size", ctypes.c_int), ("page_stride", ctypes.c_longlong), ("slot_stride", ctypes.c_longlong),
                ("head_stride", ctypes.c_longlong), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)]


class _CSequences(ctypes.Structure):
    _fields_ = [("block_table", ctypes.c_void_p), ("cache_lens", ctypes.c_void_p), ("cu_seqlens", ctypes.c_void_p),
                ("count", ctypes.c_int), ("max_pages", ctypes.c_int), ("table_ld", ctypes.c_longlong)]


_lib: Optional[ctypes.CDLL] = None


def library_path() -> str:
    return _build.LIB_PATH


def load(build_if_missing: bool = True) -> ctypes.CDLL:
    """Load libhsq.so (building it first if it is absent and nvcc is available)."""
    global _lib
    if _lib is not None:
        return _lib
    path = _build.LIB_PATH
    if not os.path.exists(path):
        if not build_if_missing:
            raise RuntimeError(f"libhsq.so not built at {path}")
        _build.build()
    lib = ctypes.CDLL(path)
    c = ctypes
    vp, i, sz = c.c_void_p, c.c_int, c.c_size_t
    lib.hsq_num_groups.argtypes = [i, i]; lib.hsq_num_groups.restype = i
    lib.hsq_codes_bytes.argtypes = [i, i, i]; lib.hsq_codes_bytes.restype = sz
    lib.hsq_scales_ld.argtypes = [i]; lib.hsq_scales_ld.restype = i
    lib.hsq_scales_bytes.argtypes = [i, i, i]; lib.hsq_scales_bytes.restype = sz
    lib.hsq_workspace_bytes.argtypes = [i, i, i, i]; lib.hsq_workspace_bytes.restype = sz
    lib.hsq_pack_weights.argtypes = [vp, vp, vp, vp, i, i, i, i, vp, vp, vp]
    lib.hsq_pack_weights.restype = i
    lib.hsq_quantize_act.argtypes = [vp, vp, vp, i, i, i, i, vp, vp, vp, vp]
    lib.hsq_quantize_act.restype = i
    lib.hsq_linear_forward.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, vp, i, vp, sz, vp]
    lib.hsq_linear_forward.restype = i
    lib.hsq_linear_forward_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, vp, i, vp]
    lib.hsq_linear_forward_fused.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, vp, i, vp]
    lib.hsq_linear_forward_fused.restype = i
    lib.hsq_fused_form.argtypes = [i, i, i, i, i]
    lib.hsq_fused_form.restype = i
    lib.hsq_weights_e4m3_bytes.argtypes = [i, i, i]
    lib.hsq_weights_e4m3_bytes.restype = ctypes.c_size_t
    lib.hsq_expand_weights.argtypes = [vp, i, i, i, vp, vp]
    lib.hsq_expand_weights.restype = i
    lib.hsq_workspace_bytes_pre.argtypes = [i, i, i, i]
    lib.hsq_workspace_bytes_pre.restype = ctypes.c_size_t
    lib.hsq_linear_forward_pre.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, vp, i, vp, ctypes.c_size_t, vp]
    lib.hsq_linear_forward_pre.restype = i
    lib.hsq_workspace_bytes_x.argtypes = [i, i, i, i, i, i]
    lib.hsq_workspace_bytes_x.restype = ctypes.c_size_t
    lib.hsq_linear_forward_x.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, vp, i, vp, ctypes.c_size_t, vp]
    lib.hsq_linear_forward_x.restype = i
    lib.hsq_lowrank_workspace_bytes.argtypes = [i, i, i]; lib.hsq_lowrank_workspace_bytes.restype = sz
    lib.hsq_lowrank_init.argtypes = [vp, vp, i, i, i, i, c.c_ulonglong, vp, vp, vp, sz, vp]
    lib.hsq_lowrank_init.restype = i
    lib.hsq_linear_forward_noalloc.restype = i
    lib.hsq_status_string.argtypes = [i]; lib.hsq_status_string.restype = c.c_char_p
    lib.hsq_get_device_status.argtypes = [vp]; lib.hsq_get_device_status.restype = i
    lib.hsq_debug_force_timeout.argtypes = [i, i]; lib.hsq_debug_force_timeout.restype = None
    lib.hsq_fp4_codes_bytes.argtypes = [i, i]; lib.hsq_fp4_codes_bytes.restype = sz
    lib.hsq_fp4_scales_bytes.argtypes = [i, i]; lib.hsq_fp4_scales_bytes.restype = sz
    lib.hsq_fp4_pack_weights.argtypes = [vp, vp, vp, vp, i, i, i, vp, vp, vp, vp]
    lib.hsq_fp4_pack_weights.restype = i
    lib.hsq_fp4_quantize_act.argtypes = [vp, vp, vp, i, i, i, vp, vp, vp, vp, vp]
    lib.hsq_fp4_quantize_act.restype = i
    lib.hsq_fp4_linear_forward.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, vp, i, vp]
    lib.hsq_fp4_linear_forward.restype = i
    lib.hsq_linear_forward_ep.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, vp, i, vp, vp, sz, vp]
    lib.hsq_linear_forward_ep.restype = i
    lib.hsq_linear_forward_noalloc_ep.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, vp, i, vp, vp]
    lib.hsq_linear_forward_noalloc_ep.restype = i
    lib.hsq_linear_forward_x_ep.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, vp, i, vp, vp, sz, vp]
    lib.hsq_linear_forward_x_ep.restype = i
    lib.hsq_linear_forward_fused_ep.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, vp, i, vp, vp]
    lib.hsq_linear_forward_fused_ep.restype = i
    lib.hsq_fp4_linear_forward_ep.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, vp, i, vp, vp]
    lib.hsq_fp4_linear_forward_ep.restype = i
    lib.hsq_rope.argtypes = [vp, vp, i, i, i, i, vp, vp, vp]
    lib.hsq_rope.restype = i
    lib.hsq_kv_append.argtypes = [vp, vp, vp, vp, i, i, i, i, i, vp, vp, vp, vp, vp]
    lib.hsq_kv_append.restype = i
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().hsq_status_string(int(status)).decode()


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libhsq takes CUDA tensors only")
    if not t.is_contiguous():
        raise ValueError("libhsq takes contiguous tensors only")
    return t.data_ptr()


#: The current stream's handle without a Stream object around it (3 us a call), where torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check(status: int, what: str) -> None:
    if status != HSQ_OK:
        raise HsqError(status, what)


# ---------------------------------------------------------------- sizes
def hsq_num_groups(K: int, group: int = GROUP) -> int:
    return load().hsq_num_groups(K, group)


def hsq_codes_bytes(rows: int, K: int, group: int = GROUP) -> int:
    return load().hsq_codes_bytes(rows, K, group)


def hsq_scales_ld(rows: int) -> int:
    return load().hsq_scales_ld(rows)


def hsq_scales_bytes(rows: int, K: int, group: int = GROUP) -> int:
    return load().hsq_scales_bytes(rows, K, group)


def hsq_workspace_bytes(M: int, N: int, K: int, r: int) -> int:
    return load().hsq_workspace_bytes(M, N, K, r)


# ---------------------------------------------------------------- the three calls
def hsq_pack_weights(W, s, L1, L2, N, K, r, w_codes, w_scales, group=GROUP, stream=None) -> None:
    _check(load().hsq_pack_weights(_ptr(W), _ptr(s), _ptr(L1), _ptr(L2), N, K, r, group,
                                   _ptr(w_codes), _ptr(w_scales), _stream(stream)), "hsq_pack_weights")


def hsq_quantize_act(X, s, L1, M, K, r, x_codes, x_scales, U, group=GROUP, stream=None) -> None:
    _check(load().hsq_quantize_act(_ptr(X), _ptr(s), _ptr(L1), M, K, r, group,
                                   _ptr(x_codes), _ptr(x_scales), _ptr(U), _stream(stream)),
           "hsq_quantize_act")


def hsq_linear_forward(x_codes, x_scales, U, w_codes, w_scales, L2, bias, M, N, K, r, Y,
                       out: int = HSQ_OUT_BF16, workspace=None, ws_bytes: int = 0,
                       group=GROUP, stream=None) -> None:
    _check(load().hsq_linear_forward(_ptr(x_codes), _ptr(x_scales), _ptr(U), _ptr(w_codes),
                                     _ptr(w_scales), _ptr(L2), _ptr(bias), M, N, K, r, group,
                                     _ptr(Y), int(out), _ptr(workspace), int(ws_bytes),
                                     _stream(stream)), "hsq_linear_forward")


def hsq_linear_forward_noalloc(x_codes, x_scales, U, w_codes, w_scales, L2, bias, M, N, K, r, Y,
                               out: int = HSQ_OUT_BF16, group=GROUP, stream=None) -> None:
    """hsq_linear_forward with the library's own scratch array instead of a
    workspace: for callers that must not allocate.  Calls that overlap on the
    GPU share that array and race; the first call on a device must come
    before any stream capture."""
    _check(load().hsq_linear_forward_noalloc(_ptr(x_codes), _ptr(x_scales), _ptr(U), _ptr(w_codes),
                                             _ptr(w_scales), _ptr(L2), _ptr(bias), M, N, K, r, group,
                                             _ptr(Y), int(out), _stream(stream)),
           "hsq_linear_forward_noalloc")


def hsq_weights_e4m3_bytes(N: int, K: int, group: int = GROUP) -> int:
    return int(load().hsq_weights_e4m3_bytes(N, K, group))


def hsq_expand_weights(w_codes, N, K, w_e4m3, group=GROUP, stream=None) -> None:
    _check(load().hsq_expand_weights(_ptr(w_codes), N, K, group, _ptr(w_e4m3), _stream(stream)),
           "hsq_expand_weights")


def hsq_workspace_bytes_pre(M: int, N: int, K: int, r: int) -> int:
    return int(load().hsq_workspace_bytes_pre(M, N, K, r))


def hsq_linear_forward_pre(x_codes, x_scales, U, w_codes, w_scales, w_e4m3, L2, bias, M, N, K, r, Y,
                           out: int = HSQ_OUT_BF16, workspace=None, ws_bytes: int = 0,
                           group=GROUP, stream=None) -> None:
    _check(load().hsq_linear_forward_pre(_ptr(x_codes), _ptr(x_scales), _ptr(U), _ptr(w_codes),
                                         _ptr(w_scales), _ptr(w_e4m3), _ptr(L2), _ptr(bias), M, N, K, r, group,
                                         _ptr(Y), int(out), _ptr(workspace), int(ws_bytes),
                                         _stream(stream)), "hsq_linear_forward_pre")


def hsq_workspace_bytes_x(M: int, N: int, K: int, r: int, group: int = GROUP, with_w_e4m3: bool = True) -> int:
    return int(load().hsq_workspace_bytes_x(M, N, K, r, group, 1 if with_w_e4m3 else 0))


def hsq_linear_forward_x(X, s, L1, w_codes, w_scales, w_e4m3, L2, bias, M, N, K, r, Y,
                         out: int = HSQ_OUT_BF16, workspace=None, ws_bytes: int = 0,
                         group=GROUP, stream=None) -> None:
    _check(load().hsq_linear_forward_x(_ptr(X), _ptr(s), _ptr(L1), _ptr(w_codes), _ptr(w_scales), _ptr(w_e4m3),
                                       _ptr(L2), _ptr(bias), M, N, K, r, group, _ptr(Y), int(out),
                                       _ptr(workspace), int(ws_bytes), _stream(stream)), "hsq_linear_forward_x")


def hsq_linear_forward_fused(X, s, L1, w_codes, w_scales, L2, bias, M, N, K, r, Y,
                             out: int = HSQ_OUT_BF16, group=GROUP, stream=None) -> None:
    """The activation step and the forward in one launch (M <= 4, r in
    {0, 1, 2, 4}); HSQ_ERR_UNSUPPORTED otherwise."""
    _check(load().hsq_linear_forward_fused(_ptr(X), _ptr(s), _ptr(L1), _ptr(w_codes), _ptr(w_scales),
                                           _ptr(L2), _ptr(bias), M, N, K, r, group, _ptr(Y), int(out),
                                           _stream(stream)),
           "hsq_linear_forward_fused")


# ---------------------------------------------------------------- forwards with an epilogue
def _out_dtype(t: torch.Tensor, what: str) -> int:
    if t.dtype == torch.bfloat16:
        return HSQ_OUT_BF16
    if t.dtype == torch.float32:
        return HSQ_OUT_F32
    raise ValueError(f"{what} is bfloat16 or float32, not {t.dtype}")


#: hsq_epilogue as C lays it out.
_EPILOGUE = struct.Struct("@iPiiqPiq")


class Epilogue:
    """What a forward does to its result before it is rounded and written:
    ``act(z) * mul + residual`` (hsq_epilogue).  ``act``: a name of ACTIVATIONS.
    ``mul``: rows of N values, token m takes row ``m // mul_rows``; ``residual``:
    M rows of N values (Y itself adds onto it in place).  Both may be column
    ranges of wider tensors (last dimension dense, row stride a multiple of 8).
    The object keeps the tensors and is reused from call to call; which tensors it
    was made with is fixed, where they live is asked in every call."""

    act = property(lambda self: self._act)
    mul = property(lambda self: self._mul)
    mul_rows = property(lambda self: self._mul_rows)
    residual = property(lambda self: self._residual)

    def __init__(self, act: str = "none", mul: Optional[torch.Tensor] = None, mul_rows: int = 1,
                 residual: Optional[torch.Tensor] = None):
        if act not in ACTIVATIONS:
            raise ValueError(f"unknown activation {act!r} (one of {', '.join(ACTIVATIONS)})")
        self._act, self._mul, self._mul_rows, self._residual = act, mul, int(mul_rows), residual
        self._operand("mul", mul), self._operand("residual", residual)

    @staticmethod
    def _operand(name: str, t: Optional[torch.Tensor]):
        """Address, type and row stride of an operand as it is now."""
        if t is None:
            return 0, 0, 0
        if not t.is_cuda:
            raise ValueError("libhsq takes CUDA tensors only")
        if t.dim() != 2 or t.stride(1) != 1:
            raise ValueError(f"{name} is a matrix with a dense last dimension")
        return t.data_ptr(), _out_dtype(t, name), t.stride(0) if t.shape[0] > 1 else -(-t.shape[1] // 8) * 8

    def _for(self, Y: torch.Tensor, M: int, N: int) -> bytes:
        """The C struct, once the operands' shapes and device are those of Y."""
        mul, residual = self._mul, self._residual
        if mul is not None and (self._mul_rows < 1 or tuple(mul.shape) != (-(-M // self._mul_rows), N)):
            raise ValueError(f"mul has {tuple(mul.shape)} values; {M} tokens at {self._mul_rows} a row, {N} outputs")
        if residual is not None and tuple(residual.shape) != (M, N):
            raise ValueError(f"residual is {tuple(residual.shape)}, Y is {(M, N)}")
        for t in (mul, residual):
            if t is not None and t.get_device() != Y.get_device():
                raise ValueError("the epilogue's operands live on another device than Y")
        p, kind, ld = self._operand("mul", mul)
        # (a call has at most 2^20 tokens: a larger row count means one row)
        return _EPILOGUE.pack(ACTIVATIONS[self._act], p, kind, min(max(self._mul_rows, 0), 1 << 20), ld,
                              *self._operand("residual", residual))


def _ep(epilogue: Optional[Epilogue], Y, M, N, out, *inputs):
    """The epilogue's C struct (None for none), once Y has the shape and type that the
    call writes and the call's tensors live on one device."""
    if tuple(Y.shape) != (M, N) or _out_dtype(Y, "Y") != out:
        raise ValueError(f"Y is {tuple(Y.shape)} {Y.dtype}, the call writes {(M, N)} with out={out}")
    _same_device(Y.get_device(), *inputs)
    return None if epilogue is None else epilogue._for(Y, M, N)


def hsq_linear_forward_ep(x_codes, x_scales, U, w_codes, w_scales, w_e4m3, L2, bias, M, N, K, r, Y,
                          epilogue: Optional[Epilogue], out: int = HSQ_OUT_BF16, workspace=None, ws_bytes: int = 0,
                          group=GROUP, stream=None) -> None:
    """hsq_linear_forward (w_e4m3 None) or hsq_linear_forward_pre with an epilogue."""
    ep = _ep(epilogue, Y, M, N, out, x_codes, x_scales, U, w_codes, w_scales, w_e4m3, L2, bias, workspace)
    _check(_on_device(Y.get_device(), stream, lambda s: load().hsq_linear_forward_ep(
        _ptr(x_codes), _ptr(x_scales), _ptr(U), _ptr(w_codes), _ptr(w_scales), _ptr(w_e4m3), _ptr(L2), _ptr(bias), M, N,
        K, r, group, _ptr(Y), int(out), ep, _ptr(workspace), int(ws_bytes), s)), "hsq_linear_forward_ep")


def hsq_linear_forward_noalloc_ep(x_codes, x_scales, U, w_codes, w_scales, L2, bias, M, N, K, r, Y,
                                  epilogue: Optional[Epilogue], out: int = HSQ_OUT_BF16, group=GROUP,
                                  stream=None) -> None:
    """hsq_linear_forward_noalloc with an epilogue."""
    ep = _ep(epilogue, Y, M, N, out, x_codes, x_scales, U, w_codes, w_scales, L2, bias)
    _check(_on_device(Y.get_device(), stream, lambda s: load().hsq_linear_forward_noalloc_ep(
        _ptr(x_codes), _ptr(x_scales), _ptr(U), _ptr(w_codes), _ptr(w_scales), _ptr(L2), _ptr(bias), M, N, K, r, group,
        _ptr(Y), int(out), ep, s)), "hsq_linear_forward_noalloc_ep")


def hsq_linear_forward_x_ep(X, s, L1, w_codes, w_scales, w_e4m3, L2, bias, M, N, K, r, Y,
                            epilogue: Optional[Epilogue], out: int = HSQ_OUT_BF16, workspace=None, ws_bytes: int = 0,
                            group=GROUP, stream=None) -> None:
    """hsq_linear_forward_x with an epilogue."""
    ep = _ep(epilogue, Y, M, N, out, X, s, L1, w_codes, w_scales, w_e4m3, L2, bias, workspace)
    _check(_on_device(Y.get_device(), stream, lambda st: load().hsq_linear_forward_x_ep(
        _ptr(X), _ptr(s), _ptr(L1), _ptr(w_codes), _ptr(w_scales), _ptr(w_e4m3), _ptr(L2), _ptr(bias), M, N, K, r, group,
        _ptr(Y), int(out), ep, _ptr(workspace), int(ws_bytes), st)), "hsq_linear_forward_x_ep")


def hsq_linear_forward_fused_ep(X, s, L1, w_codes, w_scales, L2, bias, M, N, K, r, Y, epilogue: Optional[Epilogue],
                                out: int = HSQ_OUT_BF16, group=GROUP, stream=None) -> None:
    """hsq_linear_forward_fused with an epilogue."""
    ep = _ep(epilogue, Y, M, N, out, X, s, L1, w_codes, w_scales, L2, bias)
    _check(_on_device(Y.get_device(), stream, lambda st: load().hsq_linear_forward_fused_ep(
        _ptr(X), _ptr(s), _ptr(L1), _ptr(w_codes), _ptr(w_scales), _ptr(L2), _ptr(bias), M, N, K, r, group, _ptr(Y),
        int(out), ep, st)), "hsq_linear_forward_fused_ep")


def hsq_fp4_linear_forward_ep(x_codes, x_sf, x_gs, U, w_codes, w_sf, w_gs, L2, bias, M, N, K, r, Y,
                              epilogue: Optional[Epilogue], out: int = HSQ_OUT_BF16, stream=None) -> None:
    """hsq_fp4_linear_forward with an epilogue."""
    ep = _ep(epilogue, Y, M, N, out, x_codes, x_sf, x_gs, U, w_codes, w_sf, w_gs, L2, bias)
    _check(_on_device(Y.get_device(), stream, lambda s: load().hsq_fp4_linear_forward_ep(
        _ptr(x_codes), _ptr(x_sf), _ptr(x_gs), _ptr(U), _ptr(w_codes), _ptr(w_sf), _ptr(w_gs), _ptr(L2), _ptr(bias), M,
        N, K, r, _ptr(Y), int(out), ep, s)), "hsq_fp4_linear_forward_ep")


# ---------------------------------------------------------------- rotary positions, cache append
_HEAD_DTYPES = {torch.bfloat16: HSQ_BF16, torch.float32: HSQ_F32}
_CACHE_DTYPES = {**_HEAD_DTYPES, torch.float8_e4m3fn: HSQ_E4M3}
_POS_DTYPES = {torch.int32: HSQ_POS_I32, torch.int64: HSQ_POS_I64, torch.float32: HSQ_POS_F32}


_POINTER = struct.Struct("@P")


class Rotation:
    """A rotation of heads by positions (hsq_rotation): ``freqs`` [pairs] fp32,
    ``pair_axes`` the axis of every pair (None: one axis).  The object keeps the
    frequencies and is reused from call to call; what it was made with is fixed (their
    values are read on the GPU by every call, and where they live is asked in each)."""

    freqs = property(lambda self: self._freqs)
    pairs = property(lambda self: self._c.pairs)
    n_axes = property(lambda self: self._n_axes)
    interleaved = property(lambda self: bool(self._c.interleaved))
    transpose = property(lambda self: bool(self._c.transpose))
    scale = property(lambda self: self._c.scale)

    def __init__(self, freqs: torch.Tensor, pair_axes=None, interleaved: bool = False, transpose: bool = False,
                 scale: float = 1.0):
        if not freqs.is_cuda or freqs.dtype != torch.float32 or freqs.dim() != 1 or not freqs.is_contiguous():
            raise ValueError("freqs is a contiguous float32 CUDA vector")
        axes = [0] * freqs.numel() if pair_axes is None else [int(a) for a in pair_axes]
        if len(axes) != freqs.numel() or not axes:
            raise ValueError(f"{freqs.numel()} frequencies and {len(axes)} pair axes")
        if min(axes) < 0 or max(axes) >= HSQ_ROPE_MAX_AXES:
            raise ValueError(f"axes are 0 .. {HSQ_ROPE_MAX_AXES - 1}")
        self._freqs, self._n_axes, self._axes = freqs, max(axes) + 1, bytes(axes)
        self._c = _CRotation(freqs=None, pair_axis=self._axes, pairs=len(axes), n_axes=self._n_axes,
                             interleaved=int(bool(interleaved)), transpose=int(bool(transpose)), scale=float(scale))
        self._rest = bytes(self._c)[ctypes.sizeof(ctypes.c_void_p):]  # (holds the address of self._axes)

    def _struct(self) -> bytes:
        """The C struct, with the frequencies where they are now."""
        f = self._freqs
        if f.numel() != self._c.pairs or f.dtype != torch.float32 or not f.is_contiguous():
            raise ValueError(f"freqs is no longer a contiguous float32 vector of {self._c.pairs}")
        return _POINTER.pack(f.data_ptr()) + self._rest


# The structures of the two calls below, packed as C lays them out: a call of a few
# microseconds does not wait for ctypes to build them.
_HEADS = struct.Struct("@Pqq")
_POSITIONS = struct.Struct("@Piiq")
_PAGED_CACHE = struct.Struct("@PPiiiqqqPP")
_SEQUENCES = struct.Struct("@PPPiiq")


def _heads(t: torch.Tensor, name: str, shape=None) -> bytes:
    if not t.is_cuda:
        raise ValueError("libhsq takes CUDA tensors only")
    strides = t.stride()
    if len(strides) != 3 or (strides[2] != 1 and t.shape[2] > 1):
        raise ValueError(f"{name} is [tokens, heads, head_dim] with a dense last dimension")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} is {tuple(t.shape)}, expected {tuple(shape)}")
    return _HEADS.pack(t.data_ptr(), strides[0], strides[1])


def _positions(p: torch.Tensor, rotation: Rotation) -> bytes:
    if not p.is_cuda:
        raise ValueError("libhsq takes CUDA tensors only")
    kind = _POS_DTYPES.get(p.dtype)
    if kind is None:
        raise ValueError(f"positions are int32, int64 or float32, not {p.dtype}")
    shape, strides = p.shape, p.stride()
    rows, axes = (shape[0], 1) if len(shape) == 1 else (shape[0], shape[1]) if len(shape) == 2 else (0, 0)
    if axes != rotation._n_axes or (axes > 1 and strides[1] != 1):
        raise ValueError(f"positions are [rows, {rotation._n_axes}] with a dense last dimension")
    return _POSITIONS.pack(p.data_ptr(), kind, rows, strides[0] if rows > 1 else axes)


def _same_device(index: int, *tensors) -> None:
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError("the call's tensors live on different devices")


def _on_device(index: int, stream, call):
    """call(stream) with device `index` current; stream None: that device's current stream."""
    if index != torch.cuda.current_device():
        with torch.cuda.device(index):
            return call(_stream(stream))
    return call(_raw_stream(index) if stream is None and _raw_stream is not None else _stream(stream))


def hsq_rope(x: torch.Tensor, y: torch.Tensor, positions: torch.Tensor, rotation: Rotation, stream=None) -> None:
    """y = x rotated by its positions: x and y [tokens, heads, head_dim] (any token
    and head strides; y may be x), positions [rows] or [rows, axes], token t taking
    row t % rows.  With rotation.transpose the gradient of that map."""
    kind = _HEAD_DTYPES.get(x.dtype)
    if kind is None or y.dtype != x.dtype:
        raise ValueError("x and y are both bfloat16 or both float32")
    shape = x.shape
    hx = _heads(x, "x")
    hy = hx if y is x else _heads(y, "y", shape)
    pos, rot = _positions(positions, rotation), rotation._struct()
    index = x.get_device()
    _same_device(index, y, positions, rotation._freqs)
    _check(_on_device(index, stream, lambda s: load().hsq_rope(
        hx, hy, kind, shape[0], shape[1], shape[2], rot, pos, s)), "hsq_rope")


def hsq_kv_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                  block_table: torch.Tensor, cache_lens: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None,
                  rotation: Optional[Rotation] = None, positions: Optional[torch.Tensor] = None,
                  q: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                  k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                  stream=None) -> None:
    """Appends the new tokens' k and v [tokens, kv_heads, head_dim] to the paged
    caches [pages, page_size, kv_heads, head_dim] (any order of pages, slots and
    heads in memory), k rotated, and writes q [tokens, q_heads, head_dim] rotated to
    q_out.  block_table int32 [sequences, max_pages], cache_lens int32
    [sequences], cu_seqlens int32 [sequences + 1] or None for one token per
    sequence.  See include/hsq.h."""
    kind = _HEAD_DTYPES.get(k.dtype)
    if kind is None or v.dtype != k.dtype:
        raise ValueError("k and v are both bfloat16 or both float32")
    shape = k.shape
    hk, hv = _heads(k, "k"), _heads(v, "v", shape)
    T, H, D = shape
    hq = hqo = None
    q_heads = 0
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out go together")
    if q is not None:
        if q.dtype != k.dtype or q_out.dtype != k.dtype:
            raise ValueError("q, q_out and k have one type")
        q_shape = q.shape
        if len(q_shape) != 3 or q_shape[0] != T or q_shape[2] != D or q_shape[1] < 1:
            raise ValueError(f"q is {tuple(q_shape)}, k is {tuple(shape)}")
        hq, hqo = _heads(q, "q"), _heads(q_out, "q_out", q_shape)
        q_heads = q_shape[1]
    cache_kind = _CACHE_DTYPES.get(k_cache.dtype)
    if cache_kind is None or v_cache.dtype != k_cache.dtype:
        raise ValueError("the caches are both bfloat16, float32 or float8_e4m3fn")
    c_shape, c_strides = k_cache.shape, k_cache.stride()
    if len(c_shape) != 4 or c_shape[2:] != shape[1:] or v_cache.shape != c_shape:
        raise ValueError(f"the caches are [pages, page_size, {H}, {D}], both")
    if v_cache.stride() != c_strides or (D > 1 and c_strides[3] != 1):
        raise ValueError("the caches have equal strides and a dense last dimension")
    B = cache_lens.shape[0] if cache_lens.dim() == 1 else -1
    t_shape, t_strides = block_table.shape, block_table.stride()
    if block_table.dtype != torch.int32 or len(t_shape) != 2 or t_shape[0] != B or \
            (t_shape[1] > 1 and t_strides[1] != 1):
        raise ValueError("block_table is int32 [sequences, max_pages], dense in the last dimension")
    if cache_lens.dtype != torch.int32 or not cache_lens.is_contiguous():
        raise ValueError("cache_lens is a contiguous int32 vector")
    cu = 0
    if cu_seqlens is not None:
        if cu_seqlens.dtype != torch.int32 or tuple(cu_seqlens.shape) != (B + 1,) or not cu_seqlens.is_contiguous():
            raise ValueError(f"cu_seqlens is a contiguous int32 [{B + 1}]")
        cu = cu_seqlens.data_ptr()
    scales = [0, 0]
    for i, t in enumerate((k_scale, v_scale)):
        if t is not None:
            if t.dtype != torch.float32 or tuple(t.shape) != (H,) or not t.is_contiguous():
                raise ValueError(f"k_scale and v_scale are float32 [{H}]")
            scales[i] = t.data_ptr()
    rot = pos = None
    index = k.get_device()
    if rotation is not None:
        rot = rotation._struct()
        _same_device(index, rotation._freqs)
        if positions is not None:
            pos = _positions(positions, rotation)
    elif positions is not None:
        raise ValueError("positions without a rotation")
    _same_device(index, v, k_cache, v_cache, block_table, cache_lens, cu_seqlens, positions, q, q_out, k_scale, v_scale)
    cache = _PAGED_CACHE.pack(k_cache.data_ptr(), v_cache.data_ptr(), cache_kind, c_shape[0], c_shape[1], c_strides[0],
                              c_strides[1], c_strides[2], scales[0], scales[1])
    seqs = _SEQUENCES.pack(block_table.data_ptr(), cache_lens.data_ptr(), cu, B, t_shape[1],
                           t_strides[0] if B > 1 else t_shape[1])
    _check(_on_device(index, stream, lambda s: load().hsq_kv_append(
        hk, hv, hq, hqo, kind, T, q_heads, H, D, rot, pos, cache, seqs, s)), "hsq_kv_append")


def _sm_count() -> int:
    if torch.cuda.is_available():
        return torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    return 148


def _a16(v: int) -> int:
    return (v + 15) // 16 * 16


def stream_smem_fits(M: int, N: int, K: int, group: int = GROUP, nsm: Optional[int] = None) -> bool:
    """Whether the weight stream's shared memory fits one block for this shape:
    the restatement, in integer arithmetic, of the limit include/hsq.h gives for
    hsq_linear_forward_fused (no library call, so it can be asked without a GPU).
    T = M rounded up to 1, 2, 4 or 8; RB = rows per block = ceil(N / SMs) rounded
    up to 4; a ring of at least two stages (one if one stage holds all RB rows)
    of rs rows, rs = max(1, max(16384, min(RB Kp/4, budget/2)) // (Kp/2))."""
    nsm = nsm or _sm_count()
    G = -(-K // group)
    Kp = G * group
    T = 1 if M <= 1 else 2 if M <= 2 else 4 if M <= 4 else 8
    RB = (-(-N // nsm) + 3) // 4 * 4
    if RB > 256 or G > 256:  # the block's scales are one copy of at most 256 x 256
        return False
    rowbytes = Kp // 2
    fixed = _a16(G * RB * 4) + _a16(T * Kp) + _a16(G * T * 4) + _a16(T * 16) + _a16(16 * T * 16)
    budget = max(0, 227 * 1024 - fixed - 1024)
    target = max(16384, min(RB * rowbytes // 2, budget // 2))
    rs = min(RB, max(1, target // rowbytes))
    min_stages = 1 if -(-RB // rs) == 1 else 2
    return min_stages * rs * rowbytes <= budget


def _dec16_scratch_bytes(M: int, N: int, K: int, r: int, group: int, nsm: int) -> int:
    """Bytes of the library's array that the decode-tile form of
    hsq_linear_forward_fused uses for this shape (restated from the planner: the
    barrier's 256 bytes, stream-K counters and partials, codes, scales, U
    partials and per-CTA copies of U, each rounded up to 256)."""
    up = lambda v: -(-v // 256) * 256
    G = -(-K // group)
    Kp = G * group
    gps = 4 if group == 64 else 2          # scale groups per pipeline stage
    tiles = -(-N // 128)                   # 128 weight rows x 16 tokens
    S = -(-G // gps)
    waves = -(-tiles // nsm)
    fill = tiles / (waves * nsm)
    total = tiles * S
    if (tiles >= nsm and fill >= 0.9) or total <= nsm or total >= (1 << 30):
        grid = min(tiles, nsm)
    else:
        sl = -(-total // nsm)
        grid = -(-total // sl)
    counters = up(tiles * 4 * 4)
    partials = grid * 2 * 16 * 128 * 4
    ldx = (M + 3) // 4 * 4
    rr = max(r, 1)
    nchk = -(-Kp // 256)
    off = 256
    for b in (counters, partials, M * (Kp // 2), G * ldx * 4, M * nchk * rr * 4, grid * M * rr * 4):
        off = up(off + b)
    return off


FUSED_SCRATCH_BYTES = 8 << 20


def fused_supported(M: int, K: int, r: int, group: int = GROUP, N: int = 8, nsm: Optional[int] = None) -> bool:
    """Whether hsq_linear_forward_fused takes this shape (the limits stated in
    include/hsq.h, restated without a library call so it can be asked without a
    GPU): the weight stream for M <= 4, r in {0, 1, 2, 4} and a block's shared
    memory, else the decode tiles for M <= 16, r <= 32 and the library's array."""
    if M < 1 or M > 16 or r < 0 or r > 32 or group not in (64, 128) or K % 8 or N % 8:
        return False
    nsm = nsm or _sm_count()
    if M <= 4 and r in (0, 1, 2, 4) and stream_smem_fits(M, N, K, group, nsm):
        return True
    return _dec16_scratch_bytes(M, N, K, r, group, nsm) <= FUSED_SCRATCH_BYTES


def hsq_fused_form(M: int, N: int, K: int, r: int, group: int = GROUP) -> int:
    return int(load().hsq_fused_form(M, N, K, r, group))


def hsq_lowrank_workspace_bytes(N: int, K: int, r: int) -> int:
    return int(load().hsq_lowrank_workspace_bytes(N, K, r))


def lowrank_init(W: torch.Tensor, s: torch.Tensor, r: int, iters: int = 8, seed: int = 0, stream=None):
    """Plain truncated-SVD L1 [K, r], L2 [r, N] (bf16) of W diag(s) on the GPU
    (pack-time helper; see hsq_lowrank_init)."""
    N, K = W.shape
    ws = torch.empty(max(1, hsq_lowrank_workspace_bytes(N, K, r)), dtype=torch.uint8, device=W.device)
    L1 = torch.empty((K, r), dtype=torch.bfloat16, device=W.device)
    L2 = torch.empty((r, N), dtype=torch.bfloat16, device=W.device)
    _check(load().hsq_lowrank_init(_ptr(W), _ptr(s), N, K, r, iters, int(seed) & ((1 << 64) - 1), _ptr(L1),
                                   _ptr(L2), _ptr(ws), ws.numel(), _stream(stream)),
           "hsq_lowrank_init")
    return L1, L2


def hsq_get_device_status(stream=None) -> int:
    return load().hsq_get_device_status(_stream(stream))


def hsq_debug_force_timeout(flags: int, limit_ms: int) -> None:
    load().hsq_debug_force_timeout(int(flags), int(limit_ms))


# ---------------------------------------------------------------- buffers
def alloc_codes(rows: int, K: int, device, group: int = GROUP) -> torch.Tensor:
    Kp = hsq_num_groups(K, group) * group
    return torch.empty((rows, Kp // 2), dtype=torch.uint8, device=device)


def alloc_scales(rows: int, K: int, device, group: int = GROUP) -> torch.Tensor:
    return torch.empty((hsq_num_groups(K, group), hsq_scales_ld(rows)), dtype=torch.float32, device=device)


class PackedLinear:
    """A packed layer: INT4 residual codes and scales plus the low-rank pair,
    the smoothing vector and the bias, all resident on one device."""

    def __init__(self, W, s, L1, L2, bias=None, stream=None, group: int = GROUP):
        N, K = W.shape
        r = 0 if L1 is None else int(L1.shape[1])
        dev = W.device
        self.N, self.K, self.r, self.group = N, K, r, group
        self.s = s.contiguous()
        self.L1 = None if r == 0 else L1.contiguous()
        self.L2 = None if r == 0 else L2.contiguous()
        self.bias = None if bias is None else bias.contiguous()
        self.w_codes = alloc_codes(N, K, dev, group)
        self.w_scales = alloc_scales(N, K, dev, group)
        self.w_e4m3 = None  # the weights' expanded copy, once expand() has run
        hsq_pack_weights(W.contiguous(), self.s, self.L1, self.L2, N, K, r,
                         self.w_codes, self.w_scales, group=group, stream=stream)

    def expand(self, stream=None) -> None:
        """Keep the weights' E4M3-expanded copy (hsq_expand_weights): forwards
        with many tokens then skip re-expanding the weights on every call."""
        if self.w_e4m3 is None:
            self.w_e4m3 = torch.empty(hsq_weights_e4m3_bytes(self.N, self.K, self.group), dtype=torch.uint8,
                                      device=self.w_codes.device)
            hsq_expand_weights(self.w_codes, self.N, self.K, self.w_e4m3, group=self.group, stream=stream)

    def workspace_x(self, M: int) -> torch.Tensor:
        """Workspace of forward_x for M tokens."""
        n = hsq_workspace_bytes_x(M, self.N, self.K, self.r, self.group, self.w_e4m3 is not None)
        return torch.zeros(max(n, 16), dtype=torch.uint8, device=self.w_codes.device)

    def workspace(self, M: int) -> Optional[torch.Tensor]:
        n = (hsq_workspace_bytes(M, self.N, self.K, self.r) if self.w_e4m3 is None
             else hsq_workspace_bytes_pre(M, self.N, self.K, self.r))
        if n == 0:
            return None
        return torch.zeros(n, dtype=torch.uint8, device=self.w_codes.device)


class ActBuffers:
    """Per-forward buffers of the activation step for M tokens."""

    def __init__(self, M: int, K: int, r: int, device, group: int = GROUP):
        self.M, self.K, self.r, self.group = M, K, r, group
        self.x_codes = alloc_codes(M, K, device, group)
        self.x_scales = alloc_scales(M, K, device, group)
        self.U = torch.empty((M, r), dtype=torch.float32, device=device) if r > 0 else None


def forward_fused(layer: PackedLinear, X: torch.Tensor, Y: torch.Tensor, out: int = HSQ_OUT_BF16,
                  stream=None, epilogue: Optional[Epilogue] = None) -> torch.Tensor:
    """One forward of the layer in a single launch (decode sizes, see
    hsq_linear_forward_fused), with an epilogue where one is given."""
    if epilogue is not None:
        hsq_linear_forward_fused_ep(X, layer.s, layer.L1, layer.w_codes, layer.w_scales, layer.L2, layer.bias,
                                    X.shape[0], layer.N, layer.K, layer.r, Y, epilogue, out=out, group=layer.group,
                                    stream=stream)
        return Y
    hsq_linear_forward_fused(X, layer.s, layer.L1, layer.w_codes, layer.w_scales, layer.L2, layer.bias,
                             X.shape[0], layer.N, layer.K, layer.r, Y, out=out, group=layer.group,
                             stream=stream)
    return Y


def forward_x(layer: PackedLinear, X: torch.Tensor, Y: torch.Tensor, workspace: torch.Tensor,
              out: int = HSQ_OUT_BF16, stream=None, epilogue: Optional[Epilogue] = None) -> torch.Tensor:
    """The activation step and the forward in one call (hsq_linear_forward_x), with
    an epilogue where one is given; `workspace` of at least layer.workspace_x(M)
    bytes."""
    M = X.shape[0]
    if epilogue is not None:
        hsq_linear_forward_x_ep(X, layer.s, layer.L1, layer.w_codes, layer.w_scales, layer.w_e4m3, layer.L2,
                                layer.bias, M, layer.N, layer.K, layer.r, Y, epilogue, out=out, workspace=workspace,
                                ws_bytes=workspace.numel(), group=layer.group, stream=stream)
        return Y
    hsq_linear_forward_x(X, layer.s, layer.L1, layer.w_codes, layer.w_scales, layer.w_e4m3, layer.L2, layer.bias,
                         M, layer.N, layer.K, layer.r, Y, out=out, workspace=workspace, ws_bytes=workspace.numel(),
                         group=layer.group, stream=stream)
    return Y


def forward(layer: PackedLinear, X: torch.Tensor, act: ActBuffers, Y: torch.Tensor,
            workspace: Optional[torch.Tensor] = None, out: int = HSQ_OUT_BF16, stream=None,
            epilogue: Optional[Epilogue] = None) -> torch.Tensor:
    """One forward of the layer: the activation step, then the GEMM + epilogue
    (U L2 + bias, and where one is given act, mul and residual)."""
    M = X.shape[0]
    if act.group != layer.group:
        raise ValueError("activation buffers and packed layer use different group sizes")
    ws_bytes = 0 if workspace is None else workspace.numel()
    if epilogue is not None:
        _ep(epilogue, Y, M, layer.N, out, X, layer.s, layer.L1, act.x_codes, act.x_scales, act.U)

        def both(st):  # on the tensors' device
            hsq_quantize_act(X, layer.s, layer.L1, M, layer.K, layer.r, act.x_codes, act.x_scales, act.U,
                             group=layer.group, stream=st)
            hsq_linear_forward_ep(act.x_codes, act.x_scales, act.U, layer.w_codes, layer.w_scales, layer.w_e4m3,
                                  layer.L2, layer.bias, M, layer.N, layer.K, layer.r, Y, epilogue, out=out,
                                  workspace=workspace, ws_bytes=ws_bytes, group=layer.group, stream=st)

        _on_device(Y.get_device(), stream, both)
        return Y
    hsq_quantize_act(X, layer.s, layer.L1, M, layer.K, layer.r, act.x_codes, act.x_scales, act.U,
                     group=layer.group, stream=stream)
    if layer.w_e4m3 is not None:
        hsq_linear_forward_pre(act.x_codes, act.x_scales, act.U, layer.w_codes, layer.w_scales, layer.w_e4m3,
                               layer.L2, layer.bias, M, layer.N, layer.K, layer.r, Y, out=out, workspace=workspace,
                               ws_bytes=ws_bytes, group=layer.group, stream=stream)
    else:
        hsq_linear_forward(act.x_codes, act.x_scales, act.U, layer.w_codes, layer.w_scales, layer.L2,
                           layer.bias, M, layer.N, layer.K, layer.r, Y, out=out, workspace=workspace,
                           ws_bytes=ws_bytes, group=layer.group, stream=stream)
    return Y


# ---------------------------------------------------------------- NVFP4 variant
def hsq_fp4_codes_bytes(rows: int, K: int) -> int:
    return int(load().hsq_fp4_codes_bytes(rows, K))


def hsq_fp4_scales_bytes(rows: int, K: int) -> int:
    return int(load().hsq_fp4_scales_bytes(rows, K))


def hsq_fp4_pack_weights(W, s, L1, L2, N, K, r, w_codes, w_sf, w_gs, stream=None) -> None:
    _check(load().hsq_fp4_pack_weights(_ptr(W), _ptr(s), _ptr(L1), _ptr(L2), N, K, r, _ptr(w_codes),
                                       _ptr(w_sf), _ptr(w_gs), _stream(stream)), "hsq_fp4_pack_weights")


def hsq_fp4_quantize_act(X, s, L1, M, K, r, x_codes, x_sf, x_gs, U, stream=None) -> None:
    _check(load().hsq_fp4_quantize_act(_ptr(X), _ptr(s), _ptr(L1), M, K, r, _ptr(x_codes), _ptr(x_sf),
                                       _ptr(x_gs), _ptr(U), _stream(stream)), "hsq_fp4_quantize_act")


def hsq_fp4_linear_forward(x_codes, x_sf, x_gs, U, w_codes, w_sf, w_gs, L2, bias, M, N, K, r, Y,
                           out: int = HSQ_OUT_BF16, stream=None) -> None:
    _check(load().hsq_fp4_linear_forward(_ptr(x_codes), _ptr(x_sf), _ptr(x_gs), _ptr(U), _ptr(w_codes),
                                         _ptr(w_sf), _ptr(w_gs), _ptr(L2), _ptr(bias), M, N, K, r, _ptr(Y),
                                         int(out), _stream(stream)), "hsq_fp4_linear_forward")


def _fp4_kq(K: int) -> int:
    return -(-K // 64) * 64


class Fp4Linear:
    """A layer packed in the NVFP4 variant: E2M1 residual codes, E4M3 block
    scales and the tensor scale, plus the low-rank pair, smoothing and bias."""

    def __init__(self, W, s, L1, L2, bias=None, stream=None):
        N, K = W.shape
        r = 0 if L1 is None else int(L1.shape[1])
        dev = W.device
        self.N, self.K, self.r = N, K, r
        self.s = s.contiguous()
        self.L1 = None if r == 0 else L1.contiguous()
        self.L2 = None if r == 0 else L2.contiguous()
        self.bias = None if bias is None else bias.contiguous()
        self.w_codes = torch.empty((N, _fp4_kq(K) // 2), dtype=torch.uint8, device=dev)
        self.w_sf = torch.empty(hsq_fp4_scales_bytes(N, K), dtype=torch.uint8, device=dev)
        self.w_gs = torch.empty(4, dtype=torch.float32, device=dev)
        hsq_fp4_pack_weights(W.contiguous(), self.s, self.L1, self.L2, N, K, r, self.w_codes, self.w_sf,
                             self.w_gs, stream=stream)

    def workspace(self, M: int) -> None:
        """The NVFP4 forward needs no workspace."""
        return None


class Fp4ActBuffers:
    """Per-forward buffers of the NVFP4 activation step for M tokens."""

    def __init__(self, M: int, K: int, r: int, device):
        self.M, self.K, self.r = M, K, r
        self.x_codes = torch.empty((M, _fp4_kq(K) // 2), dtype=torch.uint8, device=device)
        self.x_sf = torch.empty(hsq_fp4_scales_bytes(M, K), dtype=torch.uint8, device=device)
        self.x_gs = torch.empty(4, dtype=torch.float32, device=device)
        self.U = torch.empty((M, r), dtype=torch.float32, device=device) if r > 0 else None


def fp4_forward(layer: Fp4Linear, X: torch.Tensor, act: Fp4ActBuffers, Y: torch.Tensor,
                out: int = HSQ_OUT_BF16, stream=None, epilogue: Optional[Epilogue] = None) -> torch.Tensor:
    """One NVFP4 forward: the activation step, then the block-scaled GEMM + epilogue
    (U L2 + bias, and where one is given act, mul and residual)."""
    M = X.shape[0]
    if epilogue is not None:
        _ep(epilogue, Y, M, layer.N, out, X, layer.s, layer.L1, act.x_codes, act.x_sf, act.x_gs, act.U)

        def both(st):  # on the tensors' device
            hsq_fp4_quantize_act(X, layer.s, layer.L1, M, layer.K, layer.r, act.x_codes, act.x_sf, act.x_gs, act.U,
                                 stream=st)
            hsq_fp4_linear_forward_ep(act.x_codes, act.x_sf, act.x_gs, act.U, layer.w_codes, layer.w_sf, layer.w_gs,
                                      layer.L2, layer.bias, M, layer.N, layer.K, layer.r, Y, epilogue, out=out, stream=st)

        _on_device(Y.get_device(), stream, both)
        return Y
    hsq_fp4_quantize_act(X, layer.s, layer.L1, M, layer.K, layer.r, act.x_codes, act.x_sf, act.x_gs, act.U,
                         stream=stream)
    hsq_fp4_linear_forward(act.x_codes, act.x_sf, act.x_gs, act.U, layer.w_codes, layer.w_sf, layer.w_gs,
                           layer.L2, layer.bias, M, layer.N, layer.K, layer.r, Y, out=out, stream=stream)
    return Y
