"""ctypes binding of libswimba.so (include/swimba.h): argument marshalling only.

Every function named ``swimba_*`` here calls the C function of the same name with device pointers
taken from torch tensors (``tensor.data_ptr()``) and the current torch CUDA stream unless one is
given. Every step of the layer runs in the library's CUDA kernels; there is no Python or CPU
compute path. The linear attention and block norm calls answer SWIMBA_ERR_INVALID_ARG where a tensor's
type, size, layout or device is not what the call's dims say; a workspace counts for what it holds. Importing this module fails loudly when the library has not been built.
"""
from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libswimba.so")
if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -m parameter_space_moe_swimba_b200.build` "
        "(nvcc, sm_100a)"
    )
_lib = ctypes.CDLL(LIB_PATH)

import torch  # noqa: E402  (after the library check so a missing build is reported first)

SWIMBA_F32 = 0
SWIMBA_BF16 = 1
(SWIMBA_OP_ROUTE, SWIMBA_OP_PROJ, SWIMBA_OP_SCAN, SWIMBA_OP_STEP, SWIMBA_OP_LAYER, SWIMBA_OP_SUMMARY,
 SWIMBA_OP_SEPARATE, SWIMBA_OP_SCAN_BWD, SWIMBA_OP_PROJ_BWD, SWIMBA_OP_ROUTE_BWD) = range(10)
SWIMBA_OP_LINATTN_FWD, SWIMBA_OP_LINATTN_BWD = 10, 11

STATUS = {
    0: "SWIMBA_OK",
    1: "SWIMBA_ERR_INVALID_ARG",
    2: "SWIMBA_ERR_UNSUPPORTED",
    3: "SWIMBA_ERR_ALIGN",
    4: "SWIMBA_ERR_WORKSPACE",
    5: "SWIMBA_ERR_CUDA",
    6: "SWIMBA_ERR_TIMEOUT",
}

# Every symbol include/swimba.h declares.
EXPORTED = [
    "swimba_workspace_size",
    "swimba_route",
    "swimba_mixed_proj",
    "swimba_scan_fwd",
    "swimba_scan_fwd_zoh",
    "swimba_scan_fwd_noalloc",
    "swimba_scan_fwd_noalloc_status",
    "swimba_scan_fwd_noalloc_status_block",
    "swimba_scan_summary",
    "swimba_scan_chain",
    "swimba_scan_bwd",
    "swimba_proj_bwd",
    "swimba_route_bwd",
    "swimba_ssd_scan",
    "swimba_separate_proj",
    "swimba_separate_scan",
    "swimba_step",
    "swimba_get_device_status",
    "swimba_check_wait_timeout",
    "swimba_status_string",
    "swimba_kernel_launches",
    "swimba_last_error_string",
    "swimba_conv1d_fwd",
    "swimba_conv1d_step",
    "swimba_block_gemm",
    "swimba_block_workspace_size",
    "swimba_block_fwd",
    "swimba_block_step",
    "swimba_linattn_workspace_size",
    "swimba_linattn_fwd",
    "swimba_linattn_step",
    "swimba_linattn_bwd",
    "swimba_block_norm_fwd",
    "swimba_block_norm_workspace_size",
    "swimba_block_norm_bwd",
]


class swimba_dims(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int64),
        ("seqlen", ctypes.c_int64),
        ("d_inner", ctypes.c_int32),
        ("d_state", ctypes.c_int32),
        ("dt_rank", ctypes.c_int32),
        ("n_experts", ctypes.c_int32),
        ("top_k", ctypes.c_int32),
        ("io_dtype", ctypes.c_int32),
        ("w_dtype", ctypes.c_int32),
    ]


class swimba_ssd_dims(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int64),
        ("seqlen", ctypes.c_int64),
        ("n_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("d_state", ctypes.c_int32),
        ("top_k", ctypes.c_int32),
    ]


class swimba_linattn_dims(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int64),
        ("seqlen", ctypes.c_int64),
        ("n_heads", ctypes.c_int32),
        ("n_kv_heads", ctypes.c_int32),
        ("d_k", ctypes.c_int32),
        ("d_v", ctypes.c_int32),
        ("q_stride", ctypes.c_int64),
        ("k_stride", ctypes.c_int64),
        ("v_stride", ctypes.c_int64),
        ("io_dtype", ctypes.c_int32),
        ("scale", ctypes.c_float),
    ]


class swimba_norm_dims(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int64),
        ("width", ctypes.c_int32),
        ("groups", ctypes.c_int32),
        ("io_dtype", ctypes.c_int32),
        ("res_dtype", ctypes.c_int32),
        ("gate_last", ctypes.c_int32),
        ("eps", ctypes.c_float),
        ("res_scale", ctypes.c_float),
        ("out_scale", ctypes.c_float),
    ]


class swimba_weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("W_r", "W_x", "W_dt", "b_dt", "A", "D_skip")]


class swimba_block_dims(ctypes.Structure):
    _fields_ = [("layer", swimba_dims), ("d_model", ctypes.c_int32), ("d_conv", ctypes.c_int32)]


class swimba_block_weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("W_in", "conv_w", "conv_b", "W_out")] + [("layer", swimba_weights)]


_P = ctypes.c_void_p
_lib.swimba_workspace_size.argtypes = [ctypes.POINTER(swimba_dims), ctypes.c_int]
_lib.swimba_workspace_size.restype = ctypes.c_size_t
_lib.swimba_route.argtypes = [ctypes.POINTER(swimba_dims), _P, _P, _P, _P, _P]
_lib.swimba_route.restype = ctypes.c_int
_lib.swimba_mixed_proj.argtypes = [ctypes.POINTER(swimba_dims), _P, _P, _P, ctypes.POINTER(swimba_weights), _P, _P,
                                   _P, _P, ctypes.c_size_t, _P]
_lib.swimba_mixed_proj.restype = ctypes.c_int
_lib.swimba_scan_fwd.argtypes = [ctypes.POINTER(swimba_dims), _P, _P, _P, _P, _P, _P, _P,
                                 ctypes.POINTER(swimba_weights), _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
_lib.swimba_scan_fwd.restype = ctypes.c_int
_lib.swimba_scan_fwd_zoh.argtypes = _lib.swimba_scan_fwd.argtypes
_lib.swimba_scan_fwd_zoh.restype = ctypes.c_int
_lib.swimba_scan_fwd_noalloc.argtypes = [ctypes.POINTER(swimba_dims), _P, _P, _P, _P, _P, _P, _P,
                                         ctypes.POINTER(swimba_weights), _P, _P, _P, _P, _P]
_lib.swimba_scan_fwd_noalloc.restype = ctypes.c_int
_lib.swimba_scan_fwd_noalloc_status.argtypes = [_P]
_lib.swimba_scan_fwd_noalloc_status.restype = ctypes.c_int
_lib.swimba_scan_fwd_noalloc_status_block.argtypes = []
_lib.swimba_scan_fwd_noalloc_status_block.restype = ctypes.c_void_p
_lib.swimba_scan_summary.argtypes = [ctypes.POINTER(swimba_dims), _P, _P, _P, _P, _P, ctypes.POINTER(swimba_weights),
                                     _P, _P, _P, ctypes.c_size_t, _P]
_lib.swimba_scan_summary.restype = ctypes.c_int
_lib.swimba_scan_chain.argtypes = [ctypes.POINTER(swimba_dims), ctypes.c_int32, _P, _P, _P, _P, _P]
_lib.swimba_scan_chain.restype = ctypes.c_int
_lib.swimba_scan_bwd.argtypes = [ctypes.POINTER(swimba_dims)] + [_P] * 7 + [ctypes.POINTER(swimba_weights)] + \
    [_P] * 11 + [_P, ctypes.c_size_t, _P]
_lib.swimba_scan_bwd.restype = ctypes.c_int
_lib.swimba_proj_bwd.argtypes = [ctypes.POINTER(swimba_dims), _P, _P, _P, ctypes.POINTER(swimba_weights)] + \
    [_P] * 5 + [ctypes.c_int32] + [_P] * 5 + [ctypes.c_size_t, _P]
_lib.swimba_proj_bwd.restype = ctypes.c_int
_lib.swimba_route_bwd.argtypes = [ctypes.POINTER(swimba_dims)] + [_P] * 7 + [ctypes.c_int32, _P, _P, ctypes.c_size_t, _P]
_lib.swimba_route_bwd.restype = ctypes.c_int
_lib.swimba_ssd_scan.argtypes = [ctypes.POINTER(swimba_ssd_dims)] + [_P] * 10 + [_P, ctypes.c_size_t, _P]
_lib.swimba_ssd_scan.restype = ctypes.c_int
_lib.swimba_separate_proj.argtypes = [ctypes.POINTER(swimba_dims), _P, _P, _P, ctypes.POINTER(swimba_weights), _P,
                                      _P, _P, _P]
_lib.swimba_separate_proj.restype = ctypes.c_int
_lib.swimba_separate_scan.argtypes = [ctypes.POINTER(swimba_dims), _P, _P, _P, _P, _P, _P, _P,
                                      ctypes.POINTER(swimba_weights), _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
_lib.swimba_separate_scan.restype = ctypes.c_int
_lib.swimba_step.argtypes = [ctypes.POINTER(swimba_dims), _P, _P, _P, _P, _P, _P, _P,
                             ctypes.POINTER(swimba_weights), _P, _P, _P]
_lib.swimba_step.restype = ctypes.c_int
_lib.swimba_get_device_status.argtypes = [_P, _P]
_lib.swimba_get_device_status.restype = ctypes.c_int
_lib.swimba_check_wait_timeout.argtypes = [_P, ctypes.c_size_t, ctypes.c_uint64, _P]
_lib.swimba_check_wait_timeout.restype = ctypes.c_int
_lib.swimba_status_string.argtypes = [ctypes.c_int]
_lib.swimba_status_string.restype = ctypes.c_char_p
_lib.swimba_last_error_string.argtypes = []
_lib.swimba_last_error_string.restype = ctypes.c_char_p
_lib.swimba_kernel_launches.argtypes = []
_lib.swimba_kernel_launches.restype = ctypes.c_uint64
_lib.swimba_conv1d_fwd.argtypes = [ctypes.POINTER(swimba_dims), ctypes.c_int32, _P, _P, _P, _P, _P, _P, _P]
_lib.swimba_conv1d_fwd.restype = ctypes.c_int
_lib.swimba_conv1d_step.argtypes = [ctypes.POINTER(swimba_dims), ctypes.c_int32, _P, _P, _P, _P, _P, _P]
_lib.swimba_conv1d_step.restype = ctypes.c_int
_I = ctypes.c_int32
_lib.swimba_block_gemm.argtypes = [_I, _I, _I, _I, _P, _I, _P, _I, _P, _I, _P, _I, _I, _P, _I, _P, ctypes.c_size_t, _P]
_lib.swimba_block_gemm.restype = ctypes.c_int
_lib.swimba_block_workspace_size.argtypes = [ctypes.POINTER(swimba_block_dims)]
_lib.swimba_block_workspace_size.restype = ctypes.c_size_t
_lib.swimba_block_fwd.argtypes = [ctypes.POINTER(swimba_block_dims), _P, ctypes.POINTER(swimba_block_weights), _P, _P,
                                  _P, _P, _P, _P, ctypes.c_size_t, _P]
_lib.swimba_block_fwd.restype = ctypes.c_int
_lib.swimba_block_step.argtypes = [ctypes.POINTER(swimba_block_dims), _P, ctypes.POINTER(swimba_block_weights), _P,
                                   _P, _P, _P, ctypes.c_size_t, _P]
_lib.swimba_block_step.restype = ctypes.c_int

_LD, _ND = ctypes.POINTER(swimba_linattn_dims), ctypes.POINTER(swimba_norm_dims)
_lib.swimba_linattn_workspace_size.argtypes = [_LD, ctypes.c_int]
_lib.swimba_linattn_workspace_size.restype = ctypes.c_size_t
_lib.swimba_linattn_fwd.argtypes = [_LD] + [_P] * 9 + [ctypes.c_size_t, _P]
_lib.swimba_linattn_fwd.restype = ctypes.c_int
_lib.swimba_linattn_step.argtypes = [_LD] + [_P] * 8
_lib.swimba_linattn_step.restype = ctypes.c_int
_lib.swimba_linattn_bwd.argtypes = [_LD] + [_P] * 13 + [ctypes.c_size_t, _P]
_lib.swimba_linattn_bwd.restype = ctypes.c_int
_lib.swimba_block_norm_fwd.argtypes = [_ND] + [_P] * 8
_lib.swimba_block_norm_fwd.restype = ctypes.c_int
_lib.swimba_block_norm_workspace_size.argtypes = [_ND]
_lib.swimba_block_norm_workspace_size.restype = ctypes.c_size_t
_lib.swimba_block_norm_bwd.argtypes = [_ND] + [_P] * 13 + [ctypes.c_size_t, _P]
_lib.swimba_block_norm_bwd.restype = ctypes.c_int


class SwimbaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        detail = f"; {swimba_last_error_string()}" if status == 5 else ""
        super().__init__(f"{where}: {STATUS.get(status, status)} ({swimba_status_string(status)}{detail})")


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int | None:
    if stream is None:
        if _raw_stream is not None:  # the same handle without a Stream object: 0.1 in place of 3 us of a call
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _same_places(t, st, lay, dims) -> bool:
    """Whether strides that differ from `lay` still name the same elements: an axis of one has none."""
    return (len(st) == 4 and (st[0] == lay[0] or dims.batch == 1) and (st[1] == lay[1] or dims.seqlen == 1)
            and (st[2] == lay[2] or t.shape[2] == 1) and (st[3] == 1 or t.shape[3] == 1))


def _pointers(dense, dims=None, strided=(), Tensor=torch.Tensor):
    """Device pointers of a call's tensors: [B, L, heads, d] ones, each with the token stride that the call's dims
    state for it and its dtype, shape and strides (or only its channels per head), then those that have to be dense,
    with their dtype and number of elements (or alone: a workspace). None where one has another type or size, is
    laid out differently or lies on another device than the current one, whose stream the call would use (a CPU
    tensor's is -1, no device yet -2): it would be read as other values, or read and written past its end.
    Integers are taken as pointers and not looked at."""
    device = torch.cuda.current_device() if torch.cuda.is_initialized() else -2
    out = []
    for t, stride, of in strided:
        if isinstance(t, Tensor):
            if of.__class__ is tuple:
                dtype, shape, lay = of
                if t.dtype is not dtype or t.shape != shape:
                    return None
            else:
                lay = (dims.seqlen * stride, stride, of, 1)
            st = t.stride()
            if t.get_device() != device or (st != lay and not _same_places(t, st, lay, dims)):
                return None
            t = t.data_ptr()
        out.append(t)
    for t in dense:
        if t.__class__ is tuple:
            t, dtype, size = t
            if isinstance(t, Tensor):
                if t.dtype is not dtype or t.numel() != size or t.get_device() != device or not t.is_contiguous():
                    return None
                t = t.data_ptr()
        elif isinstance(t, Tensor):
            if t.get_device() != device or not t.is_contiguous():
                return None
            t = t.data_ptr()
        out.append(t)
    return out


_F32, _IO_DTYPE = torch.float32, {SWIMBA_F32: torch.float32, SWIMBA_BF16: torch.bfloat16}
_LINATTN_FIELDS, _NORM_FIELDS = struct.Struct("qqiiiiqqqif"), struct.Struct("qiiiiifff")  # all of them in 0.2 us


def _linattn_sizes(dims):
    """What a linear attention call's tensors have to be: the io dtype, heads, sequences, the token stride of q, k and v
    with (dtype, shape, strides), the elements of o and of the states."""
    B, L, H, KV, dk, dv, qs, ks, vs, io, _ = _LINATTN_FIELDS.unpack_from(dims)
    io = _IO_DTYPE.get(io)
    return (io, H, B, qs, (io, (B, L, H, dk), (L * qs, qs, dk, 1)), ks, (io, (B, L, KV, dk), (L * ks, ks, dk, 1)),
            vs, (io, (B, L, KV, dv), (L * vs, vs, dv, 1)), B * L * H * dv, B * H * dk * dv)


def _norm_sizes(dims):
    """The io and residual dtypes of a block norm call, its width and its elements."""
    rows, width, _, io, res, _, _, _, _ = _NORM_FIELDS.unpack_from(dims)
    return _IO_DTYPE.get(io), _IO_DTYPE.get(res), width, rows * width


def _room(ws, ws_bytes) -> int:
    """The workspace bytes that a call may use: what the caller says, but no more than the tensor has."""
    return min(int(ws_bytes), ws.nbytes) if isinstance(ws, torch.Tensor) else int(ws_bytes)


def check(status: int, where: str = "swimba") -> None:
    if status != 0:
        raise SwimbaError(status, where)


# ------------------------------------------------------------------------------------------------
# the C functions, same names
# ------------------------------------------------------------------------------------------------

def swimba_status_string(status: int) -> str:
    return _lib.swimba_status_string(int(status)).decode()


def swimba_last_error_string() -> str:
    return _lib.swimba_last_error_string().decode()


def swimba_kernel_launches() -> int:
    return int(_lib.swimba_kernel_launches())


def swimba_workspace_size(dims: swimba_dims, op: int) -> int:
    return int(_lib.swimba_workspace_size(ctypes.byref(dims), op))


def swimba_route(dims, x, W_r, idx, gates, stream=None) -> int:
    return _lib.swimba_route(ctypes.byref(dims), _ptr(x), _ptr(W_r), _ptr(idx), _ptr(gates), _stream(stream))


def swimba_mixed_proj(dims, x, idx, gates, weights, delta, B_mix, C_mix, ws, ws_bytes, stream=None) -> int:
    return _lib.swimba_mixed_proj(ctypes.byref(dims), _ptr(x), _ptr(idx), _ptr(gates), ctypes.byref(weights),
                                  _ptr(delta), _ptr(B_mix), _ptr(C_mix), _ptr(ws), int(ws_bytes), _stream(stream))


def swimba_scan_fwd(dims, x, z, delta, B_mix, C_mix, idx, gates, weights, h0, out, h_final, y_pre, ws, ws_bytes,
                    stream=None) -> int:
    return _lib.swimba_scan_fwd(ctypes.byref(dims), _ptr(x), _ptr(z), _ptr(delta), _ptr(B_mix), _ptr(C_mix),
                                _ptr(idx), _ptr(gates), ctypes.byref(weights), _ptr(h0), _ptr(out), _ptr(h_final),
                                _ptr(y_pre), _ptr(ws), int(ws_bytes), _stream(stream))


def swimba_scan_fwd_zoh(dims, x, z, delta, B_mix, C_mix, idx, gates, weights, h0, out, h_final, y_pre, ws, ws_bytes,
                        stream=None) -> int:
    return _lib.swimba_scan_fwd_zoh(ctypes.byref(dims), _ptr(x), _ptr(z), _ptr(delta), _ptr(B_mix), _ptr(C_mix),
                                    _ptr(idx), _ptr(gates), ctypes.byref(weights), _ptr(h0), _ptr(out),
                                    _ptr(h_final), _ptr(y_pre), _ptr(ws), int(ws_bytes), _stream(stream))


def swimba_scan_fwd_noalloc(dims, x, z, delta, B_mix, C_mix, idx, gates, weights, h0, out, h_final, y_pre,
                            stream=None) -> int:
    return _lib.swimba_scan_fwd_noalloc(ctypes.byref(dims), _ptr(x), _ptr(z), _ptr(delta), _ptr(B_mix), _ptr(C_mix),
                                        _ptr(idx), _ptr(gates), ctypes.byref(weights), _ptr(h0), _ptr(out),
                                        _ptr(h_final), _ptr(y_pre), _stream(stream))


def swimba_scan_fwd_noalloc_status(stream=None) -> int:
    return _lib.swimba_scan_fwd_noalloc_status(_stream(stream))


def swimba_scan_fwd_noalloc_status_block() -> int | None:
    return _lib.swimba_scan_fwd_noalloc_status_block()


def swimba_scan_summary(dims, x, delta, B_mix, idx, gates, weights, h_zero, log_decay, ws, ws_bytes,
                        stream=None) -> int:
    return _lib.swimba_scan_summary(ctypes.byref(dims), _ptr(x), _ptr(delta), _ptr(B_mix), _ptr(idx), _ptr(gates),
                                    ctypes.byref(weights), _ptr(h_zero), _ptr(log_decay), _ptr(ws), int(ws_bytes),
                                    _stream(stream))


def swimba_scan_chain(dims, parts, h_zero, log_decay, h0, h_start, stream=None) -> int:
    return _lib.swimba_scan_chain(ctypes.byref(dims), int(parts), _ptr(h_zero), _ptr(log_decay), _ptr(h0),
                                  _ptr(h_start), _stream(stream))


def swimba_scan_bwd(dims, x, z, delta, B_mix, C_mix, idx, gates, weights, h0, g_out, dx, dz, ddelta, dB, dC, dgates,
                    dA, dD, dh0, ws, ws_bytes, stream=None) -> int:
    return _lib.swimba_scan_bwd(ctypes.byref(dims), _ptr(x), _ptr(z), _ptr(delta), _ptr(B_mix), _ptr(C_mix), _ptr(idx),
                                _ptr(gates), ctypes.byref(weights), _ptr(h0), _ptr(g_out), _ptr(dx), _ptr(dz),
                                _ptr(ddelta), _ptr(dB), _ptr(dC), _ptr(dgates), _ptr(dA), _ptr(dD), _ptr(dh0), _ptr(ws),
                                int(ws_bytes), _stream(stream))


def swimba_proj_bwd(dims, x, idx, gates, weights, delta, g_delta, g_B, g_C, dx, dx_accumulate, dgates, dW_x, dW_dt,
                    db_dt, ws, ws_bytes, stream=None) -> int:
    return _lib.swimba_proj_bwd(ctypes.byref(dims), _ptr(x), _ptr(idx), _ptr(gates), ctypes.byref(weights), _ptr(delta),
                                _ptr(g_delta), _ptr(g_B), _ptr(g_C), _ptr(dx), int(dx_accumulate), _ptr(dgates),
                                _ptr(dW_x), _ptr(dW_dt), _ptr(db_dt), _ptr(ws), int(ws_bytes), _stream(stream))


def swimba_route_bwd(dims, x, W_r, idx, gates, g_gates_a, g_gates_b, dx, dx_accumulate, dW_r, ws, ws_bytes,
                     stream=None) -> int:
    return _lib.swimba_route_bwd(ctypes.byref(dims), _ptr(x), _ptr(W_r), _ptr(idx), _ptr(gates), _ptr(g_gates_a),
                                 _ptr(g_gates_b), _ptr(dx), int(dx_accumulate), _ptr(dW_r), _ptr(ws), int(ws_bytes),
                                 _stream(stream))


def swimba_ssd_scan(dims, X, B_j, C_mix, gates, delta, A, D_skip, S0, y, S_final, ws, ws_bytes, stream=None) -> int:
    return _lib.swimba_ssd_scan(ctypes.byref(dims), _ptr(X), _ptr(B_j), _ptr(C_mix), _ptr(gates), _ptr(delta), _ptr(A),
                                _ptr(D_skip), _ptr(S0), _ptr(y), _ptr(S_final), _ptr(ws), int(ws_bytes),
                                _stream(stream))


def swimba_separate_proj(dims, x, idx, gates, weights, delta_j, B_j, C_j, stream=None) -> int:
    return _lib.swimba_separate_proj(ctypes.byref(dims), _ptr(x), _ptr(idx), _ptr(gates), ctypes.byref(weights),
                                     _ptr(delta_j), _ptr(B_j), _ptr(C_j), _stream(stream))


def swimba_separate_scan(dims, x, z, delta_j, B_j, C_j, idx, gates, weights, h0, out, h_final, y_pre, ws, ws_bytes,
                         stream=None) -> int:
    return _lib.swimba_separate_scan(ctypes.byref(dims), _ptr(x), _ptr(z), _ptr(delta_j), _ptr(B_j), _ptr(C_j),
                                     _ptr(idx), _ptr(gates), ctypes.byref(weights), _ptr(h0), _ptr(out),
                                     _ptr(h_final), _ptr(y_pre), _ptr(ws), int(ws_bytes), _stream(stream))


def swimba_step(dims, x, z, delta, B_mix, C_mix, idx, gates, weights, h, out, stream=None) -> int:
    return _lib.swimba_step(ctypes.byref(dims), _ptr(x), _ptr(z), _ptr(delta), _ptr(B_mix), _ptr(C_mix), _ptr(idx),
                            _ptr(gates), ctypes.byref(weights), _ptr(h), _ptr(out), _stream(stream))


def swimba_get_device_status(ws, stream=None) -> int:
    return _lib.swimba_get_device_status(_ptr(ws), _stream(stream))


def swimba_check_wait_timeout(ws, ws_bytes, limit_ns, stream=None) -> int:
    return _lib.swimba_check_wait_timeout(_ptr(ws), ws_bytes, limit_ns, _stream(stream))


def swimba_conv1d_fwd(dims, d_conv, x_pre, conv_w, conv_b, conv_state_in, x, conv_state_out, stream=None) -> int:
    return _lib.swimba_conv1d_fwd(ctypes.byref(dims), int(d_conv), _ptr(x_pre), _ptr(conv_w), _ptr(conv_b),
                                  _ptr(conv_state_in), _ptr(x), _ptr(conv_state_out), _stream(stream))


def swimba_conv1d_step(dims, d_conv, x_pre, conv_w, conv_b, conv_state, x, stream=None) -> int:
    return _lib.swimba_conv1d_step(ctypes.byref(dims), int(d_conv), _ptr(x_pre), _ptr(conv_w), _ptr(conv_b),
                                   _ptr(conv_state), _ptr(x), _stream(stream))


def swimba_block_workspace_size(bdims: swimba_block_dims) -> int:
    return int(_lib.swimba_block_workspace_size(ctypes.byref(bdims)))


def swimba_block_gemm(dtype, M, N, K, A, lda, B, ldb, C0, ldc0, C1, ldc1, split, R, ldr, ws, ws_bytes,
                      stream=None) -> int:
    return _lib.swimba_block_gemm(int(dtype), int(M), int(N), int(K), _ptr(A), int(lda), _ptr(B), int(ldb), _ptr(C0),
                                  int(ldc0), _ptr(C1), int(ldc1), int(split), _ptr(R), int(ldr), _ptr(ws),
                                  int(ws_bytes), _stream(stream))


def swimba_block_fwd(bdims, u, bweights, h0, conv_state_in, out, h_final, conv_state_out, ws, ws_bytes,
                     stream=None) -> int:
    return _lib.swimba_block_fwd(ctypes.byref(bdims), _ptr(u), ctypes.byref(bweights), _ptr(h0), _ptr(conv_state_in),
                                 _ptr(out), _ptr(h_final), _ptr(conv_state_out), _ptr(ws), int(ws_bytes),
                                 _stream(stream))


def swimba_block_step(bdims, u, bweights, h, conv_state, out, ws, ws_bytes, stream=None) -> int:
    return _lib.swimba_block_step(ctypes.byref(bdims), _ptr(u), ctypes.byref(bweights), _ptr(h), _ptr(conv_state),
                                  _ptr(out), _ptr(ws), int(ws_bytes), _stream(stream))


def swimba_linattn_workspace_size(dims: swimba_linattn_dims, op: int) -> int:
    return int(_lib.swimba_linattn_workspace_size(ctypes.byref(dims), op))


def swimba_linattn_fwd(dims, q, k, v, log_decay, lens, S0, o, S_final, ws, ws_bytes, stream=None) -> int:
    io, H, B, qs, of_q, ks, of_k, vs, of_v, outs, states = _linattn_sizes(dims)
    p = _pointers(((log_decay, _F32, H), (lens, torch.int32, B), (S0, _F32, states), (o, io, outs),
                   (S_final, _F32, states), ws), dims, ((q, qs, of_q), (k, ks, of_k), (v, vs, of_v)))
    return 1 if p is None else _lib.swimba_linattn_fwd(ctypes.byref(dims), *p, _room(ws, ws_bytes), _stream(stream))


def swimba_linattn_step(dims, q, k, v, log_decay, S_in, o, S_out, stream=None) -> int:
    io, H, _, qs, of_q, ks, of_k, vs, of_v, outs, states = _linattn_sizes(dims)
    p = _pointers(((log_decay, _F32, H), (S_in, _F32, states), (o, io, outs), (S_out, _F32, states)), dims,
                  ((q, qs, of_q), (k, ks, of_k), (v, vs, of_v)))
    return 1 if p is None else _lib.swimba_linattn_step(ctypes.byref(dims), *p, _stream(stream))


def swimba_linattn_bwd(dims, q, k, v, log_decay, lens, S0, g_o, g_S, dq, dk, dv, dS0, ws, ws_bytes, stream=None) -> int:
    io, H, B, qs, of_q, ks, of_k, vs, of_v, outs, states = _linattn_sizes(dims)
    p = _pointers(((log_decay, _F32, H), (lens, torch.int32, B), (S0, _F32, states), (g_o, io, outs), (g_S, _F32, states),
                   (dS0, _F32, states), ws), dims,
                  ((q, qs, of_q), (k, ks, of_k), (v, vs, of_v), (dq, qs, of_q), (dk, ks, of_k), (dv, vs, of_v)))
    if p is None:
        return 1
    room = _room(ws, ws_bytes)
    q, k, v, dq, dk, dv, log_decay, lens, S0, g_o, g_S, dS0, ws = p
    return _lib.swimba_linattn_bwd(ctypes.byref(dims), q, k, v, log_decay, lens, S0, g_o, g_S, dq, dk, dv, dS0, ws,
                                   room, _stream(stream))


def swimba_block_norm_fwd(dims, y, z, w_post, res, w_pre, h, n, stream=None) -> int:
    io, rt, width, size = _norm_sizes(dims)
    p = _pointers(((y, io, size), (z, io, size), (w_post, _F32, width), (res, rt, size), (w_pre, _F32, width),
                   (h, rt, size), (n, io, size)))
    return 1 if p is None else _lib.swimba_block_norm_fwd(ctypes.byref(dims), *p, _stream(stream))


def swimba_block_norm_workspace_size(dims: swimba_norm_dims) -> int:
    return int(_lib.swimba_block_norm_workspace_size(ctypes.byref(dims)))


def swimba_block_norm_bwd(dims, y, z, w_post, res, w_pre, g_h, g_n, dy, dz, dres, dw_post, dw_pre, ws, ws_bytes,
                          stream=None) -> int:
    io, rt, width, size = _norm_sizes(dims)
    p = _pointers(((y, io, size), (z, io, size), (w_post, _F32, width), (res, rt, size), (w_pre, _F32, width),
                   (g_h, rt, size), (g_n, io, size), (dy, io, size), (dz, io, size), (dres, rt, size),
                   (dw_post, _F32, width), (dw_pre, _F32, width), ws))
    return 1 if p is None else _lib.swimba_block_norm_bwd(ctypes.byref(dims), *p, _room(ws, ws_bytes), _stream(stream))


# ------------------------------------------------------------------------------------------------
# marshalling helpers: shapes, host arrays -> device tensors, buffers of one layer call
# ------------------------------------------------------------------------------------------------

def dtype_code(name: str) -> int:
    return {"f32": SWIMBA_F32, "bf16": SWIMBA_BF16}[name]


_dtype_code = dtype_code


def make_dims(cfg, seqlen=None, batch=None, n_experts=None, top_k=None) -> swimba_dims:
    return swimba_dims(
        batch=cfg.batch if batch is None else batch,
        seqlen=cfg.seqlen if seqlen is None else seqlen,
        d_inner=cfg.d_inner,
        d_state=cfg.d_state,
        dt_rank=cfg.dt_rank,
        n_experts=cfg.n_experts if n_experts is None else n_experts,
        top_k=cfg.top_k if top_k is None else top_k,
        io_dtype=_dtype_code(cfg.io_dtype),
        w_dtype=_dtype_code(cfg.w_dtype),
    )


def _io_code(t: torch.Tensor) -> int:
    for code, dtype in _IO_DTYPE.items():
        if t.dtype is dtype:
            return code
    raise SwimbaError(1, f"tensor of {t.dtype}, not float32 or bfloat16")


def _token_stride(t: torch.Tensor) -> int:
    """Token stride in elements of a [B, L, heads, d] tensor that include/swimba.h's layout covers: heads
    contiguous inside a row, sequences L rows apart."""
    B, L, heads, d = t.shape
    stride = t.stride(1) if L > 1 else (t.stride(0) if B > 1 else heads * d)
    inner = (d == 1 or t.stride(3) == 1) and (heads == 1 or t.stride(2) == d)
    if not inner or (B > 1 and t.stride(0) != L * stride):
        raise SwimbaError(1, f"linear attention tensor of shape {tuple(t.shape)} and strides {t.stride()}")
    return stride


def make_linattn_dims(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, scale: float) -> swimba_linattn_dims:
    """Dims of q [B, L, H, d_k], k [B, L, Hkv, d_k], v [B, L, Hkv, d_v] as they lie in memory: dense, or
    columns of one projection's output."""
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise SwimbaError(1, f"linear attention of q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)}")
    B, L, H, dk = q.shape
    if k.shape[:2] != (B, L) or k.shape[3] != dk or v.shape[:3] != k.shape[:3] or len({q.dtype, k.dtype, v.dtype}) > 1:
        raise SwimbaError(1, f"linear attention of q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)}")
    return swimba_linattn_dims(batch=B, seqlen=L, n_heads=H, n_kv_heads=k.shape[2], d_k=dk, d_v=v.shape[3],
                               q_stride=_token_stride(q), k_stride=_token_stride(k), v_stride=_token_stride(v),
                               io_dtype=_io_code(q), scale=float(scale))


def new_linattn_workspace(dims: swimba_linattn_dims, op: int, device="cuda") -> torch.Tensor:
    n = swimba_linattn_workspace_size(dims, op)
    if n == 0:
        raise SwimbaError(1, "swimba_linattn_workspace_size")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def make_norm_dims(y: torch.Tensor, h: torch.Tensor, groups: int = 1, eps: float = 1e-5, gate_last: bool = False,
                   res_scale: float = 1.0, out_scale: float = 1.0) -> swimba_norm_dims:
    """Dims of a block norm whose mixer output looks like ``y`` and residual stream like ``h`` (the last
    axis is the width)."""
    if y.shape != h.shape:
        raise SwimbaError(1, f"block norm of y {tuple(y.shape)} and h {tuple(h.shape)}")
    width = y.shape[-1]
    return swimba_norm_dims(rows=y.numel() // max(1, width), width=width, groups=groups, io_dtype=_io_code(y),
                            res_dtype=_io_code(h), gate_last=int(gate_last), eps=eps, res_scale=res_scale,
                            out_scale=out_scale)


def new_norm_workspace(dims: swimba_norm_dims, device="cuda") -> torch.Tensor:
    n = swimba_block_norm_workspace_size(dims)
    if n == 0:
        raise SwimbaError(1, "swimba_block_norm_workspace_size")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def to_device(stored: np.ndarray, dtype: str, device="cuda", pin=False) -> torch.Tensor:
    """A stored array (uint16 bf16 bits or float32) as a torch tensor of the matching dtype."""
    if dtype == "bf16":
        t = torch.from_numpy(np.ascontiguousarray(stored).view(np.int16)).view(torch.bfloat16)
    else:
        t = torch.from_numpy(np.ascontiguousarray(stored))
    if device == "cpu":
        return t.pin_memory() if pin else t
    return t.to(device, non_blocking=False)


@dataclass
class DeviceWeights:
    W_r: torch.Tensor
    W_x: torch.Tensor
    W_dt: torch.Tensor
    b_dt: torch.Tensor
    A: torch.Tensor
    D_skip: torch.Tensor

    def struct(self) -> swimba_weights:
        return swimba_weights(*(t.data_ptr() for t in (self.W_r, self.W_x, self.W_dt, self.b_dt, self.A, self.D_skip)))


def upload_weights(w, device="cuda") -> DeviceWeights:
    """``w`` is a ``synth.LayerWeights`` (or anything with the same fields)."""
    return DeviceWeights(
        W_r=to_device(w.W_r, "f32", device),
        W_x=to_device(w.W_x, w.w_dtype, device),
        W_dt=to_device(w.W_dt, w.w_dtype, device),
        b_dt=to_device(w.b_dt, "f32", device),
        A=to_device(w.A, "f32", device),
        D_skip=to_device(w.D_skip, "f32", device),
    )


def new_workspace(dims: swimba_dims, op: int = SWIMBA_OP_LAYER, device="cuda") -> torch.Tensor:
    n = swimba_workspace_size(dims, op)
    if n == 0:
        raise SwimbaError(1, "swimba_workspace_size")
    return torch.zeros(n, dtype=torch.uint8, device=device)


class LayerBuffers:
    """The intermediate and output buffers of one layer call for ``dims`` (allocated by torch)."""

    def __init__(self, dims: swimba_dims, io_torch_dtype, device="cuda", with_y=False):
        B, L, D, N, k = dims.batch, dims.seqlen, dims.d_inner, dims.d_state, dims.top_k
        f32 = dict(dtype=torch.float32, device=device)
        self.idx = torch.empty((B, L, k), dtype=torch.int32, device=device)
        self.gates = torch.empty((B, L, k), **f32)
        self.delta = torch.empty((B, L, D), **f32)
        self.B_mix = torch.empty((B, L, N), **f32)
        self.C_mix = torch.empty((B, L, N), **f32)
        self.out = torch.empty((B, L, D), dtype=io_torch_dtype, device=device)
        self.h_final = torch.empty((B, D, N), **f32)
        self.y = torch.empty((B, L, D), **f32) if with_y else None
        self.ws = new_workspace(dims, SWIMBA_OP_LAYER, device)


def layer_forward(dims, x, z, weights: swimba_weights, buf: LayerBuffers, h0=None, stream=None) -> LayerBuffers:
    """route -> mixed_proj -> scan_fwd on one stream (three library calls)."""
    check(swimba_route(dims, x, ctypes.c_void_p(weights.W_r).value, buf.idx, buf.gates, stream), "swimba_route")
    ws_bytes = buf.ws.numel()
    check(swimba_mixed_proj(dims, x, buf.idx, buf.gates, weights, buf.delta, buf.B_mix, buf.C_mix, buf.ws, ws_bytes,
                            stream), "swimba_mixed_proj")
    check(swimba_scan_fwd(dims, x, z, buf.delta, buf.B_mix, buf.C_mix, buf.idx, buf.gates, weights, h0, buf.out,
                          buf.h_final, buf.y, buf.ws, ws_bytes, stream), "swimba_scan_fwd")
    return buf


def decode_step(dims, x, z, weights: swimba_weights, buf: LayerBuffers, h, stream=None) -> LayerBuffers:
    """route -> mixed_proj -> step (seqlen 1), updating the cached state ``h`` in place."""
    check(swimba_route(dims, x, ctypes.c_void_p(weights.W_r).value, buf.idx, buf.gates, stream), "swimba_route")
    ws_bytes = buf.ws.numel()
    check(swimba_mixed_proj(dims, x, buf.idx, buf.gates, weights, buf.delta, buf.B_mix, buf.C_mix, buf.ws, ws_bytes,
                            stream), "swimba_mixed_proj")
    check(swimba_step(dims, x, z, buf.delta, buf.B_mix, buf.C_mix, buf.idx, buf.gates, weights, h, buf.out, stream),
          "swimba_step")
    return buf
