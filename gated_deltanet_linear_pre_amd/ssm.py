"""Thin ctypes binding of the state space layer in libgdn.so (include/gdn_ssm.h).

Same manner as binding.py: the C names, tensors become device pointers, the
stream defaults to torch's current stream, a non-zero status raises GdnError.
None stands for the optional buffers.  A tensor that is not on the current HIP
device is refused here (the library sees addresses only); everything else is
checked by the library.  Rows of the raw xbc and of dt may be column blocks of
a wider tensor: pass the view and its stride(0) in the shape.
"""
from __future__ import annotations

import ctypes
import math

import torch

from .binding import GDN_F16, GDN_F32, GdnError, lib as _base_lib

GDN_BF16 = 2
DTYPE_CODE = {"f32": GDN_F32, "f16": GDN_F16, "bf16": GDN_BF16}
GDN_NORM_CENTRE, GDN_NORM_GATE_LAST = 1, 2


class gdn_ssm_shape(ctypes.Structure):
    _fields_ = [("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("state_dim", ctypes.c_int32), ("conv_width", ctypes.c_int32),
                ("n_seq", ctypes.c_int32), ("io_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("total_T", ctypes.c_int64),
                ("max_T", ctypes.c_int64), ("xbc_stride", ctypes.c_int64),
                ("dt_stride", ctypes.c_int64), ("dt_min", ctypes.c_float), ("dt_max", ctypes.c_float)]


class gdn_norm_shape(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("channels", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("x_dtype", ctypes.c_int32), ("io_dtype", ctypes.c_int32),
                ("x_stride", ctypes.c_int64), ("z_stride", ctypes.c_int64),
                ("flags", ctypes.c_int32), ("eps", ctypes.c_float)]


def make_ssm_shape(heads: int, head_dim: int, groups: int, state_dim: int, n_seq: int,
                   total_T: int, max_T: int, io: str = "bf16", out: str | None = None,
                   conv_width: int = 4, xbc_stride: int = 0, dt_stride: int = 0,
                   dt_min: float = 0.0, dt_max: float = math.inf) -> gdn_ssm_shape:
    out = io if out is None else out
    return gdn_ssm_shape(heads, head_dim, groups, state_dim, conv_width, n_seq,
                         DTYPE_CODE.get(io, io), DTYPE_CODE.get(out, out), total_T, max_T,
                         xbc_stride, dt_stride, dt_min, dt_max)


def make_norm_shape(rows: int, channels: int, groups: int, x: str = "f32", io: str = "bf16",
                    eps: float = 1e-5, centre: bool = False, gate_last: bool = False,
                    x_stride: int = 0, z_stride: int = 0) -> gdn_norm_shape:
    flags = (GDN_NORM_CENTRE if centre else 0) | (GDN_NORM_GATE_LAST if gate_last else 0)
    return gdn_norm_shape(rows, channels, groups, DTYPE_CODE.get(x, x), DTYPE_CODE.get(io, io),
                          x_stride, z_stride, flags, eps)


_lib = None


def lib() -> ctypes.CDLL:
    """libgdn.so with this header's prototypes; raises if it has not been built."""
    global _lib
    if _lib is None:
        L = _base_lib()
        P, I, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        SP, NP = ctypes.POINTER(gdn_ssm_shape), ctypes.POINTER(gdn_norm_shape)
        L.gdn_ssm_conv.restype = I
        L.gdn_ssm_conv.argtypes = [SP] + [P] * 8
        L.gdn_ssm_scan_workspace_bytes.restype = S
        L.gdn_ssm_scan_workspace_bytes.argtypes = [SP]
        L.gdn_ssm_scan.restype = I
        L.gdn_ssm_scan.argtypes = [SP] + [P] * 10 + [S, P]
        L.gdn_ssm_step.restype = I
        L.gdn_ssm_step.argtypes = [SP] + [P] * 13
        L.gdn_group_norm.restype = I
        L.gdn_group_norm.argtypes = [NP] + [P] * 6
        _lib = L
    return _lib


_current_device = torch.cuda.current_device
# the address torch.cuda.current_stream().cuda_stream holds, without the stream
# object around it (2.8 us of a call's 8)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, device: int) -> int:
    if stream is None:
        return _raw_stream(device) if _raw_stream else torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _call(name: str, shape, tensors, tail, stream, check: bool) -> int:
    """One library call: addresses, then `tail`, then the stream."""
    dev = -1
    args = []
    for x in tensors:
        if x is None or isinstance(x, int):
            args.append(x)
            continue
        at = x.get_device()
        if at != dev or at < 0:
            if at < 0:
                raise ValueError(f"{name}: a tensor in host memory")
            dev = _current_device()
            if at != dev:
                raise ValueError(f"{name}: a tensor on {x.device}, but the current HIP device is {dev}")
        args.append(x.data_ptr())
    if stream is None or not isinstance(stream, int):
        stream = _stream(stream, dev if dev >= 0 else _current_device())
    st = getattr(_lib or lib(), name)(ctypes.byref(shape), *args, *tail, stream)
    if check and st != 0:
        raise GdnError(name, st)
    return st


def gdn_ssm_conv(shape, cu_seqlens, xbc, conv_w, conv_b, hist, hist_out, out, stream=None,
                 check=True) -> int:
    return _call("gdn_ssm_conv", shape, (cu_seqlens, xbc, conv_w, conv_b, hist, hist_out, out), (),
                 stream, check)


def gdn_ssm_scan_workspace_bytes(shape) -> int:
    return int(lib().gdn_ssm_scan_workspace_bytes(ctypes.byref(shape)))


def gdn_ssm_scan(shape, cu_seqlens, xbc, dt, A_log, dt_bias, D, state, state_out, y,
                 workspace=None, workspace_bytes=None, stream=None, check=True) -> int:
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return _call("gdn_ssm_scan", shape,
                 (cu_seqlens, xbc, dt, A_log, dt_bias, D, state, state_out, y, workspace),
                 (int(workspace_bytes),), stream, check)


def gdn_ssm_step(shape, xbc, conv_w, conv_b, dt, A_log, dt_bias, D, hist, hist_out, state,
                 state_out, y, stream=None, check=True) -> int:
    return _call("gdn_ssm_step", shape, (xbc, conv_w, conv_b, dt, A_log, dt_bias, D, hist, hist_out,
                                         state, state_out, y), (), stream, check)


def gdn_group_norm(shape, x, z, weight, bias, y, stream=None, check=True) -> int:
    return _call("gdn_group_norm", shape, (x, z, weight, bias, y), (), stream, check)
