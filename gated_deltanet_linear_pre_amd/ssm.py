"""Thin ctypes binding of the state space layer in libgdn.so (include/gdn_ssm.h).

Same manner as binding.py: the C names, tensors become device pointers, the
stream defaults to torch's current stream, a non-zero status raises GdnError.
None stands for the optional buffers.  The library sees addresses only, so what
they stand for is checked here: a tensor has to be on the current HIP device, of
the type that the shape names, with elements enough for it and without gaps
(ValueError otherwise).  Rows of the raw xbc, of dt and of the norm's x and z may
be column blocks of a wider tensor: pass the view and its stride(0) in the shape.
Addresses given as integers are not checked.  Everything else is the library's.
"""
from __future__ import annotations

import ctypes
import functools
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


_TORCH = {GDN_F32: torch.float32, GDN_F16: torch.float16, GDN_BF16: torch.bfloat16}


@functools.lru_cache(maxsize=256)
def _plan(name: str, raw: bytes):
    """(argument, type, elements, strides, rows) of a call's tensors, from the bytes
    of its shape.  strides None: a tensor without gaps, of that many elements."""
    def flat(arg, dtype, least):
        return arg, dtype, least, None, None

    def rows(arg, dtype, n, cols, stride):
        return arg, dtype, n * cols, (stride or cols, 1), n

    i32, f32 = torch.int32, torch.float32
    if name == "gdn_group_norm":
        s = gdn_norm_shape.from_buffer_copy(raw)
        io, ch = _TORCH.get(s.io_dtype), s.channels
        return (rows("x", _TORCH.get(s.x_dtype), s.rows, ch, s.x_stride), rows("z", io, s.rows, ch, s.z_stride),
                flat("weight", io, ch), flat("bias", io, ch), flat("y", io, s.rows * ch))
    s = gdn_ssm_shape.from_buffer_copy(raw)
    H, T, io, out = s.heads, s.total_T, _TORCH.get(s.io_dtype), _TORCH.get(s.out_dtype)
    x = H * s.head_dim
    C = x + 2 * s.groups * s.state_dim
    cu, w, b = flat("cu_seqlens", i32, s.n_seq + 1), flat("conv_w", io, C * s.conv_width), flat("conv_b", io, C)
    raw_x, dt = rows("xbc", io, T, C, s.xbc_stride), rows("dt", io, T, H, s.dt_stride)
    heads = tuple(flat(k, f32, H) for k in ("A_log", "dt_bias", "D"))
    hist = tuple(flat(k, io, s.n_seq * (s.conv_width - 1) * C) for k in ("hist", "hist_out"))
    state = tuple(flat(k, f32, s.n_seq * x * s.state_dim) for k in ("state", "state_out"))
    y = flat("y", out, T * x)
    if name == "gdn_ssm_conv":
        return (cu, raw_x, w, b, *hist, flat("out", io, T * C))
    if name == "gdn_ssm_scan":
        return (cu, flat("xbc", io, T * C), dt, *heads, *state, y, flat("workspace", None, 0))
    return (raw_x, w, b, dt, *heads, *hist, *state, y)


def _refuse(name: str, x, arg, dtype, least, strides, n):
    """ValueError if `x` is not the tensor of this entry of the plan; _call comes
    here with what is not so at first sight."""
    if dtype is not None and x.dtype is not dtype:
        raise ValueError(f"{name}: {arg} is {x.dtype}, the shape says {dtype}")
    if strides is None:
        if not x.is_contiguous():
            raise ValueError(f"{name}: {arg} has gaps between its elements (strides {x.stride()})")
        if x.numel() < least:
            raise ValueError(f"{name}: {arg} has {x.numel()} elements of {least}")
        return
    cols = least // n if n > 0 else 0
    if x.is_contiguous():
        fits = n <= 0 or x.numel() >= (n - 1) * strides[0] + cols
    else:
        fits = x.dim() == 2 and x.shape[0] >= n and x.shape[1] >= cols and x.stride(1) == 1 and (n <= 1 or x.stride(0) == strides[0])
    if not fits:
        raise ValueError(f"{name}: {arg} of {tuple(x.shape)}, strides {x.stride()}, is not {n} rows of {cols} elements, {strides[0]} apart")


# torch.cuda.current_device() without its look at whether torch has started (0.2 us),
# which a tensor on a device answers, and the address torch.cuda.current_stream()
# holds without the stream object around it (2.8 us of a call's 8)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, device: int) -> int:
    if stream is None:
        return _raw_stream(device) if _raw_stream else torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _call(name: str, shape, tensors, tail, stream, check: bool) -> int:
    """One library call: addresses, then `tail`, then the stream."""
    dev = -1
    args = []
    for x, (arg, dtype, least, strides, n) in zip(tensors, _plan(name, bytes(shape))):
        if x is None or type(x) is int:
            args.append(x)
            continue
        if x.dtype is not dtype or not (x.is_contiguous() and x.numel() >= least if strides is None
                                        else x.stride() == strides and x.size(0) == n and x.numel() == least):
            _refuse(name, x, arg, dtype, least, strides, n)
        at = x.get_device()
        if at != dev or at < 0:
            if at < 0:
                raise ValueError(f"{name}: a tensor in host memory")
            dev = _current_device()
            if at != dev:
                raise ValueError(f"{name}: a tensor on {x.device}, but the current HIP device is {dev}")
        args.append(x.data_ptr())
    if stream is None or not isinstance(stream, int):
        stream = _stream(stream, dev if dev >= 0 else torch.cuda.current_device())
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
    held = workspace.nbytes if isinstance(workspace, torch.Tensor) else 0
    if workspace_bytes is None:
        workspace_bytes = held
    elif workspace_bytes < 0 or isinstance(workspace, torch.Tensor) and workspace_bytes > held:
        raise ValueError(f"gdn_ssm_scan: a workspace of {held} bytes, not {workspace_bytes}")
    return _call("gdn_ssm_scan", shape,
                 (cu_seqlens, xbc, dt, A_log, dt_bias, D, state, state_out, y, workspace),
                 (int(workspace_bytes),), stream, check)


def gdn_ssm_step(shape, xbc, conv_w, conv_b, dt, A_log, dt_bias, D, hist, hist_out, state,
                 state_out, y, stream=None, check=True) -> int:
    return _call("gdn_ssm_step", shape, (xbc, conv_w, conv_b, dt, A_log, dt_bias, D, hist, hist_out,
                                         state, state_out, y), (), stream, check)


def gdn_group_norm(shape, x, z, weight, bias, y, stream=None, check=True) -> int:
    return _call("gdn_group_norm", shape, (x, z, weight, bias, y), (), stream, check)
