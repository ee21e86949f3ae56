"""Thin ctypes binding of the attention operators in libgdn.so (include/gdn_attn.h).

Same manner as ssm.py: the C names, tensors become device pointers, the stream
defaults to torch's current stream, a non-zero status raises GdnError.  None stands
for the optional buffers.  The library sees addresses only, so what they stand for is
checked here: a tensor has to be on the current HIP device, of the type that the shape
names, with elements enough for it and without gaps (ValueError otherwise).  Rows of q,
k, v and gate may be column blocks of a wider tensor, and the caches may be the halves
of one (pages[:, 0] and pages[:, 1]): pass the view and its stride(0) in the shape.
Addresses given as integers are not checked.  Everything else is the library's.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from .binding import GDN_F16, GDN_F32, GdnError, lib as _base_lib
from .ssm import DTYPE_CODE, GDN_BF16, _current_device, _stream

GDN_ROPE_PAIRS = 1
GDN_ROPE_PLAIN, GDN_ROPE_LINEAR, GDN_ROPE_BASE, GDN_ROPE_PARTS = range(4)
ROPE_KIND = {"plain": GDN_ROPE_PLAIN, "linear": GDN_ROPE_LINEAR, "base": GDN_ROPE_BASE, "parts": GDN_ROPE_PARTS}


class gdn_attn_shape(ctypes.Structure):
    _fields_ = [(k, ctypes.c_int32) for k in ("heads", "kv_heads", "head_dim", "page_size", "n_seq", "io_dtype",
                                              "rope_dim", "flags")] + \
               [(k, ctypes.c_int64) for k in ("total_T", "max_T", "max_kv", "n_pages", "table_pages", "page_stride",
                                              "q_stride", "k_stride", "v_stride", "gate_stride", "window")] + \
               [(k, ctypes.c_float) for k in ("scale", "rope_scale", "eps")] + [("reserved", ctypes.c_int32)]


class gdn_rope(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("rope_dim", ctypes.c_int32)] + \
               [(k, ctypes.c_double) for k in ("base", "factor", "trained", "slow", "fast")]


def make_attn_shape(heads: int, kv_heads: int, head_dim: int, n_seq: int = 1, total_T: int = 0, max_T: int = 0,
                    max_kv: int = 0, n_pages: int = 1, table_pages: int = 1, page_size: int = 64, io: str = "bf16",
                    rope_dim: int = 0, interleaved: bool = False, rope_scale: float = 1.0, eps: float = 1e-6,
                    scale: float | None = None, window: int = 0, page_stride: int = 0, q_stride: int = 0,
                    k_stride: int = 0, v_stride: int = 0, gate_stride: int = 0) -> gdn_attn_shape:
    """scale None: 1 / sqrt(head_dim)."""
    if scale is None:
        scale = head_dim ** -0.5 if head_dim > 0 else 1.0
    return gdn_attn_shape(heads, kv_heads, head_dim, page_size, n_seq, DTYPE_CODE.get(io, io), rope_dim,
                          GDN_ROPE_PAIRS if interleaved else 0, total_T, max_T, max_kv, n_pages, table_pages, page_stride,
                          q_stride, k_stride, v_stride, gate_stride, window, scale, rope_scale, eps, 0)


_lib = None


def lib() -> ctypes.CDLL:
    """libgdn.so with this header's prototypes; raises if it has not been built."""
    global _lib
    if _lib is None:
        L = _base_lib()
        P, I, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        SP = ctypes.POINTER(gdn_attn_shape)
        L.gdn_attn_append.restype = I
        L.gdn_attn_append.argtypes = [SP] + [P] * 14
        for name, n in (("gdn_attn_prefill", 8), ("gdn_attn_step", 7)):
            f, w = getattr(L, name), getattr(L, name + "_workspace_bytes")
            f.restype, f.argtypes = I, [SP] + [P] * (n + 1) + [S, P]
            w.restype, w.argtypes = S, [SP]
        L.gdn_attn_copy_pages.restype = I
        L.gdn_attn_copy_pages.argtypes = [SP, P, ctypes.c_int64, P, P, P]
        L.gdn_attn_rope_freqs.restype = I
        L.gdn_attn_rope_freqs.argtypes = [ctypes.POINTER(gdn_rope), P, P]
        _lib = L
    return _lib


_TORCH = {GDN_F32: torch.float32, GDN_F16: torch.float16, GDN_BF16: torch.bfloat16}


@functools.lru_cache(maxsize=256)
def _plan(name: str, raw: bytes):
    """(argument, type, least elements, natural sizes, natural strides, piece) of a call's
    tensors, from the bytes of its shape.  A tensor without gaps needs the elements, any other
    the sizes and strides; of other views _refuse looks at the piece: elements, stride and
    count of its rows or pages (None: it has to be without gaps)."""
    s = gdn_attn_shape.from_buffer_copy(raw)
    io, f32, i32 = _TORCH.get(s.io_dtype), torch.float32, torch.int32
    T, D, q, kv = s.total_T, s.head_dim, s.heads * s.head_dim, s.kv_heads * s.head_dim

    def flat(arg, dtype, least):
        return arg, dtype, least, None, None, None

    def rows(arg, cols, stride):
        stride = stride or cols
        return arg, io, (T - 1) * stride + cols if T > 0 else 0, (T, cols), (stride, 1), (cols, stride, T)

    page = kv * s.page_size
    stride = s.page_stride or page
    cache = tuple((k, io, (s.n_pages - 1) * stride + page, (s.n_pages, s.kv_heads, s.page_size, D),
                   (stride, s.page_size * D, D, 1), (page, stride, s.n_pages)) for k in ("k_cache", "v_cache"))
    if name == "gdn_attn_copy_pages":
        return (flat("pairs", i32, 0), *cache)
    seqs = (flat("kv_len", i32, s.n_seq), flat("page_table", i32, s.n_seq * s.table_pages))
    if name != "gdn_attn_step":
        seqs = (flat("cu_seqlens", i32, s.n_seq + 1), *seqs)
    if name == "gdn_attn_append":
        return (*seqs, flat("positions", i32, T), rows("q", q, s.q_stride), rows("k", kv, s.k_stride), rows("v", kv, s.v_stride),
                flat("inv_freq", f32, s.rope_dim // 2), flat("q_norm", io, D), flat("k_norm", io, D), flat("q_out", io, T * q),
                *cache)
    return (*seqs, rows("q", q, s.q_stride), *cache, rows("gate", q, s.gate_stride), flat("out", io, T * q),
            flat("workspace", torch.uint8, 0))


def _dense(x) -> bool:
    """Without gaps from its second dimension on."""
    least = 1
    for n, at in zip(reversed(x.shape[1:]), reversed(x.stride()[1:])):
        if n != 1 and at != least:
            return False
        least *= n
    return True


def _refuse(name: str, x, arg, dtype, least, piece):
    """ValueError if `x` is not the tensor of this entry of the plan; _call comes here with
    what is not so at first sight."""
    if x.dtype is not dtype and arg != "workspace":  # (bytes of any type)
        raise ValueError(f"{name}: {arg} is {x.dtype}, the shape says {dtype}")
    if piece is None or x.is_contiguous():
        if not x.is_contiguous():
            raise ValueError(f"{name}: {arg} has gaps between its elements (strides {x.stride()})")
        if x.numel() < least:
            raise ValueError(f"{name}: {arg} has {x.numel()} elements of {least}")
        return
    size, stride, count = piece
    n = x.shape[0] if x.dim() else 0
    if x.dim() < 2 or n < count or n > 0 and x.numel() // n < size or not _dense(x) or count > 1 and x.stride(0) != stride:
        raise ValueError(f"{name}: {arg} of {tuple(x.shape)}, strides {x.stride()}, is not {count} pieces of {size} elements, {stride} apart")


def _call(name: str, shape, tensors, tail, stream, check: bool, between=()) -> int:
    """One library call: addresses (`between` after the first of them), then `tail`, then the stream."""
    dev = -1
    args = []
    for x, (arg, dtype, least, sizes, strides, piece) in zip(tensors, _plan(name, bytes(shape))):
        if x is None or type(x) is int:
            args.append(x)
            continue
        if x.dtype is not dtype or not (x.numel() >= least if x.is_contiguous()
                                        else x.stride() == strides and x.shape == sizes):
            _refuse(name, x, arg, dtype, least, piece)
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
    st = getattr(_lib or lib(), name)(ctypes.byref(shape), *args[:1], *between, *args[1:], *tail, stream)
    if check and st != 0:
        raise GdnError(name, st)
    return st


def _held(name: str, workspace, workspace_bytes) -> int:
    held = workspace.nbytes if isinstance(workspace, torch.Tensor) else 0
    if workspace_bytes is None:
        return held
    if workspace_bytes < 0 or isinstance(workspace, torch.Tensor) and workspace_bytes > held:
        raise ValueError(f"{name}: a workspace of {held} bytes, not {workspace_bytes}")
    return int(workspace_bytes)


def gdn_attn_append(shape, cu_seqlens, kv_len, page_table, positions, q, k, v, inv_freq, q_norm, k_norm, q_out, k_cache,
                    v_cache, stream=None, check=True) -> int:
    return _call("gdn_attn_append", shape, (cu_seqlens, kv_len, page_table, positions, q, k, v, inv_freq, q_norm, k_norm,
                                            q_out, k_cache, v_cache), (), stream, check)


def gdn_attn_prefill_workspace_bytes(shape) -> int:
    return int(lib().gdn_attn_prefill_workspace_bytes(ctypes.byref(shape)))


def gdn_attn_prefill(shape, cu_seqlens, kv_len, page_table, q, k_cache, v_cache, gate, out, workspace=None,
                     workspace_bytes=None, stream=None, check=True) -> int:
    held = _held("gdn_attn_prefill", workspace, workspace_bytes)
    return _call("gdn_attn_prefill", shape, (cu_seqlens, kv_len, page_table, q, k_cache, v_cache, gate, out, workspace),
                 (held,), stream, check)


def gdn_attn_step_workspace_bytes(shape) -> int:
    return int(lib().gdn_attn_step_workspace_bytes(ctypes.byref(shape)))


def gdn_attn_step(shape, kv_len, page_table, q, k_cache, v_cache, gate, out, workspace=None, workspace_bytes=None,
                  stream=None, check=True) -> int:
    held = _held("gdn_attn_step", workspace, workspace_bytes)
    return _call("gdn_attn_step", shape, (kv_len, page_table, q, k_cache, v_cache, gate, out, workspace), (held,),
                 stream, check)


def gdn_attn_copy_pages(shape, pairs, n, k_cache, v_cache, stream=None, check=True) -> int:
    if isinstance(pairs, torch.Tensor) and pairs.numel() < 2 * n:
        raise ValueError(f"gdn_attn_copy_pages: pairs has {pairs.numel()} elements of {2 * n}")
    return _call("gdn_attn_copy_pages", shape, (pairs, k_cache, v_cache), (), stream, check, between=(n,))


def gdn_attn_rope_freqs(rope_dim: int, base: float = 10000.0, kind: str = "plain", factor: float = 1.0, trained: float = 1.0,
                        slow: float = 1.0, fast: float = 32.0, check=True):
    """(inv_freq, rope_scale): a host tensor of rope_dim / 2 frequencies, to be moved to the
    device once, and the factor for the shape."""
    freqs, scale = torch.zeros(max(0, min(rope_dim, 256)) // 2), ctypes.c_float()
    r = gdn_rope(ROPE_KIND.get(kind, kind), rope_dim, base, factor, trained, slow, fast)
    st = lib().gdn_attn_rope_freqs(ctypes.byref(r), freqs.data_ptr(), ctypes.byref(scale))
    if check and st != 0:
        raise GdnError("gdn_attn_rope_freqs", st)
    return freqs, scale.value
