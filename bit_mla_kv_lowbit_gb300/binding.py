"""ctypes binding of ``libmla_lowbit.so`` (the C ABI in include/mla_lowbit.h).

Argument marshalling only: each function checks tensor devices, dtypes,
shapes and contiguity, then passes raw pointers and the current CUDA stream
to the library.  Every step of the computation runs in the library's CUDA
kernels; there is no fallback, and loading fails loudly when the library is
missing.
"""

from __future__ import annotations

import ctypes
import math
import os
from typing import Optional, Sequence

import numpy as np

from . import build as _build

_LIB: Optional[ctypes.CDLL] = None

EXPORTS = (
    "mla_lowbit_page_bytes",
    "mla_lowbit_bytes_per_token",
    "mla_lowbit_write",
    "mla_lowbit_decode_plan",
    "mla_lowbit_decode",
    "mla_lowbit_decode_noalloc",
    "mla_lowbit_write_decode",
    "mla_lowbit_decode_multi",
    "mla_lowbit_assign",
    "mla_lowbit_rope_table",
    "mla_lowbit_norm_rope",
    "mla_lowbit_norm_rope_write",
    "mla_lowbit_read",
    "mla_lowbit_window_plan",
    "mla_lowbit_decode_window",
    "mla_lowbit_set_fault_injection",
    "mla_lowbit_read_error",
    "mla_lowbit_strerror",
    "mla_lowbit_version",
)

DEV_BAD_SEQ, DEV_BAD_POS, DEV_BAD_PAGE, DEV_BAD_LEN, DEV_PLAN, DEV_PIPELINE = 1, 2, 4, 8, 16, 32
DEV_NO_ROOM = 64
_CLEAR_SKIPPED = 0x100  # MLA_LOWBIT_CLEAR_SKIPPED
ROPE_SCALINGS = ("none", "linear", "ntk", "yarn")  # the ABI's MLA_LOWBIT_ROPE_* values, in order


class Layout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in
                ("content_bits", "rope_bits", "group", "sink", "local", "page_tokens",
                 "latent", "rope", "rotate")]


def layout(content_bits: int = 4, rope_bits: int = 4, rotate: bool = False) -> Layout:
    return Layout(_int32(content_bits, "content_bits"), _int32(rope_bits, "rope_bits"), 64, 4, 128, 64, 512, 64,
                  int(bool(rotate)))


class LibraryError(RuntimeError):
    pass


# The ABI's ints hold 32 bits, and ctypes keeps the low 32 of a larger number
# without an error: what does not fit is refused here.
_INT32_MAX = 2 ** 31 - 1
_ESIZE = -4


def _whole(v, name: str) -> int:
    if v != int(v):
        raise ValueError(f"{name} must be a whole number, got {v}")
    return int(v)


def _int32(v, name: str) -> int:
    v = _whole(v, name)
    if not -_INT32_MAX - 1 <= v <= _INT32_MAX:
        raise ValueError(f"{name} must fit in 32 bits, got {v}")
    return v


def _tokens(v, name: str) -> int:
    """A window or a number of first tokens: they may exceed every sequence, and
    no sequence is longer than an int32, so what is beyond that is all tokens (and
    below 0 out of range)."""
    return min(max(_whole(v, name), -1), _INT32_MAX)


def _check_sizes(what: str, *sizes: int):
    if max(sizes) > _INT32_MAX:
        _check(_ESIZE, what)


def lib_path() -> str:
    return _build.LIB


def load(path: Optional[str] = None) -> ctypes.CDLL:
    """Load the library (building it first if it is missing or stale)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = path or lib_path()
    if not os.path.exists(path):
        _build.build_library()
    if not os.path.exists(path):
        raise LibraryError(f"libmla_lowbit.so not found at {path}")
    lib = ctypes.CDLL(path)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    lp = ctypes.POINTER(Layout)
    lib.mla_lowbit_page_bytes.argtypes = [lp]
    lib.mla_lowbit_page_bytes.restype = sz
    lib.mla_lowbit_bytes_per_token.argtypes = [lp]
    lib.mla_lowbit_bytes_per_token.restype = sz
    lib.mla_lowbit_write.argtypes = [lp, i32, vp, vp, vp, vp, vp, i32, vp, i32, vp, i64, vp, vp,
                                     vp, vp]
    lib.mla_lowbit_write.restype = i32
    lib.mla_lowbit_decode_plan.argtypes = [lp, i32, i32, vp, i32, ctypes.POINTER(i32),
                                           ctypes.POINTER(i32), ctypes.POINTER(sz)]
    lib.mla_lowbit_decode_plan.restype = i32
    lib.mla_lowbit_decode.argtypes = [lp, i32, i32, ctypes.c_float, vp, vp, i64, vp, i32, vp, vp,
                                      vp, vp, vp, vp, vp, sz, vp, vp]
    lib.mla_lowbit_decode.restype = i32
    lib.mla_lowbit_decode_noalloc.argtypes = [lp, i32, i32, ctypes.c_float, vp, vp, i64, vp, i32,
                                              vp, vp, vp, vp, vp, vp, vp, vp]
    lib.mla_lowbit_decode_noalloc.restype = i32
    lib.mla_lowbit_write_decode.argtypes = [lp, i32, i32, ctypes.c_float, vp, vp, vp, vp, i64, vp,
                                            i32, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp]
    lib.mla_lowbit_write_decode.restype = i32
    lib.mla_lowbit_decode_multi.argtypes = [lp, i32, i32, i32, ctypes.c_float, vp, vp, i64, vp,
                                            i32, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp]
    lib.mla_lowbit_decode_multi.restype = i32
    f32, f64 = ctypes.c_float, ctypes.c_double
    lib.mla_lowbit_assign.argtypes = [i32] * 4 + [vp] * 14
    lib.mla_lowbit_assign.restype = i32
    lib.mla_lowbit_rope_table.argtypes = [i32, f64, i32, f64, i32, f64, f64, vp, vp]
    lib.mla_lowbit_rope_table.restype = i32
    lib.mla_lowbit_norm_rope.argtypes = [i32, i32, i32, i32, vp, i64, i64, vp, i64, i64, i32, vp, f32,
                                         i32, i32, i32, vp, f32, vp, vp]
    lib.mla_lowbit_norm_rope.restype = i32
    lib.mla_lowbit_norm_rope_write.argtypes = [lp, i32, vp, i64, vp, f32, i32, vp, f32, vp, vp, vp,
                                               i32, vp, i32, vp, i64, vp, vp, vp, vp, vp, vp]
    lib.mla_lowbit_norm_rope_write.restype = i32
    lib.mla_lowbit_read.argtypes = [lp, i32, vp, vp, i32, vp, vp, i32, vp, i64, vp, vp, i32, vp, vp, vp]
    lib.mla_lowbit_read.restype = i32
    lib.mla_lowbit_window_plan.argtypes = [lp, i32, i32, i32, i32, i32, i32, i32, ctypes.POINTER(i32),
                                           ctypes.POINTER(sz)]
    lib.mla_lowbit_window_plan.restype = i32
    lib.mla_lowbit_decode_window.argtypes = [lp, i32, i32, i32, f32, i32, i32, vp, vp, i64, vp, i32, vp,
                                             vp, vp, i32, vp, vp, vp, sz, vp, vp]
    lib.mla_lowbit_decode_window.restype = i32
    lib.mla_lowbit_set_fault_injection.argtypes = [i32, i64]
    lib.mla_lowbit_set_fault_injection.restype = i32
    lib.mla_lowbit_read_error.argtypes = [vp, ctypes.POINTER(ctypes.c_int32)]
    lib.mla_lowbit_read_error.restype = i32
    lib.mla_lowbit_strerror.argtypes = [i32]
    lib.mla_lowbit_strerror.restype = ctypes.c_char_p
    lib.mla_lowbit_version.argtypes = []
    lib.mla_lowbit_version.restype = i32
    _LIB = lib
    return lib


def strerror(status: int) -> str:
    return load().mla_lowbit_strerror(int(status)).decode()


def _check(status: int, what: str):
    if status != 0:
        raise LibraryError(f"{what}: {strerror(status)} ({status})")


def page_bytes(lay: Layout) -> int:
    return int(load().mla_lowbit_page_bytes(ctypes.byref(lay)))


def bytes_per_token(lay: Layout) -> int:
    return int(load().mla_lowbit_bytes_per_token(ctypes.byref(lay)))


def version() -> int:
    return int(load().mla_lowbit_version())


def decode_plan(lay: Layout, heads: int, seq_lens_host: Sequence[int], num_sms: int = 0):
    """Returns ``(total_splits, chunk_pages, workspace_bytes)``."""
    lens = np.ascontiguousarray(np.asarray(seq_lens_host, dtype=np.int32))
    tot, chunk, ws = ctypes.c_int(), ctypes.c_int(), ctypes.c_size_t()
    st = load().mla_lowbit_decode_plan(ctypes.byref(lay), len(lens), _int32(heads, "heads"),
                                       lens.ctypes.data_as(ctypes.c_void_p), _int32(num_sms, "num_sms"),
                                       ctypes.byref(tot), ctypes.byref(chunk), ctypes.byref(ws))
    _check(st, "mla_lowbit_decode_plan")
    return tot.value, chunk.value, ws.value


# ---------------------------------------------------------------- torch marshalling

_TORCH = None


def _torch():
    global _TORCH
    if _TORCH is None:
        import torch
        _TORCH = torch
    return _TORCH


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream, device) -> Optional[int]:
    """The given stream, or the current stream of the device the call runs on."""
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream


def _same_device(device, **tensors):
    """Every CUDA tensor of a call must be on the page pool's device: the
    library launches on the current device, which the call sets to that one."""
    for name, t in tensors.items():
        if t is not None and t.device.type == "cuda" and t.device != device:
            raise ValueError(f"{name} is on {t.device}, the page pool on {device}")


def _expect(t, name, dtype, shape=None, device=True):
    torch = _torch()
    if t is None:
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if device and t.device.type != "cuda":
        raise ValueError(f"{name} must be on a CUDA device")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def write(lay: Layout, ckv, krope, pos, block_table, page_pool, sink_buf, recent_buf, err_word,
          seq_idx=None, seq_lens_after=None, stream=None):
    """Pack ``n`` tokens into the paged cache (mla_lowbit_write)."""
    torch = _torch()
    n = ckv.shape[0]
    _expect(ckv, "ckv", torch.bfloat16, (n, 512))
    _expect(krope, "krope", torch.bfloat16, (n, 64))
    _expect(pos, "pos", torch.int32, (n,))
    _expect(block_table, "block_table", torch.int32)
    _expect(page_pool, "page_pool", torch.uint8)
    _expect(err_word, "err_word", torch.int32, (1,))
    num_seqs, max_pages = block_table.shape
    _check_sizes("mla_lowbit_write", n, num_seqs, max_pages)
    if seq_idx is not None:
        _expect(seq_idx, "seq_idx", torch.int32, (n,))
    if seq_lens_after is not None:
        _expect(seq_lens_after, "seq_lens_after", torch.int32, (num_seqs,))
    if lay.content_bits != 16:
        _expect(sink_buf, "sink_buf", torch.bfloat16, (num_seqs, 4, 576))
        _expect(recent_buf, "recent_buf", torch.bfloat16, (num_seqs, 128, 576))
    pb = page_bytes(lay)
    if page_pool.dim() != 2 or page_pool.shape[1] != pb:
        raise ValueError(f"page_pool must be [num_pages][{pb}] uint8")
    _same_device(page_pool.device, ckv=ckv, krope=krope, pos=pos, block_table=block_table,
                 sink_buf=sink_buf, recent_buf=recent_buf, err_word=err_word, seq_idx=seq_idx,
                 seq_lens_after=seq_lens_after)
    with torch.cuda.device(page_pool.device):
        st = load().mla_lowbit_write(ctypes.byref(lay), n, _ptr(ckv), _ptr(krope), _ptr(seq_idx),
                                     _ptr(pos), _ptr(seq_lens_after), num_seqs, _ptr(block_table),
                                     max_pages, _ptr(page_pool), page_pool.shape[0], _ptr(sink_buf),
                                     _ptr(recent_buf), _ptr(err_word), _stream(stream, page_pool.device))
    _check(st, "mla_lowbit_write")


def decode(lay: Layout, q, page_pool, block_table, seq_lens, seq_lens_host, sink_buf, recent_buf,
           out, workspace, err_word, softmax_scale: float, lse=None, stream=None):
    """Low-bit MLA decode (mla_lowbit_decode); writes ``out`` (and ``lse``)."""
    torch = _torch()
    B, H, _ = q.shape
    _expect(q, "q", torch.bfloat16, (B, H, 576))
    _expect(page_pool, "page_pool", torch.uint8)
    _expect(block_table, "block_table", torch.int32)
    _expect(seq_lens, "seq_lens", torch.int32, (B,))
    _expect(out, "out", torch.float32, (B, H, 512))
    _expect(workspace, "workspace", torch.uint8)
    _expect(err_word, "err_word", torch.int32, (1,))
    if lse is not None:
        _expect(lse, "lse", torch.float32, (B, H))
    if block_table.shape[0] != B:
        raise ValueError("block_table must have one row per sequence")
    _check_sizes("mla_lowbit_decode", B, H, block_table.shape[1])
    if lay.content_bits != 16:
        _expect(sink_buf, "sink_buf", torch.bfloat16, (B, 4, 576))
        _expect(recent_buf, "recent_buf", torch.bfloat16, (B, 128, 576))
    lens = np.ascontiguousarray(np.asarray(seq_lens_host, dtype=np.int32))
    if lens.shape != (B,):
        raise ValueError("seq_lens_host must have one entry per sequence")
    _same_device(page_pool.device, q=q, block_table=block_table, seq_lens=seq_lens, sink_buf=sink_buf,
                 recent_buf=recent_buf, out=out, workspace=workspace, err_word=err_word, lse=lse)
    with torch.cuda.device(page_pool.device):
        st = load().mla_lowbit_decode(
            ctypes.byref(lay), B, H, ctypes.c_float(softmax_scale), _ptr(q), _ptr(page_pool),
            page_pool.shape[0], _ptr(block_table), block_table.shape[1], _ptr(seq_lens),
            lens.ctypes.data_as(ctypes.c_void_p), _ptr(sink_buf), _ptr(recent_buf), _ptr(out),
            _ptr(lse), _ptr(workspace), workspace.numel(), _ptr(err_word), _stream(stream, page_pool.device))
    _check(st, "mla_lowbit_decode")


def write_decode(lay: Layout, q, ckv_new, krope_new, page_pool, block_table, seq_lens,
                 seq_lens_host, sink_buf, recent_buf, out, workspace, err_word,
                 softmax_scale: float, lse=None, stream=None):
    """mla_lowbit_write_decode: append one token per sequence (at position
    seq_lens[s] - 1) and decode, in one call."""
    torch = _torch()
    B, H, _ = q.shape
    _expect(q, "q", torch.bfloat16, (B, H, 576))
    _expect(ckv_new, "ckv_new", torch.bfloat16, (B, 512))
    _expect(krope_new, "krope_new", torch.bfloat16, (B, 64))
    _expect(page_pool, "page_pool", torch.uint8)
    _expect(block_table, "block_table", torch.int32)
    _expect(seq_lens, "seq_lens", torch.int32, (B,))
    _expect(out, "out", torch.float32, (B, H, 512))
    _expect(workspace, "workspace", torch.uint8)
    _expect(err_word, "err_word", torch.int32, (1,))
    if lse is not None:
        _expect(lse, "lse", torch.float32, (B, H))
    if block_table.shape[0] != B:
        raise ValueError("block_table must have one row per sequence")
    _check_sizes("mla_lowbit_write_decode", B, H, block_table.shape[1])
    if lay.content_bits != 16:
        _expect(sink_buf, "sink_buf", torch.bfloat16, (B, 4, 576))
        _expect(recent_buf, "recent_buf", torch.bfloat16, (B, 128, 576))
    lens = np.ascontiguousarray(np.asarray(seq_lens_host, dtype=np.int32))
    if lens.shape != (B,):
        raise ValueError("seq_lens_host must have one entry per sequence")
    _same_device(page_pool.device, q=q, ckv_new=ckv_new, krope_new=krope_new, block_table=block_table,
                 seq_lens=seq_lens, sink_buf=sink_buf, recent_buf=recent_buf, out=out,
                 workspace=workspace, err_word=err_word, lse=lse)
    with torch.cuda.device(page_pool.device):
        st = load().mla_lowbit_write_decode(
            ctypes.byref(lay), B, H, ctypes.c_float(softmax_scale), _ptr(q), _ptr(ckv_new),
            _ptr(krope_new), _ptr(page_pool), page_pool.shape[0], _ptr(block_table),
            block_table.shape[1], _ptr(seq_lens), lens.ctypes.data_as(ctypes.c_void_p), _ptr(sink_buf),
            _ptr(recent_buf), _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(),
            _ptr(err_word), _stream(stream, page_pool.device))
    _check(st, "mla_lowbit_write_decode")


def decode_multi(lay: Layout, q, page_pool, block_table, seq_lens, seq_lens_host, sink_buf,
                 recent_buf, out, workspace, err_word, softmax_scale: float, lse=None,
                 stream=None):
    """mla_lowbit_decode_multi: n causal queries per sequence, q [B][n][H][576]."""
    torch = _torch()
    B, n, H, _ = q.shape
    _expect(q, "q", torch.bfloat16, (B, n, H, 576))
    _expect(page_pool, "page_pool", torch.uint8)
    _expect(block_table, "block_table", torch.int32)
    _expect(seq_lens, "seq_lens", torch.int32, (B,))
    _expect(out, "out", torch.float32, (B, n, H, 512))
    _expect(workspace, "workspace", torch.uint8)
    _expect(err_word, "err_word", torch.int32, (1,))
    if lse is not None:
        _expect(lse, "lse", torch.float32, (B, n, H))
    if block_table.shape[0] != B:
        raise ValueError("block_table must have one row per sequence")
    _check_sizes("mla_lowbit_decode_multi", B, H, block_table.shape[1])
    if lay.content_bits != 16:
        _expect(sink_buf, "sink_buf", torch.bfloat16, (B, 4, 576))
        _expect(recent_buf, "recent_buf", torch.bfloat16, (B, 128, 576))
    lens = np.ascontiguousarray(np.asarray(seq_lens_host, dtype=np.int32))
    if lens.shape != (B,):
        raise ValueError("seq_lens_host must have one entry per sequence")
    _same_device(page_pool.device, q=q, block_table=block_table, seq_lens=seq_lens, sink_buf=sink_buf,
                 recent_buf=recent_buf, out=out, workspace=workspace, err_word=err_word, lse=lse)
    with torch.cuda.device(page_pool.device):
        st = load().mla_lowbit_decode_multi(
            ctypes.byref(lay), B, n, H, ctypes.c_float(softmax_scale), _ptr(q), _ptr(page_pool),
            page_pool.shape[0], _ptr(block_table), block_table.shape[1], _ptr(seq_lens),
            lens.ctypes.data_as(ctypes.c_void_p), _ptr(sink_buf), _ptr(recent_buf), _ptr(out),
            _ptr(lse), _ptr(workspace), workspace.numel(), _ptr(err_word), _stream(stream, page_pool.device))
    _check(st, "mla_lowbit_decode_multi")


def decode_noalloc(lay: Layout, q, page_pool, block_table, seq_lens, seq_lens_host, sink_buf,
                   recent_buf, out, err_word, softmax_scale: float, lse=None, stream=None):
    """mla_lowbit_decode_noalloc: the decode without a caller workspace.

    For hosts that can hand the library only inputs and outputs (no device
    allocation allowed); the split partials go to a fixed 32 MiB array the
    library keeps on each device.  Calls that overlap on the GPU race on that
    array, so keep them on one stream."""
    torch = _torch()
    B, H, _ = q.shape
    _expect(q, "q", torch.bfloat16, (B, H, 576))
    _expect(page_pool, "page_pool", torch.uint8)
    _expect(block_table, "block_table", torch.int32)
    _expect(seq_lens, "seq_lens", torch.int32, (B,))
    _expect(out, "out", torch.float32, (B, H, 512))
    _expect(err_word, "err_word", torch.int32, (1,))
    if lse is not None:
        _expect(lse, "lse", torch.float32, (B, H))
    if block_table.shape[0] != B:
        raise ValueError("block_table must have one row per sequence")
    _check_sizes("mla_lowbit_decode_noalloc", B, H, block_table.shape[1])
    if lay.content_bits != 16:
        _expect(sink_buf, "sink_buf", torch.bfloat16, (B, 4, 576))
        _expect(recent_buf, "recent_buf", torch.bfloat16, (B, 128, 576))
    lens = np.ascontiguousarray(np.asarray(seq_lens_host, dtype=np.int32))
    if lens.shape != (B,):
        raise ValueError("seq_lens_host must have one entry per sequence")
    _same_device(page_pool.device, q=q, block_table=block_table, seq_lens=seq_lens, sink_buf=sink_buf,
                 recent_buf=recent_buf, out=out, err_word=err_word, lse=lse)
    with torch.cuda.device(page_pool.device):
        st = load().mla_lowbit_decode_noalloc(
            ctypes.byref(lay), B, H, ctypes.c_float(softmax_scale), _ptr(q), _ptr(page_pool),
            page_pool.shape[0], _ptr(block_table), block_table.shape[1], _ptr(seq_lens),
            lens.ctypes.data_as(ctypes.c_void_p), _ptr(sink_buf), _ptr(recent_buf), _ptr(out),
            _ptr(lse), _ptr(err_word), _stream(stream, page_pool.device))
    _check(st, "mla_lowbit_decode_noalloc")


# ---------------------------------------------------------------- the rest of a serving step

# A decode step is a handful of kernels of a few microseconds each, so the way to
# these calls is kept short: csrc/marshal.cpp checks a call's arguments and
# launches it in one pass.  What it does not take (a wrong argument, tensors that
# are not on the current device) goes through the arguments here, as every call
# does where that extension cannot be built.

def _load_native():
    """The extension, bound to the library, or None."""
    try:
        from importlib import machinery, util
        path = _build.marshal_path()
        lib = load()
        if not os.path.exists(path):
            return None
        _torch()
        loader = machinery.ExtensionFileLoader("_marshal", path)
        module = util.module_from_spec(util.spec_from_loader("_marshal", loader))
        loader.exec_module(module)
        module.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
            lib.mla_lowbit_page_bytes, lib.mla_lowbit_assign, lib.mla_lowbit_norm_rope, lib.mla_lowbit_norm_rope_write,
            lib.mla_lowbit_read, lib.mla_lowbit_decode_window)))
        return module
    except (ImportError, OSError):
        return None


_NATIVE = False  # not looked for yet


def _native(name, *args):
    """Whether the extension has made the call ``name``."""
    global _NATIVE
    if _NATIVE is False:
        _NATIVE = _load_native()
    if _NATIVE is None:
        return False
    st = getattr(_NATIVE, name)(*args)
    if st:
        _check(st, "mla_lowbit_" + name)
    return st is not None


def _launch(call, what, index, args, stream):
    """Calls the library with the current device set to CUDA device ``index``."""
    torch = _torch()
    for v, kind in zip(args, call.argtypes):
        if kind is ctypes.c_int and not -_INT32_MAX - 1 <= v <= _INT32_MAX:
            _check(_ESIZE, what)
    s = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    if torch._C._cuda_getDevice() == index:
        st = call(*args, s)
    else:
        with torch.cuda.device(index):
            st = call(*args, s)
    if st:
        _check(st, what)


def _pointers(index, checks):
    """The data pointers of (tensor, name, dtype, shape) entries: contiguous
    tensors on CUDA device ``index`` (shape None: any).  None has the pointer
    None where the entry's shape is given in a list (an optional argument)."""
    out = []
    for t, name, dtype, shape in checks:
        if t is None:
            if type(shape) is not list:
                raise ValueError(f"{name} is required")
            out.append(None)
            continue
        if type(shape) is list:
            shape = shape[0]
        try:
            fine = (t.dtype is dtype and t.get_device() == index and t.is_contiguous()
                    and (shape is None or t.shape == shape))
        except AttributeError:
            fine = False
        if not fine:
            _expect(t, name, dtype, shape)
            raise ValueError(f"{name} is on {t.device}, the call runs on cuda:{index}")
        out.append(t.data_ptr())
    return out


def _index_of(t, name):
    """The CUDA device of a call's leading tensor."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise (ValueError if t is None else TypeError)(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    return t.get_device()


def new_output(shape, dtype, device, stream):
    """A tensor for a call on ``stream`` (None: the current one) to write.  On
    another stream than the current one it is that stream's memory, since what
    the current one has freed its pending work may still use, and is kept for
    the current one's reads too."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream(stream.device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if stream != current:
        t.record_stream(current)
    return t


def _rows_and_columns(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions")
    return t.shape


def assign(new_lens, seq_lens, block_table, free_pages, free_count, seq_idx, pos, err_word, *,
           slots=None, token_start=None, release=None, seq_lens_after=None, free_count_after=None,
           stream=None):
    """Pages and slots for ``new_lens[s]`` tokens of every sequence
    (mla_lowbit_assign).  ``seq_lens`` and ``free_count`` are updated in place
    unless ``seq_lens_after`` / ``free_count_after`` are given."""
    if _native("assign", new_lens, seq_lens, block_table, free_pages, free_count, seq_idx, pos, err_word, slots, token_start,
               release, seq_lens_after, free_count_after, stream):
        return
    torch = _torch()
    index = _index_of(block_table, "block_table")
    S, max_pages = _rows_and_columns(block_table, "block_table")
    if seq_lens_after is None:
        seq_lens_after = seq_lens
    if free_count_after is None:
        free_count_after = free_count
    if seq_idx is None or free_pages is None:
        raise ValueError("seq_idx and free_pages are required")
    n, i32, per_seq = seq_idx.numel(), torch.int32, (S,)
    ptrs = _pointers(index, (
        (new_lens, "new_lens", i32, per_seq), (release, "release", i32, [per_seq]), (seq_lens, "seq_lens", i32, per_seq),
        (free_count, "free_count", i32, (1,)), (block_table, "block_table", i32, None),
        (free_pages, "free_pages", i32, None), (seq_lens_after, "seq_lens_after", i32, per_seq),
        (free_count_after, "free_count_after", i32, (1,)), (token_start, "token_start", i32, [(S + 1,)]),
        (seq_idx, "seq_idx", i32, (n,)), (pos, "pos", i32, (n,)), (slots, "slots", torch.int64, [(n,)]),
        (err_word, "err_word", i32, (1,))))
    _launch(load().mla_lowbit_assign, "mla_lowbit_assign", index, (S, max_pages, free_pages.numel(), n, *ptrs), stream)


def rope_table(dim: int, theta: float = 10000.0, scaling: str = "none", factor: float = 1.0,
               original_len: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """``(phase, mscale)``: the uint64 numpy table of mla_lowbit_rope_table (a
    pair's turn per position in 2^-64 turns) and the factor on rotated values."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {ROPE_SCALINGS}, got {scaling!r}")
    dim = _int32(dim, "dim")
    phase = np.zeros(max(dim // 2, 1), np.uint64)
    mscale = ctypes.c_float()
    _check(load().mla_lowbit_rope_table(dim, float(theta), ROPE_SCALINGS.index(scaling), float(factor),
                                        _int32(original_len, "original_len"), float(beta_fast), float(beta_slow),
                                        phase.ctypes.data_as(ctypes.c_void_p), ctypes.byref(mscale)),
           "mla_lowbit_rope_table")
    return phase, mscale.value


class Rope:
    """A rotation of ``dim`` channels: frequencies, pair layout and scaling for
    long contexts (``none``, ``linear``, ``ntk`` or ``yarn``), its table on
    ``device``.  Made once and given to rope, norm_rope and norm_rope_write.

    YaRN sharpens attention over long contexts by t(m) = 0.1 m ln(factor) + 1 on
    queries and keys.  Where all channels of a head are rotated, all of it is in the
    rotation (the default: mscale 1, mscale_all_dim 0).  A decoupled key rotates only
    a part of them, and its checkpoints give both parameters: rotated channels are
    multiplied by ``self.mscale`` = t(mscale) / t(mscale_all_dim), and the attention's
    scale by ``self.softmax_factor`` = t(mscale_all_dim)^2, which the caller does."""

    def __init__(self, dim: int, theta: float = 10000.0, interleaved: bool = True, scaling: str = "none",
                 factor: float = 1.0, original_len: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0,
                 device="cuda", mscale: float = 1.0, mscale_all_dim: float = 0.0):
        phase, self.mscale = rope_table(dim, theta, scaling, factor, original_len, beta_fast, beta_slow)
        self.softmax_factor = 1.0
        if scaling == "yarn":
            if not (mscale >= 0 and mscale_all_dim >= 0 and math.isfinite(mscale) and math.isfinite(mscale_all_dim)):
                raise ValueError(f"mscale and mscale_all_dim must be finite and not below 0, got {mscale}, {mscale_all_dim}")
            if (mscale, mscale_all_dim) != (1, 0):
                self.mscale = (0.1 * mscale * math.log(factor) + 1) / (0.1 * mscale_all_dim * math.log(factor) + 1)
            self.softmax_factor = (0.1 * mscale_all_dim * math.log(factor) + 1) ** 2
        elif (mscale, mscale_all_dim) != (1, 0):
            raise ValueError("mscale and mscale_all_dim belong to the scaling 'yarn'")
        self.dim = int(dim)
        self.interleaved = bool(interleaved)
        self.phase = _torch().from_numpy(phase.view(np.int64)).to(device)


def _norm_rope(x, pos, rope, offset, norm, weight, eps, out, stream):
    torch = _torch()
    if out is None and isinstance(x, torch.Tensor) and x.is_cuda:
        out = new_output(x.shape, x.dtype, x.device, stream)
    if _native("norm_rope", x, pos, rope, offset, norm, weight, eps, out, stream):
        return out
    index, dtype = _index_of(x, "x"), x.dtype
    code = 0 if dtype is torch.bfloat16 else 1 if dtype is torch.float16 else 2 if dtype is torch.float32 else None
    if code is None:
        raise TypeError(f"x must be bfloat16, float16 or float32, got {dtype}")
    if x.dim() != 3:
        raise ValueError("x must be [tokens][heads][channels]")
    shape = n, heads, dim = x.shape
    if not isinstance(out, torch.Tensor) or out.shape != shape or out.dtype is not dtype or out.get_device() != index:
        raise ValueError("out must have x's shape, dtype and device")
    xt, xh, xc = x.stride()
    yt, yh, yc = out.stride()
    if dim > 1 and (xc != 1 or yc != 1):
        raise ValueError("the channels of x and out must be contiguous")
    if rope is None:
        w, = _pointers(index, ((weight, "weight", dtype, [(dim,)]),))
        rot, inter, phase, mscale, p = 0, 0, None, 1.0, None
    else:
        rot, inter, mscale = rope.dim, rope.interleaved, rope.mscale
        w, p, phase = _pointers(index, ((weight, "weight", dtype, [(dim,)]), (pos, "pos", torch.int32, (n,)),
                                        (rope.phase, "the rope's table", torch.int64, (rot // 2,))))
    _launch(load().mla_lowbit_norm_rope, "mla_lowbit_norm_rope", index,
            (code, n, heads, dim, x.data_ptr(), xt, xh, out.data_ptr(), yt, yh, norm, w, eps, rot, _whole(offset, "offset"),
             inter, phase, mscale, p), stream)
    return out


def rope(x, pos, rope, offset: int = 0, out=None, stream=None):
    """Rotates channels ``offset .. offset + rope.dim - 1`` of the rows of x
    ([tokens][heads][channels], any strides) at ``pos``; the others are copied.
    ``out`` may be x itself, a view with strides of its own, or None (new)."""
    if rope is None:
        raise ValueError("rope is required")
    return _norm_rope(x, pos, rope, offset, 0, None, 0.0, out, stream)


def norm_rope(x, pos=None, rope=None, weight=None, eps: float = 1e-6, offset: int = 0, out=None, stream=None):
    """RMS norm of every row of x ([tokens][heads][channels], any strides),
    times ``weight``, then the rotation as by ``rope`` (None: norm only), in one
    pass (mla_lowbit_norm_rope)."""
    return _norm_rope(x, pos, rope, offset, 1, weight, eps, out, stream)


_PAGE_BYTES = {4: 20736, 2: 12544, 16: 73728}  # mla_lowbit_page_bytes by content_bits


def _expect_pool(lay, block_table, page_pool):
    """(device index, num_seqs, max_pages, num_pages) of a call on a cache."""
    index = _index_of(page_pool, "page_pool")
    num_pages, pb = _rows_and_columns(page_pool, "page_pool")
    if pb != _PAGE_BYTES.get(lay.content_bits):
        want = page_bytes(lay)
        if pb != want:
            raise ValueError(f"page_pool must be [num_pages][{want}] uint8")
    if block_table is None:
        raise ValueError("block_table is required")
    S, max_pages = _rows_and_columns(block_table, "block_table")
    return index, S, max_pages, num_pages


def norm_rope_write(lay: Layout, kv, weight, rope, pos, block_table, page_pool, sink_buf, recent_buf, err_word, *,
                    eps: float = 1e-6, seq_idx=None, seq_lens_after=None, ckv_out=None, krope_out=None, stream=None):
    """Norm the latents and rotate the keys of ``kv`` ([n][576] bf16, rows of
    any stride: a projection's output) and pack them into the paged cache, in
    one pass (mla_lowbit_norm_rope_write).  ``weight`` may be None; rows with
    ``seq_idx < 0`` are skipped."""
    if _native("norm_rope_write", lay, kv, weight, rope, pos, block_table, page_pool, sink_buf, recent_buf, err_word, eps,
               seq_idx, seq_lens_after, ckv_out, krope_out, stream):
        return
    torch = _torch()
    index, S, max_pages, num_pages = _expect_pool(lay, block_table, page_pool)
    bf, i32 = torch.bfloat16, torch.int32
    if _index_of(kv, "kv") != index or kv.dtype is not bf or kv.dim() != 2 or kv.shape[1] != 576 or kv.stride(1) != 1:
        raise ValueError(f"kv must be [n][576] bfloat16 with contiguous rows on cuda:{index}")
    if rope is None or rope.dim != 64:
        raise ValueError("rope must rotate the key's 64 channels")
    n = kv.shape[0]
    packed = lay.content_bits != 16
    ptrs = _pointers(index, (
        (weight, "weight", bf, [(512,)]), (rope.phase, "the rope's table", torch.int64, (32,)),
        (seq_idx, "seq_idx", i32, [(n,)]), (pos, "pos", i32, (n,)), (seq_lens_after, "seq_lens_after", i32, [(S,)]),
        (block_table, "block_table", i32, None), (page_pool, "page_pool", torch.uint8, None),
        (sink_buf if packed else None, "sink_buf", bf, (S, 4, 576) if packed else [None]),
        (recent_buf if packed else None, "recent_buf", bf, (S, 128, 576) if packed else [None]),
        (ckv_out, "ckv_out", bf, [(n, 512)]), (krope_out, "krope_out", bf, [(n, 64)]), (err_word, "err_word", i32, (1,))))
    w, phase, idx, p, lens, table, pool, sink, recent, ckv, kr, err = ptrs
    _launch(load().mla_lowbit_norm_rope_write, "mla_lowbit_norm_rope_write", index,
            (ctypes.byref(lay), n, kv.data_ptr(), kv.stride(0) if n > 1 else 576, w, eps, rope.interleaved, phase,
             rope.mscale, idx, p, lens, S, table, max_pages, pool, num_pages, sink, recent, ckv, kr, err), stream)


def _value_type(out):
    """The ABI's number of an output that may be bf16 or float32."""
    torch = _torch()
    dtype = getattr(out, "dtype", None)
    if dtype is torch.bfloat16:
        return 0
    if dtype is torch.float32:
        return 2
    raise TypeError("out must be a bfloat16 or float32 tensor")


def read(lay: Layout, seq_idx, pos, block_table, page_pool, sink_buf, recent_buf, out, err_word, *, seq_lens=None,
         clear_skipped: bool = False, stream=None):
    """The cached tokens (seq_idx[i], pos[i]) as values, out [n][576] bf16 or
    float32 (mla_lowbit_read).  With ``seq_lens`` protected tokens come from the
    bf16 buffers, as decode sees them; without, every token's packed copy.  The
    rows of padding and of tokens with an error stay as they were, or
    (``clear_skipped``) become zeros."""
    clear_skipped = bool(clear_skipped)
    if _native("read", lay, seq_idx, pos, block_table, page_pool, sink_buf, recent_buf, out, err_word, seq_lens,
               clear_skipped, stream):
        return out
    torch = _torch()
    index, S, max_pages, num_pages = _expect_pool(lay, block_table, page_pool)
    code = _value_type(out) | (_CLEAR_SKIPPED if clear_skipped else 0)
    if pos is None:
        raise ValueError("pos is required")
    n, bf, i32 = pos.numel(), torch.bfloat16, torch.int32
    copies = seq_lens is not None and lay.content_bits != 16
    idx, p, lens, table, pool, sink, recent, o, err = _pointers(index, (
        (seq_idx, "seq_idx", i32, (n,)), (pos, "pos", i32, (n,)), (seq_lens, "seq_lens", i32, [(S,)]),
        (block_table, "block_table", i32, None), (page_pool, "page_pool", torch.uint8, None),
        (sink_buf if copies else None, "sink_buf", bf, (S, 4, 576) if copies else [None]),
        (recent_buf if copies else None, "recent_buf", bf, (S, 128, 576) if copies else [None]),
        (out, "out", out.dtype, (n, 576)), (err_word, "err_word", i32, (1,))))
    _launch(load().mla_lowbit_read, "mla_lowbit_read", index,
            (ctypes.byref(lay), n, idx, p, S, lens, table, max_pages, pool, num_pages, sink, recent, code, o, err), stream)
    return out


def window_plan(lay: Layout, num_seqs: int, heads: int, queries: int, window: int, sinks: int, max_pages: int,
                num_sms: int = 0):
    """``(splits_per_seq, workspace_bytes)`` of decode_window, for every step of
    a cache of these sizes, whatever its lengths."""
    splits, nbytes = ctypes.c_int(), ctypes.c_size_t()
    _check(load().mla_lowbit_window_plan(
        ctypes.byref(lay), _int32(num_seqs, "num_seqs"), _int32(heads, "heads"), _int32(queries, "queries"),
        _tokens(window, "window"), _tokens(sinks, "sinks"), _int32(max_pages, "max_pages"), _int32(num_sms, "num_sms"),
        ctypes.byref(splits), ctypes.byref(nbytes)), "mla_lowbit_window_plan")
    return splits.value, nbytes.value


def decode_window(lay: Layout, q, page_pool, block_table, seq_lens, sink_buf, recent_buf, out, workspace, err_word,
                  softmax_scale: float, window: int, sinks: int = 0, lse=None, stream=None):
    """Attention of the last n tokens of every sequence, q [B][n][H][576] (or
    [B][H][576]: one), over the ``window`` tokens up to each one's own and the
    first ``sinks`` tokens (mla_lowbit_decode_window); writes ``out`` (float32
    or bf16) and ``lse``.  No length is read on the host."""
    if _native("decode_window", lay, q, page_pool, block_table, seq_lens, sink_buf, recent_buf, out, workspace, err_word,
               softmax_scale, window, sinks, lse, stream):
        return out
    torch = _torch()
    index, S, max_pages, num_pages = _expect_pool(lay, block_table, page_pool)
    if q is None or workspace is None:
        raise ValueError("q and workspace are required")
    if q.dim() not in (3, 4):
        raise ValueError("q must be [B][n][H][576] or [B][H][576]")
    code = _value_type(out)
    lead = tuple(q.shape)[:-1]
    if lead[0] != S:
        raise ValueError("block_table must have one row per sequence")
    packed = lay.content_bits != 16
    bf, f32, i32, u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
    qp, pool, table, lens, sink, recent, o, ls, ws, err = _pointers(index, (
        (q, "q", bf, lead + (576,)), (page_pool, "page_pool", u8, None), (block_table, "block_table", i32, None),
        (seq_lens, "seq_lens", i32, (S,)), (sink_buf if packed else None, "sink_buf", bf, (S, 4, 576) if packed else [None]),
        (recent_buf if packed else None, "recent_buf", bf, (S, 128, 576) if packed else [None]),
        (out, "out", out.dtype, lead + (512,)), (lse, "lse", f32, [lead]), (workspace, "workspace", u8, None),
        (err_word, "err_word", i32, (1,))))
    _launch(load().mla_lowbit_decode_window, "mla_lowbit_decode_window", index,
            (ctypes.byref(lay), S, lead[1] if len(lead) == 3 else 1, lead[-1], softmax_scale, _tokens(window, "window"),
             _tokens(sinks, "sinks"), qp, pool, num_pages, table, max_pages, lens, sink, recent, code, o, ls, ws,
             workspace.numel(), err), stream)
    return out


def set_fault_injection(mode: int, wait_cycles: int = 0) -> None:
    """Self-test setting of the tcgen05 kernels' bounded waits (process-wide):
    mode 1 withholds one hand-off so that the waits run out after
    ``wait_cycles`` SM cycles (0 = the default limit); mode 0 is normal."""
    _check(load().mla_lowbit_set_fault_injection(_int32(mode, "mode"), min(max(int(wait_cycles), -1), 2 ** 63 - 1)),
           "mla_lowbit_set_fault_injection")


def read_error(err_word) -> int:
    torch = _torch()
    code = ctypes.c_int32()
    with torch.cuda.device(err_word.device):
        _check(load().mla_lowbit_read_error(_ptr(err_word), ctypes.byref(code)),
               "mla_lowbit_read_error")
    return code.value
