"""GB300 (sm_103a) paged attention over a block-tabled KV cache.

A thin ctypes binding over the C ABI in ``include/pa.h`` (``libpa.so``, built
in-tree by ``paged_kv_attention_write_gb300/build.py``).  The Python functions
carry the C names and do argument marshalling only: shapes come from the
tensors, pointers from ``data_ptr()``, the stream from torch's current CUDA
stream.  Every step of the computation runs in the CUDA kernels; there is no
CPU fallback.  If the library is missing, importing this package fails.

Operations (see ``include/pa.h`` for layouts, ownership and error behaviour):

* ``pa_reshape_and_cache`` -- write fresh K/V to their cache slots;
* ``pa_decode`` -- one query token per sequence, split-K + log-sum-exp reduce;
* ``pa_prefill_chunk`` -- chunked prefill, causal in the chunk, full over the prefix;
* ``pa_copy_blocks`` -- whole-block copies for prefix-cache reuse;
* ``pa_reshape_and_cache_rope`` / ``pa_decode_rope`` -- the same with rotary position
  embedding (GPT-J pairs, YaRN table from ``pa_rope_yarn_freqs``) fused into the key write
  and the decode query load;
* ``pa_decode_window`` / ``pa_prefill_window`` -- the attention over a sliding window and the
  first tokens (sinks);
* ``pa_reshape_and_cache_rope_axes`` -- a step's queries and keys rotated with several position
  axes (``RopeAxes``, ``pa_rope_pair_axes``), keys and values written to their slots;
* ``pa_cross_attention`` -- rows of any number per sequence over its whole cached context (an
  encoder's states, images), each row within its own range of keys;
* ``pa_tables_extend`` / ``pa_tables_trim`` -- block tables, row starts, positions and slots made on
  the GPU from lengths, blocks taken from and given back to a free list in device memory.
"""
from __future__ import annotations

import ctypes
import struct
from pathlib import Path
from typing import Optional

import torch

__all__ = [
    "PAError", "pa_reshape_and_cache", "pa_decode_workspace_size", "pa_decode", "pa_decode_noalloc",
    "pa_prefill_chunk", "pa_copy_blocks", "pa_status_string", "pa_version", "library_path",
    "Rope", "pa_rope_yarn_freqs", "pa_reshape_and_cache_rope", "pa_decode_rope", "pa_decode_write",
    "pa_decode_window", "pa_prefill_window", "RopeAxes", "pa_rope_pair_axes", "pa_reshape_and_cache_rope_axes",
    "pa_cross_attention", "pa_tables_extend", "pa_tables_trim",
    "PA_F32", "PA_F16", "PA_BF16",
]

PA_F32, PA_F16, PA_BF16 = 0, 1, 2
_DTYPES = {torch.float32: PA_F32, torch.float16: PA_F16, torch.bfloat16: PA_BF16}

_LIB_PATH = Path(__file__).resolve().parent / "libpa.so"
if not _LIB_PATH.exists():
    raise ImportError(
        f"{_LIB_PATH} is missing: build the CUDA library first "
        "(python paged_kv_attention_write_gb300/build.py); there is no fallback")
_lib = ctypes.CDLL(str(_LIB_PATH))

_vp, _i32, _f32, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_lib.pa_reshape_and_cache.argtypes = [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32,
                                      _vp, _vp]
_lib.pa_decode_workspace_size.argtypes = [_i32, _i32, _i32, _i32, _i32]
_lib.pa_decode_workspace_size.restype = _sz
_lib.pa_decode.argtypes = [_vp, _i32, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32,
                           _i32, _i32, _f32, _i32, _vp, _sz, _vp, _vp]
_lib.pa_decode_noalloc.argtypes = [_vp, _i32, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32,
                                   _i32, _i32, _i32, _f32, _i32, _vp, _vp]
_lib.pa_prefill_chunk.argtypes = [_vp, _i32, _vp, _vp, _i32, _i32, _vp, _vp, _vp, _i32, _vp, _i32,
                                  _i32, _i32, _i32, _i32, _i32, _i32, _f32, _i32, _vp, _vp]
_lib.pa_copy_blocks.argtypes = [_vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _vp, _vp]
_lib.pa_decode_write.argtypes = [_vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32,
                                 _i32, _i32, _i32, _i32, _f32, _i32, _vp, _sz, _vp, _vp]
_lib.pa_status_string.argtypes = [_i32]
_lib.pa_status_string.restype = ctypes.c_char_p
_lib.pa_version.argtypes = []


class _PaRope(ctypes.Structure):
    _fields_ = [("freqs", _vp), ("rope_dim", _i32), ("q_scale_beta", _f32), ("q_scale_orig_ctx", _i32)]


_lib.pa_rope_yarn_freqs.argtypes = [_vp, _i32, _f32, _f32, _i32, _f32, _f32]
_lib.pa_reshape_and_cache_rope.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32,
                                           ctypes.POINTER(_PaRope), _vp, _vp]
_lib.pa_decode_rope.argtypes = [_vp, _i32, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32,
                                _i32, _i32, _f32, _i32, ctypes.POINTER(_PaRope), _vp, _sz, _vp, _vp]


def _send(name: str, f, record: struct.Struct, *fields) -> None:
    try:
        args = record.pack(*fields)
    except struct.error as e:  # not an integer, or one past 32 bits
        raise PAError(-1, f"{name}: {e}") from None
    rc = f(args)
    if rc != 0:
        raise PAError(rc, name)


# The windowed, multi-axis, cross and table calls go over as one packed record each (pa_window_args,
# pa_rope_axes_args, pa_cross_args, pa_tables_args): ctypes takes about as long for their twenty arguments as the launch does.
_WINDOW_ARGS = struct.Struct("@9P14if4x")
_ROPE_AXES_ARGS = struct.Struct("@12P3q10i")
_CROSS_ARGS = struct.Struct("@10P12if4x")
_TABLES_ARGS = struct.Struct("@12P6i")
for _name in ("pa_decode_window_args", "pa_prefill_window_args", "pa_reshape_and_cache_rope_axes_args",
              "pa_cross_attention_args", "pa_tables_extend_args", "pa_tables_trim_args"):
    getattr(_lib, _name).argtypes = [ctypes.c_char_p]
    getattr(_lib, _name).restype = _i32
_lib.pa_rope_pair_axes.argtypes = [_vp, _i32, _vp, _i32, _i32]
for _name in ("pa_reshape_and_cache", "pa_decode", "pa_decode_noalloc", "pa_prefill_chunk",
              "pa_copy_blocks", "pa_version", "pa_rope_yarn_freqs", "pa_reshape_and_cache_rope",
              "pa_decode_rope", "pa_decode_write", "pa_rope_pair_axes"):
    getattr(_lib, _name).restype = _i32


class PAError(RuntimeError):
    """A PA_ERR_* code returned by the C ABI."""

    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {pa_status_string(code)} ({code})")
        self.code = code


def library_path() -> Path:
    return _LIB_PATH


def pa_status_string(code: int) -> str:
    return _lib.pa_status_string(int(code)).decode()


def pa_version() -> int:
    return int(_lib.pa_version())


def _check(code: int, what: str) -> None:
    if code != 0:
        raise PAError(code, what)


def _dt(t: torch.Tensor) -> int:
    try:
        return _DTYPES[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {t.dtype}") from None


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def pa_reshape_and_cache(key, value, key_cache, value_cache, slot_mapping, *, status=None,
                         stream=None) -> None:
    """key/value ``[T][Hkv][D]`` -> pools ``[NB][bs][Hkv][D]`` at ``slot_mapping`` (int64)."""
    T, Hkv, D = key.shape
    NB, bs = key_cache.shape[:2]
    _check(_lib.pa_reshape_and_cache(_ptr(key), _ptr(value), _ptr(key_cache), _ptr(value_cache),
                                     _ptr(slot_mapping), T, Hkv, D, bs, NB, _dt(key_cache),
                                     _ptr(status), _stream(stream)), "pa_reshape_and_cache")


def pa_decode_workspace_size(num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int,
                             max_context_len: int) -> int:
    return int(_lib.pa_decode_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim,
                                             max_context_len))


def pa_decode(out, query, key_cache, value_cache, block_tables, context_lens, max_context_len: int,
              scale: float, *, workspace=None, status=None, stream=None) -> None:
    """out ``[S][Hq][D]`` = attention of query ``[S][Hq][D]`` over each sequence's cache."""
    S, Hq, D = query.shape
    NB, bs, Hkv, _ = key_cache.shape
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.pa_decode(_ptr(out), _dt(out), _ptr(query), _ptr(key_cache), _ptr(value_cache),
                          _ptr(block_tables), block_tables.shape[1], _ptr(context_lens),
                          int(max_context_len), S, Hq, Hkv, D, bs, NB, float(scale),
                          _dt(key_cache), _ptr(workspace), ws_bytes, _ptr(status),
                          _stream(stream)), "pa_decode")


def pa_decode_write(out, query, key, value, slot_mapping, key_cache, value_cache, block_tables,
                    context_lens, max_context_len: int, scale: float, *, workspace=None, status=None,
                    stream=None) -> None:
    """pa_reshape_and_cache of each sequence's new token (key / value ``[S][Hkv][D]`` to
    ``slot_mapping[s]``) and pa_decode, in one launch."""
    S, Hq, D = query.shape
    NB, bs, Hkv, _ = key_cache.shape
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.pa_decode_write(_ptr(out), _dt(out), _ptr(query), _ptr(key), _ptr(value), _ptr(slot_mapping),
                                _ptr(key_cache), _ptr(value_cache), _ptr(block_tables), block_tables.shape[1],
                                _ptr(context_lens), int(max_context_len), S, Hq, Hkv, D, bs, NB, float(scale),
                                _dt(key_cache), _ptr(workspace), ws_bytes, _ptr(status), _stream(stream)),
           "pa_decode_write")


def pa_decode_noalloc(out, query, key_cache, value_cache, block_tables, context_lens,
                      max_context_len: int, scale: float, *, status=None, stream=None) -> None:
    """pa_decode with the library's static scratch instead of a caller workspace, for
    callers that cannot allocate device memory.  Calls that overlap on the GPU race."""
    S, Hq, D = query.shape
    NB, bs, Hkv, _ = key_cache.shape
    _check(_lib.pa_decode_noalloc(_ptr(out), _dt(out), _ptr(query), _ptr(key_cache),
                                  _ptr(value_cache), _ptr(block_tables), block_tables.shape[1],
                                  _ptr(context_lens), int(max_context_len), S, Hq, Hkv, D, bs, NB,
                                  float(scale), _dt(key_cache), _ptr(status), _stream(stream)),
           "pa_decode_noalloc")


def pa_prefill_chunk(out, query, query_start_loc, max_query_len: int, key_cache, value_cache,
                     block_tables, context_lens, max_context_len: int, scale: float, *,
                     status=None, stream=None) -> None:
    """out ``[Tq][Hq][D]``: chunk rows attend their prefix and, causally, their chunk."""
    Tq, Hq, D = query.shape
    NB, bs, Hkv, _ = key_cache.shape
    S = context_lens.shape[0]
    _check(_lib.pa_prefill_chunk(_ptr(out), _dt(out), _ptr(query), _ptr(query_start_loc), Tq,
                                 int(max_query_len), _ptr(key_cache), _ptr(value_cache),
                                 _ptr(block_tables), block_tables.shape[1], _ptr(context_lens),
                                 int(max_context_len), S, Hq, Hkv, D, bs, NB, float(scale),
                                 _dt(key_cache), _ptr(status), _stream(stream)),
           "pa_prefill_chunk")


def pa_copy_blocks(key_cache, value_cache, block_mapping, *, status=None, stream=None) -> None:
    """Copy whole blocks (K and V) for each (src, dst) row of ``block_mapping`` (int64 [N][2])."""
    NB, bs, Hkv, D = key_cache.shape
    _check(_lib.pa_copy_blocks(_ptr(key_cache), _ptr(value_cache), _ptr(block_mapping),
                               block_mapping.shape[0], Hkv, D, bs, NB, _dt(key_cache),
                               _ptr(status), _stream(stream)), "pa_copy_blocks")


# ----------------------------------------------------------------------------- rotary embedding

def pa_rope_yarn_freqs(rope_dim: int, base: float, yarn_scale: float = 1.0, orig_ctx: int = 0,
                       beta_fast: float = 32.0, beta_slow: float = 1.0):
    """The RoPE frequency table (host, fp32 ``[rope_dim / 2]``), YaRN-corrected when
    ``yarn_scale != 1`` and ``orig_ctx > 0`` (``include/pa.h`` states the formula)."""
    import numpy as np
    out = np.empty(rope_dim // 2, dtype=np.float32)
    _check(_lib.pa_rope_yarn_freqs(out.ctypes.data, rope_dim, float(base), float(yarn_scale), int(orig_ctx),
                                   float(beta_fast), float(beta_slow)), "pa_rope_yarn_freqs")
    return out


class Rope:
    """Rotary-embedding arguments: ``freqs`` a device fp32 tensor ``[rope_dim / 2]``, the
    rotated width, and the position-dependent query scale (off when ``q_scale_orig_ctx`` is 0)."""

    def __init__(self, freqs: torch.Tensor, rope_dim: int, q_scale_beta: float = 0.0, q_scale_orig_ctx: int = 0):
        self.freqs, self.rope_dim = freqs, rope_dim
        self.q_scale_beta, self.q_scale_orig_ctx = q_scale_beta, q_scale_orig_ctx

    def _c(self):
        return _PaRope(self.freqs.data_ptr(), int(self.rope_dim), float(self.q_scale_beta), int(self.q_scale_orig_ctx))


def pa_reshape_and_cache_rope(key, value, key_cache, value_cache, slot_mapping, positions, rope: Rope, *,
                              status=None, stream=None) -> None:
    """pa_reshape_and_cache with each key row rotated at ``positions`` (int32 [T])."""
    T, Hkv, D = key.shape
    NB, bs = key_cache.shape[:2]
    r = rope._c()
    _check(_lib.pa_reshape_and_cache_rope(_ptr(key), _ptr(value), _ptr(key_cache), _ptr(value_cache),
                                          _ptr(slot_mapping), _ptr(positions), T, Hkv, D, bs, NB,
                                          _dt(key_cache), ctypes.byref(r), _ptr(status), _stream(stream)),
           "pa_reshape_and_cache_rope")


def pa_decode_rope(out, query, key_cache, value_cache, block_tables, context_lens, max_context_len: int,
                   scale: float, rope: Rope, *, workspace=None, status=None, stream=None) -> None:
    """pa_decode with the (unrotated) query rotated and scaled at position context_len - 1."""
    S, Hq, D = query.shape
    NB, bs, Hkv, _ = key_cache.shape
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    r = rope._c()
    _check(_lib.pa_decode_rope(_ptr(out), _dt(out), _ptr(query), _ptr(key_cache), _ptr(value_cache),
                               _ptr(block_tables), block_tables.shape[1], _ptr(context_lens),
                               int(max_context_len), S, Hq, Hkv, D, bs, NB, float(scale), _dt(key_cache),
                               ctypes.byref(r), _ptr(workspace), ws_bytes, _ptr(status), _stream(stream)),
           "pa_decode_rope")


# ----------------------------------------------------------------------------- sliding window

def _refuse(what: str, why: str) -> None:
    raise PAError(-1, f"{what}: {why}")


# The calls below run with their tensors' device current (a stream given must be of it) and,
# without a stream, on torch's current stream of that device.
_current_device = getattr(torch._C, "_cuda_getDevice", None)  # absent from builds without CUDA
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _check_window(what, out, query, key_cache, value_cache, tables, lens, starts, status):
    """Shapes, types, layout and device of the windowed calls' tensors; returns the shapes of
    query, key_cache and block_tables, the cache's dtype code and the device's index."""
    qs, ks, ts, ls = query.shape, key_cache.shape, tables.shape, lens.shape
    if len(qs) != 3 or len(ks) != 4 or len(ts) != 2 or len(ls) != 1:
        _refuse(what, "query is [T][Hq][D], a cache [NB][bs][Hkv][D], block_tables [S][max_blocks], lengths [S]")
    if out.shape != qs or value_cache.shape != ks or qs[2] != ks[3]:
        _refuse(what, "out is shaped as query, value_cache as key_cache, head dims are equal")
    dt, i32 = query.dtype, torch.int32
    if key_cache.dtype is not dt or value_cache.dtype is not dt:
        _refuse(what, "query and caches share one dtype")
    if tables.dtype is not i32 or lens.dtype is not i32:
        _refuse(what, "tables, lengths, starts and status are int32")
    rows = ls[0]
    if ts[0] != rows or (starts is None and qs[0] != rows):
        _refuse(what, "one table row and length per sequence, one query row each or S + 1 row starts")
    if not (out.is_contiguous() and query.is_contiguous() and key_cache.is_contiguous() and
            value_cache.is_contiguous() and tables.is_contiguous() and lens.is_contiguous()):
        _refuse(what, "tensors must be contiguous")
    dev = query.get_device()
    if dev < 0 or not (out.get_device() == dev == key_cache.get_device() == value_cache.get_device() ==
                       tables.get_device() == lens.get_device()):
        _refuse(what, "tensors must be on one CUDA device")
    if starts is not None:
        if starts.dtype is not i32:
            _refuse(what, "tables, lengths, starts and status are int32")
        if starts.shape != (rows + 1,):
            _refuse(what, "one table row and length per sequence, one query row each or S + 1 row starts")
        if not starts.is_contiguous():
            _refuse(what, "tensors must be contiguous")
        if starts.get_device() != dev:
            _refuse(what, "tensors must be on one CUDA device")
    if status is not None:
        if status.dtype is not i32 or status.numel() < 1:
            _refuse(what, "tables, lengths, starts and status are int32")
        if status.get_device() != dev:
            _refuse(what, "tensors must be on one CUDA device")
    code = _DTYPES.get(dt)
    if code is None:
        raise TypeError(f"unsupported dtype {dt}")
    return qs, ks, ts[1], code, dev


def pa_decode_window(out, query, key_cache, value_cache, block_tables, context_lens, max_context_len: int,
                     window: int, num_sinks: int, scale: float, *, status=None, stream=None) -> None:
    """pa_decode over the newest ``window`` keys and the first ``num_sinks`` of each sequence.
    No workspace; table entries of blocks that no key is seen in are not read."""
    (S, Hq, D), (NB, bs, Hkv, _), width, code, dev = _check_window(
        "pa_decode_window", out, query, key_cache, value_cache, block_tables, context_lens, None, status)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return pa_decode_window(out, query, key_cache, value_cache, block_tables, context_lens, max_context_len,
                                    window, num_sinks, scale, status=status, stream=stream)
    _send("pa_decode_window", _lib.pa_decode_window_args, _WINDOW_ARGS,
        out.data_ptr(), query.data_ptr(), key_cache.data_ptr(), value_cache.data_ptr(), 0, block_tables.data_ptr(),
        context_lens.data_ptr(), 0 if status is None else status.data_ptr(),
        _current_stream(dev) if stream is None else _stream(stream), _dt(out), code, S, 1, width, max_context_len,
        window, num_sinks, S, Hq, Hkv, D, bs, NB, scale)


def pa_prefill_window(out, query, query_start_loc, max_query_len: int, key_cache, value_cache, block_tables,
                      context_lens, max_context_len: int, window: int, num_sinks: int, scale: float, *, status=None,
                      stream=None) -> None:
    """pa_prefill_chunk over the newest ``window`` keys before each row and the first ``num_sinks``."""
    (Tq, Hq, D), (NB, bs, Hkv, _), width, code, dev = _check_window(
        "pa_prefill_window", out, query, key_cache, value_cache, block_tables, context_lens, query_start_loc, status)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return pa_prefill_window(out, query, query_start_loc, max_query_len, key_cache, value_cache, block_tables,
                                     context_lens, max_context_len, window, num_sinks, scale, status=status,
                                     stream=stream)
    _send("pa_prefill_window", _lib.pa_prefill_window_args, _WINDOW_ARGS,
        out.data_ptr(), query.data_ptr(), key_cache.data_ptr(), value_cache.data_ptr(), query_start_loc.data_ptr(),
        block_tables.data_ptr(), context_lens.data_ptr(), 0 if status is None else status.data_ptr(),
        _current_stream(dev) if stream is None else _stream(stream), _dt(out), code, Tq, max_query_len, width,
        max_context_len, window, num_sinks, context_lens.shape[0], Hq, Hkv, D, bs, NB, scale)


# ----------------------------------------------------------------------------- rotary axes

def pa_rope_pair_axes(rope_dim: int, sections, interleaved: bool = False):
    """The axis of each rotated pair (host, int32 ``[rope_dim / 2]``) from the pairs per axis:
    in order, or with ``interleaved`` dealt out in turn."""
    import numpy as np
    sec = np.ascontiguousarray(sections, dtype=np.int32)
    out = np.empty(max(0, rope_dim // 2), dtype=np.int32)
    _check(_lib.pa_rope_pair_axes(out.ctypes.data, int(rope_dim), sec.ctypes.data, int(sec.size), int(interleaved)),
           "pa_rope_pair_axes")
    return out


class RopeAxes:
    """Arguments of the multi-axis rotation: device tensors ``freqs`` (fp32) and ``pair_axis``
    (int32), both ``[rope_dim / 2]``, the number of axes, and whether pair i is the elements
    (i, i + rope_dim / 2) (``halves``) or (2i, 2i + 1)."""

    def __init__(self, freqs: torch.Tensor, pair_axis: torch.Tensor, rope_dim: int, num_axes: int,
                 halves: bool = False):
        shape = (rope_dim // 2,)
        if not (freqs.dtype is torch.float32 and pair_axis.dtype is torch.int32 and rope_dim % 2 == 0 and
                freqs.shape == shape and pair_axis.shape == shape and freqs.is_contiguous() and
                pair_axis.is_contiguous() and freqs.get_device() == pair_axis.get_device()):
            _refuse("RopeAxes", "freqs is fp32 and pair_axis int32, both [rope_dim / 2], dense, on one device")
        self.freqs, self.pair_axis = freqs, pair_axis
        self.rope_dim, self.num_axes, self.halves = int(rope_dim), int(num_axes), bool(halves)


def pa_reshape_and_cache_rope_axes(query_out, query, key, value, key_cache, value_cache, slot_mapping, positions,
                                   rope: RopeAxes, *, status=None, stream=None) -> None:
    """query ``[T][Hq][D]`` rotated into ``query_out`` (dense; may be ``query``), key ``[T][Hkv][D]``
    rotated and value copied into the pools at ``slot_mapping`` (int64 [T]), at ``positions``
    (int32 [num_axes][T]).  query, key and value may be slices of wider rows.  ``query`` and
    ``query_out`` None: keys and values only."""
    what = "pa_reshape_and_cache_rope_axes"
    if (query is None) != (query_out is None):
        _refuse(what, "query and query_out go together")
    shape, ks = key.shape, key_cache.shape
    if len(shape) != 3 or len(ks) != 4 or value.shape != shape or value_cache.shape != ks:
        _refuse(what, "key and value are [T][Hkv][D], a cache [NB][bs][Hkv][D]")
    (T, Hkv, D), (NB, bs, ch, cd), dt, dev = shape, ks, key.dtype, key.get_device()
    if Hkv != ch or D != cd:
        _refuse(what, "key and value are [T][Hkv][D], a cache [NB][bs][Hkv][D]")
    one_device = (dev >= 0 and value.get_device() == dev == key_cache.get_device() == value_cache.get_device() ==
                  slot_mapping.get_device() == positions.get_device() == rope.freqs.get_device())
    Hq = q_stride = 0
    if query is not None:
        qs = query.shape
        if len(qs) != 3 or query_out.shape != qs:
            _refuse(what, "query and query_out are [T][Hq][D]")
        rows, Hq, width = qs
        if rows != T or width != D:
            _refuse(what, "query and query_out are [T][Hq][D]")
        q_stride, q_head, q_one = query.stride()
        if query.dtype is not dt or query_out.dtype is not dt:
            _refuse(what, "query, keys, values and caches share one dtype")
        if T and (q_one != 1 or (Hq > 1 and q_head != D)):
            _refuse(what, "a token's heads must be contiguous")
        if not query_out.is_contiguous():
            _refuse(what, "caches, query_out, slots and positions must be contiguous")
        one_device = one_device and query.get_device() == dev == query_out.get_device()
    if value.dtype is not dt or key_cache.dtype is not dt or value_cache.dtype is not dt:
        _refuse(what, "query, keys, values and caches share one dtype")
    if slot_mapping.dtype is not torch.int64 or slot_mapping.shape != (T,) or positions.dtype is not torch.int32 or (
            positions.shape != (rope.num_axes, T)) or (
            status is not None and (status.dtype is not torch.int32 or status.numel() < 1)):
        _refuse(what, "slot_mapping is int64 [T], positions int32 [num_axes][T], status int32 [1]")
    if not (key_cache.is_contiguous() and value_cache.is_contiguous() and slot_mapping.is_contiguous() and
            positions.is_contiguous()):
        _refuse(what, "caches, query_out, slots and positions must be contiguous")
    k_stride, k_head, k_one = key.stride()
    v_stride, v_head, v_one = value.stride()
    if T and (k_one != 1 or v_one != 1 or (Hkv > 1 and (k_head != D or v_head != D))):
        _refuse(what, "a token's heads must be contiguous")
    if not one_device or (status is not None and status.get_device() != dev):
        _refuse(what, "tensors must be on one CUDA device")
    code = _DTYPES.get(dt)
    if code is None:
        raise TypeError(f"unsupported dtype {dt}")
    if dev != _current_device():
        with torch.cuda.device(dev):
            return pa_reshape_and_cache_rope_axes(query_out, query, key, value, key_cache, value_cache, slot_mapping,
                                                  positions, rope, status=status, stream=stream)
    _send(what, _lib.pa_reshape_and_cache_rope_axes_args, _ROPE_AXES_ARGS,
        0 if query is None else query_out.data_ptr(), 0 if query is None else query.data_ptr(), key.data_ptr(),
        value.data_ptr(), key_cache.data_ptr(), value_cache.data_ptr(), slot_mapping.data_ptr(), positions.data_ptr(),
        rope.freqs.data_ptr(), rope.pair_axis.data_ptr(), 0 if status is None else status.data_ptr(),
        _current_stream(dev) if stream is None else _stream(stream), q_stride, k_stride, v_stride, T, Hq, Hkv, D,
        bs, NB, code, rope.rope_dim, rope.num_axes, rope.halves)


# ----------------------------------------------------------------------------- cross attention

def pa_cross_attention(out, query, query_start_loc, max_query_len: int, key_cache, value_cache, block_tables,
                       context_lens, max_context_len: int, scale: float, *, key_ranges=None, status=None,
                       stream=None) -> None:
    """out ``[T][Hq][D]`` = attention of query ``[T][Hq][D]`` over each sequence's whole cached context.
    ``query_start_loc`` (int32 [S + 1]) gives each sequence's rows; None: one row per sequence.
    ``key_ranges`` (int32 [T][2]): row t sees the keys from ``[t][0]`` up to, not including, ``[t][1]``."""
    what = "pa_cross_attention"
    (T, Hq, D), (NB, bs, Hkv, _), width, code, dev = _check_window(
        what, out, query, key_cache, value_cache, block_tables, context_lens, query_start_loc, status)
    if key_ranges is not None:
        if key_ranges.dtype is not torch.int32 or key_ranges.shape != (T, 2) or not key_ranges.is_contiguous():
            _refuse(what, "key_ranges is int32 [T][2], contiguous")
        if key_ranges.get_device() != dev:
            _refuse(what, "tensors must be on one CUDA device")
    if dev != _current_device():
        with torch.cuda.device(dev):
            return pa_cross_attention(out, query, query_start_loc, max_query_len, key_cache, value_cache, block_tables,
                                      context_lens, max_context_len, scale, key_ranges=key_ranges, status=status,
                                      stream=stream)
    _send(what, _lib.pa_cross_attention_args, _CROSS_ARGS,
        out.data_ptr(), query.data_ptr(), key_cache.data_ptr(), value_cache.data_ptr(),
        0 if query_start_loc is None else query_start_loc.data_ptr(), 0 if key_ranges is None else key_ranges.data_ptr(),
        block_tables.data_ptr(), context_lens.data_ptr(), 0 if status is None else status.data_ptr(),
        _current_stream(dev) if stream is None else _stream(stream), _dt(out), code, T, max_query_len, width,
        max_context_len, context_lens.shape[0], Hq, Hkv, D, bs, NB, scale)


# ----------------------------------------------------------------------------- tables on the GPU

_TABLES_TYPES = "tensors are int32 (slot_mapping int64) and contiguous"
_TABLES_SHAPES = "block_tables is [S][max_blocks], lengths are [S], query_start_loc [S + 1], counts [1], positions [T]"


def _check_tables(what, tables, a, b, c, free, n_in, n_out, status):
    """Types, layout, sizes and device of the tensors that both table calls take (``a``, ``b``, ``c``: lengths);
    returns S, the table's width and the device's index.  Spelled out: the calls are a few
    microseconds long, and a loop over the tensors costs one of them."""
    i32, dev = torch.int32, tables.get_device()
    if not (tables.dtype is i32 and a.dtype is i32 and b.dtype is i32 and c.dtype is i32 and free.dtype is i32 and
            n_in.dtype is i32 and n_out.dtype is i32 and tables.is_contiguous() and a.is_contiguous() and
            b.is_contiguous() and c.is_contiguous() and free.is_contiguous()):
        _refuse(what, _TABLES_TYPES)
    if not (dev >= 0 and a.get_device() == dev == b.get_device() == c.get_device() and free.get_device() == dev and
            n_in.get_device() == dev == n_out.get_device()):
        _refuse(what, "tensors must be on one CUDA device")
    shape = tables.shape
    if len(shape) != 2:
        _refuse(what, _TABLES_SHAPES)
    S, width = shape
    if not (a.numel() == S == b.numel() == c.numel()) or n_in.numel() < 1 or n_out.numel() < 1:
        _refuse(what, _TABLES_SHAPES)
    if status is not None and (status.dtype is not i32 or status.numel() < 1 or status.get_device() != dev):
        _refuse(what, "status is int32 [1] on the tensors' device")
    return S, width, dev


def pa_tables_extend(block_tables, context_lens, query_start_loc, positions, slot_mapping, num_free_out, cached_lens,
                     new_lens, free_blocks, num_free, block_size: int, num_blocks: int, *, status=None,
                     stream=None) -> None:
    """Sequences grow from ``cached_lens`` to ``cached_lens + new_lens`` tokens (int32 [S]): blocks taken
    from the stack ``free_blocks[:num_free]`` enter ``block_tables`` [S][max_blocks]; ``context_lens`` [S],
    ``query_start_loc`` [S + 1] and ``positions`` [T] (either may be None), ``slot_mapping`` (int64 [T], -1
    behind the last token) and ``num_free_out`` [1] are written."""
    what = "pa_tables_extend"
    S, width, dev = _check_tables(what, block_tables, context_lens, cached_lens, new_lens, free_blocks, num_free,
                                  num_free_out, status)
    T = slot_mapping.numel()
    if slot_mapping.dtype is not torch.int64 or not slot_mapping.is_contiguous() or slot_mapping.get_device() != dev:
        _refuse(what, _TABLES_TYPES)
    starts = 0
    if query_start_loc is not None:
        if query_start_loc.dtype is not torch.int32 or not query_start_loc.is_contiguous() or (
                query_start_loc.get_device() != dev):
            _refuse(what, _TABLES_TYPES)
        if query_start_loc.numel() != S + 1:
            _refuse(what, _TABLES_SHAPES)
        starts = query_start_loc.data_ptr()
    at = 0
    if positions is not None:
        if positions.dtype is not torch.int32 or not positions.is_contiguous() or positions.get_device() != dev:
            _refuse(what, _TABLES_TYPES)
        if positions.numel() != T:
            _refuse(what, _TABLES_SHAPES)
        at = positions.data_ptr()
    if dev != _current_device():
        with torch.cuda.device(dev):
            return pa_tables_extend(block_tables, context_lens, query_start_loc, positions, slot_mapping, num_free_out,
                                    cached_lens, new_lens, free_blocks, num_free, block_size, num_blocks,
                                    status=status, stream=stream)
    _send(what, _lib.pa_tables_extend_args, _TABLES_ARGS,
        block_tables.data_ptr(), context_lens.data_ptr(), starts, at, slot_mapping.data_ptr(), free_blocks.data_ptr(),
        num_free_out.data_ptr(), cached_lens.data_ptr(), new_lens.data_ptr(), num_free.data_ptr(),
        0 if status is None else status.data_ptr(), _current_stream(dev) if stream is None else _stream(stream), S,
        width, T, free_blocks.numel(), block_size, num_blocks)


def pa_tables_trim(free_blocks, context_lens, num_free_out, block_tables, cached_lens, keep_lens, num_free,
                   block_size: int, num_blocks: int, *, status=None, stream=None) -> None:
    """Sequences shrink from ``cached_lens`` to ``keep_lens`` tokens (int32 [S]; 0: ended): the blocks that
    they no longer need go onto the stack ``free_blocks`` behind its ``num_free`` entries; ``context_lens``
    [S] and ``num_free_out`` [1] are written."""
    what = "pa_tables_trim"
    S, width, dev = _check_tables(what, block_tables, context_lens, cached_lens, keep_lens, free_blocks, num_free,
                                  num_free_out, status)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return pa_tables_trim(free_blocks, context_lens, num_free_out, block_tables, cached_lens, keep_lens,
                                  num_free, block_size, num_blocks, status=status, stream=stream)
    _send(what, _lib.pa_tables_trim_args, _TABLES_ARGS,
        block_tables.data_ptr(), context_lens.data_ptr(), 0, 0, 0, free_blocks.data_ptr(), num_free_out.data_ptr(),
        cached_lens.data_ptr(), keep_lens.data_ptr(), num_free.data_ptr(), 0 if status is None else status.data_ptr(),
        _current_stream(dev) if stream is None else _stream(stream), S, width, 0, free_blocks.numel(), block_size,
        num_blocks)
