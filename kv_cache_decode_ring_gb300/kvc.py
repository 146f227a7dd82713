"""ctypes binding of ``libkvc.so`` (``include/kvc.h``): argument marshalling only.

Every function has the name of the C entry point it calls and raises
:class:`KvcError` on a non-zero status.  Device arguments are torch CUDA tensors
(checked for device, dtype, shape and contiguity here, then passed as raw
pointers); the stream defaults to torch's current stream.  All computation runs
in the library's kernels; if the library has not been built this module raises
on first use -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import threading
from array import array
from typing import Optional, Sequence

import numpy as np
import torch

from . import build as _build

KVC_OK, KVC_ERR_ARG, KVC_ERR_CAPACITY, KVC_ERR_EVICTED, KVC_ERR_CUDA, KVC_ERR_UNSUPPORTED, KVC_ERR_DEVICE = range(7)
KVC_F32, KVC_BF16 = 0, 1
KVC_CONTIGUOUS, KVC_RING = 0, 1
KVC_QUANT_NONE, KVC_QUANT_INT8, KVC_QUANT_INT8_DITHER, KVC_QUANT_INT4 = 0, 1, 2, 3
(KVC_EXPORT_K, KVC_EXPORT_V, KVC_EXPORT_POSITIONS, KVC_EXPORT_NEXT_POSITION, KVC_EXPORT_KQ, KVC_EXPORT_VQ,
 KVC_EXPORT_SK, KVC_EXPORT_SV, KVC_EXPORT_WITNESS, KVC_EXPORT_KTAIL, KVC_EXPORT_VTAIL, KVC_EXPORT_XMAP,
 KVC_EXPORT_PAGE_TABLE, KVC_EXPORT_K4, KVC_EXPORT_V4) = range(15)
KVC_ROPE_HALVES, KVC_ROPE_PER_AXIS = 1, 2

_STATUS_NAMES = {1: "KVC_ERR_ARG", 2: "KVC_ERR_CAPACITY", 3: "KVC_ERR_EVICTED", 4: "KVC_ERR_CUDA",
                 5: "KVC_ERR_UNSUPPORTED", 6: "KVC_ERR_DEVICE"}


class KvcError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__("%s: %s (%s)" % (where, _STATUS_NAMES.get(code, code), kvc_strerror(code)))


class kvc_config(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("layout", ctypes.c_int32), ("kv_quant", ctypes.c_int32),
                ("batch", ctypes.c_int32), ("n_q_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("capacity", ctypes.c_int32), ("window", ctypes.c_int32),
                ("max_position", ctypes.c_int32), ("rope_base", ctypes.c_float), ("max_chunk", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("int8_exact_blocks", ctypes.c_int32), ("page_pool", ctypes.c_int32),
                ("store_slots", ctypes.c_int32), ("layer_index", ctypes.c_int32),
                ("dither_key_lo", ctypes.c_uint32), ("dither_key_hi", ctypes.c_uint32),
                ("int8_split", ctypes.c_int32), ("sinks", ctypes.c_int32)]


EXPORTED = ["kvc_state_bytes", "kvc_create", "kvc_destroy", "kvc_append", "kvc_append_rows",
            "kvc_decode_attn", "kvc_trim", "kvc_chunk_attn", "kvc_export_bytes", "kvc_export",
            "kvc_next_positions", "kvc_device_status", "kvc_prefix_cut", "kvc_strerror",
            "kvc_int8_block_risk", "kvc_int8_gate", "kvc_int8_restore",
            "kvc_pstore_create", "kvc_pstore_destroy", "kvc_pstore_insert", "kvc_pstore_lookup",
            "kvc_store_save", "kvc_store_load", "kvc_store_load_batch", "kvc_set_request_id",
            "kvc_check_wait_path", "kvc_prompt_attn", "kvc_fork", "kvc_copy", "kvc_free", "kvc_compact",
            "kvc_page_counts", "kvc_region", "kvc_rope_axes"]

_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _build.LIB


def lib() -> ctypes.CDLL:
    """The loaded library.  Raises if it has not been built (no fallback path exists)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = library_path()
            if not os.path.exists(path):
                raise RuntimeError("libkvc.so is not built (%s); run kv_cache_decode_ring_gb300.build.build()" % path)
            L = ctypes.CDLL(path)
            P, i32, i64, u64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
            cfgp = ctypes.POINTER(kvc_config)
            sig = {
                "kvc_state_bytes": [cfgp, ctypes.POINTER(u64)],
                "kvc_create": [cfgp, P, u64, P, ctypes.POINTER(P)],
                "kvc_destroy": [P],
                "kvc_append": [P, P, P, P],
                "kvc_append_rows": [P, P, P, i32, P, P],
                "kvc_decode_attn": [P, P, P, P, P, P, P],
                "kvc_trim": [P, P, P],
                "kvc_chunk_attn": [P, P, P, P, i32, P, P],
                "kvc_export_bytes": [P, i32, ctypes.POINTER(u64)],
                "kvc_export": [P, i32, P, u64, P],
                "kvc_next_positions": [P, P],
                "kvc_device_status": [P, P, ctypes.POINTER(i32)],
                "kvc_prefix_cut": [P, i32, P, i32, i32, ctypes.POINTER(i32)],
                "kvc_decode_attn_noalloc": [P, P, P, P],
                "kvc_int8_block_risk": [P, P, P, P],
                "kvc_int8_gate": [P, i32, i32, i32, ctypes.c_double, i32, P, ctypes.POINTER(i32)],
                "kvc_int8_restore": [P, P, i32, P, P, P],
                "kvc_pstore_create": [cfgp, i32, ctypes.POINTER(P)],
                "kvc_pstore_destroy": [P],
                "kvc_pstore_insert": [P, P, i32, ctypes.c_char_p, P, i32, ctypes.POINTER(i32)],
                "kvc_pstore_lookup": [P, P, i32, ctypes.c_char_p, P, i32, ctypes.POINTER(i32), ctypes.POINTER(i32)],
                "kvc_store_save": [P, i32, i32, i32, P],
                "kvc_store_load": [P, i32, i32, i32, P],
                "kvc_store_load_batch": [P, i32, P, P, P, P],
                "kvc_set_request_id": [P, i32, ctypes.c_uint32, P],
                "kvc_check_wait_path": [P, P],
                "kvc_prompt_attn": [P, P, i64, P, P, i64, P, P, P],
                "kvc_fork": [P, i32, P, P, P],
                "kvc_copy": [P, P, i32, P, P, P],
                "kvc_free": [P, i32, P, P],
                "kvc_compact": [P, ctypes.POINTER(i32), P],
                "kvc_page_counts": [P, ctypes.POINTER(i32), ctypes.POINTER(i32)],
                "kvc_region": [P, i32, ctypes.POINTER(u64), ctypes.POINTER(u64)],
                "kvc_rope_axes": [P, i64, P, i64, i32, i64, i32, i32, P, i32, P, ctypes.c_double, i32, P],
            }
            for name, args in sig.items():
                fn = getattr(L, name)
                fn.argtypes = args
                fn.restype = ctypes.c_int
            L.kvc_strerror.argtypes = [ctypes.c_int]
            L.kvc_strerror.restype = ctypes.c_char_p
            _lib = L
    return _lib


def _check(rc: int, where: str):
    if rc != KVC_OK:
        raise KvcError(rc, where)


def _stream(stream) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """A new tensor in memory of ``stream``, which will write it: memory of the current stream may still
    be in use there by work enqueued before its last owner let go of it.  The current stream, where the
    caller goes on with it, is recorded: its work is over before the memory is handed out again."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    device = torch.device(device)
    raw = _stream(stream)
    index = torch.cuda.current_device() if device.index is None else device.index
    if raw == torch._C._cuda_getCurrentRawStream(index):
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        # (1 is the legacy default stream by its special handle)
        stream = torch.cuda.default_stream(index) if raw in (0, 1) else torch.cuda.ExternalStream(raw, index)
    with torch.cuda.stream(stream):
        out = torch.empty(shape, dtype=dtype, device=device)
    out.record_stream(torch.cuda.current_stream(index))
    return out


def _dev(t: Optional[torch.Tensor], dtype=None, shape=None, name="tensor") -> ctypes.c_void_p:
    if t is None:
        return ctypes.c_void_p(0)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    return ctypes.c_void_p(t.data_ptr())


def kvc_strerror(code: int) -> str:
    return lib().kvc_strerror(int(code)).decode()


def make_config(dtype="bf16", layout="contiguous", kv_quant=None, batch=1, n_q_heads=1, n_kv_heads=1,
                head_dim=128, capacity=1, window=0, max_position=0, rope_base=0.0, max_chunk=0,
                out_dtype=None, int8_exact_blocks=0, page_pool=0, store_slots=0, layer_index=0,
                dither_key=(0, 0), int8_split=0, sinks=0) -> kvc_config:
    """``out_dtype``: None (the cache dtype), "f32" or "bf16"; ``int8_exact_blocks``: pool
    entries for blocks the gated fallback restores (INT8 caches); ``page_pool``: pages of 16
    slots for paged K/V storage (0 = each request owns ``capacity`` slots); ``store_slots``:
    device slots for saved prefills (prefix store).  ``kv_quant``: None, "int8" (witness
    tier), "int4" (4-bit rows) or "int8-dither" (Tier B, with ``layer_index`` and the 64-bit Philox ``dither_key``
    as (low, high) words); ``int8_split``: positions per quantized split of the INT8 decode
    (a multiple of 64 in [1024, 2048]; 0 = chosen for the device); ``sinks``: first positions that stay
    visible behind a window (contiguous caches but INT8)."""
    od = 0 if out_dtype is None else (KVC_F32 + 1 if out_dtype == "f32" else KVC_BF16 + 1)
    return kvc_config(KVC_BF16 if dtype == "bf16" else KVC_F32,
                      KVC_RING if layout == "ring" else KVC_CONTIGUOUS,
                      {None: KVC_QUANT_NONE, "int8": KVC_QUANT_INT8, "int8-dither": KVC_QUANT_INT8_DITHER,
                       "int4": KVC_QUANT_INT4}[kv_quant],
                      batch, n_q_heads, n_kv_heads, head_dim, capacity, window, max_position,
                      float(rope_base), max_chunk, od, int(int8_exact_blocks), int(page_pool), int(store_slots),
                      int(layer_index), int(dither_key[0]) & 0xFFFFFFFF, int(dither_key[1]) & 0xFFFFFFFF,
                      int(int8_split), int(sinks))


def kvc_state_bytes(cfg: kvc_config) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().kvc_state_bytes(ctypes.byref(cfg), ctypes.byref(n)), "kvc_state_bytes")
    return n.value


def kvc_create(cfg: kvc_config, state: torch.Tensor, stream=None) -> ctypes.c_void_p:
    h = ctypes.c_void_p(0)
    _check(lib().kvc_create(ctypes.byref(cfg), _dev(state, name="state"), state.numel() * state.element_size(),
                            _stream(stream), ctypes.byref(h)), "kvc_create")
    return h


def kvc_destroy(h) -> None:
    _check(lib().kvc_destroy(h), "kvc_destroy")


def kvc_append(h, k: torch.Tensor, v: torch.Tensor, stream=None) -> None:
    _check(lib().kvc_append(h, _dev(k, name="k"), _dev(v, name="v"), _stream(stream)), "kvc_append")


def kvc_append_rows(h, k: torch.Tensor, v: torch.Tensor, n: int, counts: Optional[Sequence[int]] = None,
                    stream=None) -> None:
    c = None if counts is None else _whole(counts)
    _check(lib().kvc_append_rows(h, _dev(k, name="k"), _dev(v, name="v"), int(n), None if c is None else _at(c), _stream(stream)),
           "kvc_append_rows")


def kvc_decode_attn(h, q, out, cmax=None, tanh=None, ct=None, stream=None) -> None:
    bounds = [None if t is None else _dev(t, torch.float32, name=n) for t, n in ((cmax, "cmax"), (tanh, "tanh"), (ct, "ct"))]
    _check(lib().kvc_decode_attn(h, _dev(q, name="q"), _dev(out, name="out"), *bounds, _stream(stream)), "kvc_decode_attn")


def kvc_int8_block_risk(h, ct, risk, stream=None) -> None:
    _check(lib().kvc_int8_block_risk(h, _dev(ct, torch.float32, name="ct"), _dev(risk, torch.float32, name="risk"),
                                     _stream(stream)), "kvc_int8_block_risk")


def kvc_int8_gate(risk: np.ndarray, tau: float, max_blocks: int) -> np.ndarray:
    """Host selection: [n, 3] int32 (request, KV head, block) triples, highest risk first."""
    r = np.ascontiguousarray(np.asarray(risk, dtype=np.float32))
    if r.ndim != 3:
        raise ValueError("risk must be [B, Hkv, nblk]")
    sel = np.zeros((max(int(max_blocks), 1), 3), dtype=np.int32)
    n = ctypes.c_int32(0)
    _check(lib().kvc_int8_gate(r.ctypes.data_as(ctypes.c_void_p), r.shape[0], r.shape[1], r.shape[2],
                               ctypes.c_double(tau), int(max_blocks), sel.ctypes.data_as(ctypes.c_void_p),
                               ctypes.byref(n)), "kvc_int8_gate")
    return sel[:n.value].copy()


def kvc_int8_restore(h, blocks, k_full, v_full, stream=None) -> None:
    b = np.ascontiguousarray(np.asarray(blocks, dtype=np.int32).reshape(-1, 3))
    _check(lib().kvc_int8_restore(h, b.ctypes.data_as(ctypes.c_void_p) if len(b) else None, len(b),
                                  _dev(k_full, torch.bfloat16, name="k_full"),
                                  _dev(v_full, torch.bfloat16, name="v_full"), _stream(stream)), "kvc_int8_restore")


KVC_NOALLOC_SCRATCH_BYTES = 64 << 20


def kvc_decode_attn_noalloc(h, q, out, stream=None) -> None:
    """Decode attention whose split-K scratch is the library's fixed device array.

    For callers that cannot allocate device memory while they decode; see
    include/kvc.h.  Calls that overlap on the GPU share (and race on) that array."""
    _check(lib().kvc_decode_attn_noalloc(h, _dev(q, name="q"), _dev(out, name="out"), _stream(stream)),
           "kvc_decode_attn_noalloc")


def kvc_trim(h, cuts: Sequence[int], stream=None) -> None:
    c = _whole(cuts)
    _check(lib().kvc_trim(h, _at(c), _stream(stream)), "kvc_trim")


def kvc_chunk_attn(h, q, k, v, n: int, out, stream=None) -> None:
    _check(lib().kvc_chunk_attn(h, _dev(q, name="q"), _dev(k, name="k"), _dev(v, name="v"), int(n),
                                _dev(out, name="out"), _stream(stream)), "kvc_chunk_attn")


def _rows(t: torch.Tensor, name="tensor") -> tuple:
    """(pointer, row stride) of rows [n, heads, d] whose heads are dense; the row stride is free."""
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dim() != 3:
        raise ValueError("%s must have shape [rows, heads, head_dim], got %s" % (name, tuple(t.shape)))
    (n, heads, d), (row, head, dim) = t.shape, t.stride()
    if (d > 1 and dim != 1) or (heads > 1 and head != d) or (n > 1 and row < heads * d):
        raise ValueError("%s must have dense heads in each row, got strides %s" % (name, t.stride()))
    return t.data_ptr(), row if n > 1 else heads * d


def _ints(values):
    """Host int32 array (keep it alive during the call; its address is ``buffer_info()[0]``)."""
    return values if isinstance(values, array) and values.typecode == "i" else array("i", values)


def _whole(values):
    """_ints of any numbers, fractions cut off."""
    try:
        return _ints(values)
    except TypeError:
        return array("i", [int(x) for x in values])


def _at(a: array) -> int:
    return a.buffer_info()[0]


def kvc_prompt_attn(h, q, k, v, counts: Sequence[int], out, stream=None) -> None:
    """Packed prompts: q [T, Hq, d], k and v [T, Hkv, d] (row strides are free, k's equal to v's),
    ``counts`` rows of each request in turn; out [T, Hq, d] dense.  See include/kvc.h."""
    (qp, qs), (kp, ks), (vp, vs) = _rows(q, "q"), _rows(k, "k"), _rows(v, "v")
    if ks != vs:
        raise ValueError("k and v must have the same row stride")
    c = _ints(counts)
    _check(lib().kvc_prompt_attn(h, qp, qs, kp, vp, ks, _at(c), _dev(out, name="out"), _stream(stream)), "kvc_prompt_attn")


def _pairs(src, dst) -> tuple:
    s, d = _ints(src), _ints(dst)
    if len(s) != len(d):
        raise ValueError("src and dst must have one entry per request")
    return s, d


def kvc_fork(h, src: Sequence[int], dst: Sequence[int], stream=None) -> None:
    s, d = _pairs(src, dst)
    _check(lib().kvc_fork(h, len(s), _at(s), _at(d), _stream(stream)), "kvc_fork")


def kvc_copy(to, frm, src: Sequence[int], dst: Sequence[int], stream=None) -> None:
    s, d = _pairs(src, dst)
    _check(lib().kvc_copy(to, frm, len(s), _at(s), _at(d), _stream(stream)), "kvc_copy")


def kvc_free(h, requests: Sequence[int], stream=None) -> None:
    r = _ints(requests)
    _check(lib().kvc_free(h, len(r), _at(r), _stream(stream)), "kvc_free")


def kvc_compact(h, stream=None) -> int:
    """Pages in use after the call; they lie at [0, that many) of the pool."""
    n = ctypes.c_int32(0)
    _check(lib().kvc_compact(h, ctypes.byref(n), _stream(stream)), "kvc_compact")
    return n.value


def kvc_page_counts(h) -> tuple:
    """(free pages, pages that more than one request holds)."""
    free, shared = ctypes.c_int32(0), ctypes.c_int32(0)
    _check(lib().kvc_page_counts(h, ctypes.byref(free), ctypes.byref(shared)), "kvc_page_counts")
    return free.value, shared.value


def kvc_region(h, which: int) -> tuple:
    """(byte offset, bytes) of a stored array inside the state buffer."""
    off, n = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(lib().kvc_region(h, int(which), ctypes.byref(off), ctypes.byref(n)), "kvc_region")
    return off.value, n.value


_ROPE_DTYPES = {torch.bfloat16: KVC_BF16, torch.float32: KVC_F32}


def kvc_rope_axes(x, pos, sections: Sequence[int], base: float = 10000.0, out=None, halves=False, per_axis=False,
                  stream=None):
    """x [rows, heads, d] (bf16 or fp32, heads dense, row stride free) rotated by several axes:
    ``pos`` int32 [axes, rows], ``sections`` the pairs of each axis.  ``out`` may be x; a new dense
    tensor (memory of ``stream``) if None.  ``halves``: pairs (p, P + p) instead of (2p, 2p + 1);
    ``per_axis``: a spectrum for each axis.  See include/kvc.h."""
    dtype = _ROPE_DTYPES.get(x.dtype)
    if dtype is None:
        raise ValueError("x must be bfloat16 or float32, got %s" % x.dtype)
    xp, xs = _rows(x, "x")
    rows, heads, d = shape = x.shape
    if out is None:
        out = _empty(shape, x.dtype, x.device, stream)
    elif out.dtype != x.dtype or out.shape != shape:
        raise ValueError("out must be %s of shape %s" % (x.dtype, tuple(shape)))
    yp, ys = (xp, xs) if out is x else _rows(out, "out")
    s = _ints(sections)
    pp = _dev(pos, torch.int32, (len(s), rows), "pos")
    device = x.get_device()
    if not device == out.get_device() == pos.get_device():
        raise ValueError("x, pos and out must be on one device")
    flags = (KVC_ROPE_HALVES if halves else 0) | (KVC_ROPE_PER_AXIS if per_axis else 0)
    if device != torch._C._cuda_getDevice():
        with torch.cuda.device(device):
            return kvc_rope_axes(x, pos, s, base, out, halves, per_axis, stream)
    st = torch._C._cuda_getCurrentRawStream(device) if stream is None else _stream(stream)
    rc = lib().kvc_rope_axes(xp, xs, yp, ys, dtype, rows, heads, d, pp, len(s), s.buffer_info()[0], base, flags, st)
    if rc:
        _check(rc, "kvc_rope_axes")
    return out


def kvc_export_bytes(h, which: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().kvc_export_bytes(h, int(which), ctypes.byref(n)), "kvc_export_bytes")
    return n.value


def kvc_export(h, which: int, stream=None) -> np.ndarray:
    """Raw bytes of one state array (uint8); callers view them with the documented dtype."""
    n = kvc_export_bytes(h, which)
    buf = np.empty(n, dtype=np.uint8)
    _check(lib().kvc_export(h, int(which), buf.ctypes.data_as(ctypes.c_void_p), n, _stream(stream)), "kvc_export")
    return buf


def kvc_next_positions(h, batch: int) -> np.ndarray:
    out = np.empty(batch, dtype=np.int32)
    _check(lib().kvc_next_positions(h, out.ctypes.data_as(ctypes.c_void_p)), "kvc_next_positions")
    return out


def kvc_device_status(h, stream=None) -> int:
    s = ctypes.c_int32(0)
    _check(lib().kvc_device_status(h, _stream(stream), ctypes.byref(s)), "kvc_device_status")
    return s.value


def kvc_check_wait_path(h, stream=None) -> None:
    _check(lib().kvc_check_wait_path(h, _stream(stream)), "kvc_check_wait_path")


def kvc_prefix_cut(old_ids: Sequence[int], new_ids: Sequence[int], ring: bool = False) -> int:
    for x in list(old_ids) + list(new_ids):
        if isinstance(x, bool) or not isinstance(x, (int, np.integer)):
            raise TypeError("token IDs must be integers")
    o = np.ascontiguousarray(np.asarray(old_ids, dtype=np.int64))
    n = np.ascontiguousarray(np.asarray(new_ids, dtype=np.int64))
    cut = ctypes.c_int32(0)
    _check(lib().kvc_prefix_cut(o.ctypes.data_as(ctypes.c_void_p), len(o), n.ctypes.data_as(ctypes.c_void_p),
                                len(n), 1 if ring else 0, ctypes.byref(cut)), "kvc_prefix_cut")
    return cut.value


def _token_ids(ids) -> np.ndarray:
    """Token IDs as int64, refusing anything that is not an integer (1.0 is not the token 1)."""
    if isinstance(ids, torch.Tensor):
        if ids.dtype.is_floating_point or ids.dtype == torch.bool or ids.dtype.is_complex:
            raise TypeError("token IDs must be integers, got %s" % ids.dtype)
        return np.ascontiguousarray(ids.detach().cpu().numpy().astype(np.int64).reshape(-1))
    if isinstance(ids, np.ndarray):
        if ids.dtype.kind not in "iu":
            raise TypeError("token IDs must be integers, got %s" % ids.dtype)
        return np.ascontiguousarray(ids.astype(np.int64).reshape(-1))
    for x in ids:
        if isinstance(x, bool) or not isinstance(x, (int, np.integer)):
            raise TypeError("token IDs must be integers, got %r" % (x,))
    return np.ascontiguousarray(np.asarray(list(ids), dtype=np.int64).reshape(-1))


def _sig(signature) -> bytes:
    return signature.encode() if isinstance(signature, str) else bytes(signature)


def kvc_pstore_create(cfg: kvc_config, capacity: int) -> ctypes.c_void_p:
    ps = ctypes.c_void_p(0)
    _check(lib().kvc_pstore_create(ctypes.byref(cfg), int(capacity), ctypes.byref(ps)), "kvc_pstore_create")
    return ps


def kvc_pstore_destroy(ps) -> None:
    _check(lib().kvc_pstore_destroy(ps), "kvc_pstore_destroy")


def kvc_pstore_insert(ps, ids, scope: str, signature=b"") -> int:
    a, sg = _token_ids(ids), _sig(signature)
    slot = ctypes.c_int32(-1)
    _check(lib().kvc_pstore_insert(ps, a.ctypes.data_as(ctypes.c_void_p) if len(a) else None, len(a),
                                   scope.encode(), sg or None, len(sg), ctypes.byref(slot)), "kvc_pstore_insert")
    return slot.value


def kvc_pstore_lookup(ps, ids, scope: str, signature=b"") -> tuple:
    a, sg = _token_ids(ids), _sig(signature)
    slot, cut = ctypes.c_int32(-1), ctypes.c_int32(0)
    _check(lib().kvc_pstore_lookup(ps, a.ctypes.data_as(ctypes.c_void_p) if len(a) else None, len(a),
                                   scope.encode(), sg or None, len(sg), ctypes.byref(slot), ctypes.byref(cut)),
           "kvc_pstore_lookup")
    return slot.value, cut.value


def kvc_store_save(h, slot: int, b: int, n: int, stream=None) -> None:
    _check(lib().kvc_store_save(h, int(slot), int(b), int(n), _stream(stream)), "kvc_store_save")


def kvc_store_load(h, slot: int, b: int, cut: int, stream=None) -> None:
    _check(lib().kvc_store_load(h, int(slot), int(b), int(cut), _stream(stream)), "kvc_store_load")


def kvc_set_request_id(h, b: int, request_id: int, stream=None) -> None:
    _check(lib().kvc_set_request_id(h, int(b), int(request_id) & 0xFFFFFFFF, _stream(stream)), "kvc_set_request_id")


def kvc_store_load_batch(h, slots, bs, cuts, stream=None) -> None:
    arr = [np.ascontiguousarray(np.asarray(x, dtype=np.int32).reshape(-1)) for x in (slots, bs, cuts)]
    n = len(arr[0])
    if any(len(x) != n for x in arr):
        raise ValueError("slots, requests and cuts must have one entry per load")
    ptr = [x.ctypes.data_as(ctypes.c_void_p) if n else None for x in arr]
    _check(lib().kvc_store_load_batch(h, n, ptr[0], ptr[1], ptr[2], _stream(stream)), "kvc_store_load_batch")


class PrefixStore:
    """Host policy of the prefix store (see include/kvc.h): which stored prefill a query
    reuses, and how many rows.  The rows live in a Cache's store slots."""

    def __init__(self, cfg: kvc_config, capacity: int = 2):
        self.capacity = capacity
        self.ps = kvc_pstore_create(cfg, capacity)

    def insert(self, ids, scope: str, signature=b"") -> int:
        return kvc_pstore_insert(self.ps, ids, scope, signature)

    def lookup(self, ids, scope: str, signature=b"") -> tuple:
        """(slot, cut); slot -1 when nothing is reusable."""
        return kvc_pstore_lookup(self.ps, ids, scope, signature)

    def close(self):
        if self.ps is not None and self.ps.value:
            kvc_pstore_destroy(self.ps)
        self.ps = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Cache:
    """A KV cache of one layer on the current CUDA device: the state buffer (a torch
    uint8 tensor) plus its library handle.  Thin wrapper over the functions above.
    Outputs that a call makes for itself are memory of the stream it runs on."""

    _EXPORT_DTYPES = {KVC_EXPORT_POSITIONS: np.int32, KVC_EXPORT_NEXT_POSITION: np.int32, KVC_EXPORT_KQ: np.int8,
                      KVC_EXPORT_VQ: np.int8, KVC_EXPORT_SK: np.float32, KVC_EXPORT_SV: np.float32,
                      KVC_EXPORT_WITNESS: np.uint16, KVC_EXPORT_KTAIL: np.uint16, KVC_EXPORT_VTAIL: np.uint16,
                      KVC_EXPORT_XMAP: np.int32, KVC_EXPORT_PAGE_TABLE: np.int32, KVC_EXPORT_K4: np.uint8,
                      KVC_EXPORT_V4: np.uint8}

    def __init__(self, cfg: kvc_config, device="cuda", stream=None):
        self.cfg = cfg
        self.torch_dtype = torch.bfloat16 if cfg.dtype == KVC_BF16 else torch.float32
        if cfg.out_dtype == 0:
            self.out_dtype = self.torch_dtype
        else:
            self.out_dtype = torch.float32 if cfg.out_dtype == KVC_F32 + 1 else torch.bfloat16
        nbytes = kvc_state_bytes(cfg)
        self.state = _empty(nbytes, torch.uint8, device, stream)
        self.h = kvc_create(cfg, self.state, stream)

    @classmethod
    def from_workload(cls, w, max_chunk=0, max_position=0, device="cuda", out_dtype=None, int8_exact_blocks=0,
                      page_pool=0, store_slots=0, int8_split=0, sinks=0):
        cfg = make_config(w.dtype, w.layout, w.quant, w.batch, w.n_q_heads, w.n_kv_heads, w.head_dim, w.capacity,
                          0 if w.layout == "ring" else w.window, max_position, w.rope_base, max_chunk, out_dtype,
                          int8_exact_blocks, page_pool, store_slots, w.extra.get("layer", 0),
                          w.extra.get("dither_key", (0, 0)), int8_split, sinks)
        return cls(cfg, device)

    def close(self):
        if self.h is not None and self.h.value:
            kvc_destroy(self.h)
        self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # shapes
    @property
    def B(self): return self.cfg.batch
    @property
    def Hq(self): return self.cfg.n_q_heads
    @property
    def Hkv(self): return self.cfg.n_kv_heads
    @property
    def d(self): return self.cfg.head_dim
    @property
    def S(self): return self.cfg.capacity

    def append(self, k, v, stream=None):
        _dev(k, self.torch_dtype, (self.B, self.Hkv, self.d), "k")
        _dev(v, self.torch_dtype, (self.B, self.Hkv, self.d), "v")
        kvc_append(self.h, k, v, stream)

    def append_rows(self, k, v, counts=None, stream=None):
        n = k.shape[2]
        _dev(k, self.torch_dtype, (self.B, self.Hkv, n, self.d), "k")
        _dev(v, self.torch_dtype, (self.B, self.Hkv, n, self.d), "v")
        kvc_append_rows(self.h, k, v, n, counts, stream)

    def decode(self, q, out=None, cmax=None, tanh=None, ct=None, stream=None):
        _dev(q, self.torch_dtype, (self.B, self.Hq, self.d), "q")
        if out is None:
            # (a third of the time that a tensor of a given shape, type and device takes)
            out = torch.empty_like(q) if stream is None and self.out_dtype == q.dtype else _empty(q.shape, self.out_dtype, q.device, stream)
        _dev(out, self.out_dtype, (self.B, self.Hq, self.d), "out")
        kvc_decode_attn(self.h, q, out, cmax, tanh, ct, stream)
        return out

    def trim(self, cuts, stream=None):
        if len(cuts) != self.B:
            raise ValueError("need one cut per request")
        kvc_trim(self.h, cuts, stream)

    def chunk(self, q, k, v, out=None, stream=None):
        n = q.shape[1]
        _dev(q, self.torch_dtype, (self.B, n, self.Hq, self.d), "q")
        _dev(k, self.torch_dtype, (self.B, n, self.Hkv, self.d), "k")
        _dev(v, self.torch_dtype, (self.B, n, self.Hkv, self.d), "v")
        if out is None:
            out = _empty(q.shape, self.out_dtype, q.device, stream)
        _dev(out, self.out_dtype, (self.B, n, self.Hq, self.d), "out")
        kvc_chunk_attn(self.h, q, k, v, n, out, stream)
        return out

    def prompt(self, q, k, v, counts, out=None, stream=None):
        """Packed prompts: ``counts[b]`` rows of each request in turn, appended and attended.  q [T, Hq, d],
        k and v [T, Hkv, d] with T >= sum(counts), heads dense, any row stride (views of one projection);
        rows behind the last request's are neither read nor written."""
        counts = _ints(counts)
        if len(counts) != self.B:
            raise ValueError("need one count per request")
        T, total, device = q.shape[0], sum(counts), self.state.get_device()
        if T < total:
            raise ValueError("q has %d rows, the counts sum to %d" % (T, total))
        for t, heads, name in ((q, self.Hq, "q"), (k, self.Hkv, "k"), (v, self.Hkv, "v")):
            if t.dtype != self.torch_dtype or t.shape != (T, heads, self.d):
                raise ValueError("%s must be %s of shape %s, got %s %s" % (name, self.torch_dtype, (T, heads, self.d), t.dtype,
                                                                           tuple(t.shape)))
            if t.get_device() != device:
                raise ValueError("%s must be on %s, got %s" % (name, self.state.device, t.device))
        if out is None:
            out = _empty((T, self.Hq, self.d), self.out_dtype, q.device, stream)
        if out.get_device() != device:
            raise ValueError("out must be on %s, got %s" % (self.state.device, out.device))
        _dev(out, self.out_dtype, (T, self.Hq, self.d), "out")
        kvc_prompt_attn(self.h, q, k, v, counts, out, stream)
        return out

    # whole requests and their pages
    def fork(self, src, dst, stream=None):
        """Requests ``dst`` become copies of requests ``src``; a paged cache shares the pages."""
        kvc_fork(self.h, src, dst, stream)

    def copy_from(self, other: "Cache", src, dst, stream=None):
        """Requests ``dst`` become copies of ``other``'s requests ``src``, with rows of their own.  A bf16 cache's rows
        are quantised on the way into a 4-bit one and read back from it."""
        kvc_copy(self.h, other.h, src, dst, stream)

    def free(self, requests, stream=None):
        kvc_free(self.h, requests, stream)

    def compact(self, stream=None) -> int:
        """Moves the pages in use to the start of the pool; returns their number."""
        return kvc_compact(self.h, stream)

    def page_counts(self) -> tuple:
        """(free pages, shared pages)"""
        return kvc_page_counts(self.h)

    def rows(self) -> tuple:
        """Views of the stored K and V rows: [B, Hkv, capacity, d], paged [pages, Hkv, 16, d] (4-bit rows: uint8,
        5 d / 8 bytes each).  For reading, on the stream that the cache's calls run on."""
        bits4 = self.cfg.kv_quant == KVC_QUANT_INT4
        row, dtype = (5 * self.d // 8, torch.uint8) if bits4 else (self.d, self.torch_dtype)
        shape = (self.cfg.page_pool, self.Hkv, 16, row) if self.cfg.page_pool else (self.B, self.Hkv, self.S, row)
        views = []
        for which in (KVC_EXPORT_K4, KVC_EXPORT_V4) if bits4 else (KVC_EXPORT_K, KVC_EXPORT_V):
            off, n = kvc_region(self.h, which)
            views.append(self.state[off:off + n].view(dtype).view(shape))
        return tuple(views)

    def export(self, which, stream=None) -> np.ndarray:
        raw = kvc_export(self.h, which, stream)
        if which in (KVC_EXPORT_K, KVC_EXPORT_V):
            dt = np.uint16 if self.cfg.dtype == KVC_BF16 else np.float32
            return raw.view(dt).reshape(self.B, self.Hkv, self.S, self.d)
        arr = raw.view(self._EXPORT_DTYPES[which])
        shapes = {KVC_EXPORT_POSITIONS: (self.B, self.S), KVC_EXPORT_NEXT_POSITION: (self.B,),
                  KVC_EXPORT_KQ: (self.B, self.Hkv, self.S, self.d),
                  KVC_EXPORT_VQ: (self.B, self.Hkv, self.S, self.d),
                  KVC_EXPORT_SK: (self.B, self.Hkv, self.S // 16), KVC_EXPORT_SV: (self.B, self.Hkv, self.S // 16),
                  KVC_EXPORT_WITNESS: (self.B, self.Hkv, self.S, 16), KVC_EXPORT_KTAIL: (self.B, self.Hkv, 16, self.d),
                  KVC_EXPORT_VTAIL: (self.B, self.Hkv, 16, self.d),
                  KVC_EXPORT_XMAP: (self.B, self.Hkv, self.S // 16),
                  KVC_EXPORT_PAGE_TABLE: (self.B, self.S // 16),
                  KVC_EXPORT_K4: (self.B, self.Hkv, self.S, 5 * self.d // 8),
                  KVC_EXPORT_V4: (self.B, self.Hkv, self.S, 5 * self.d // 8)}
        return arr.reshape(shapes[which])

    def next_positions(self) -> np.ndarray:
        return kvc_next_positions(self.h, self.B)

    # gated fallback of the INT8 tier
    def block_risk(self, ct, risk=None, stream=None):
        """Per complete block, the largest c_t over its tokens and the KV head's query heads."""
        _dev(ct, torch.float32, (self.B, self.Hq, self.S), "ct")
        if risk is None:
            risk = _empty((self.B, self.Hkv, self.S // 16), torch.float32, ct.device, stream)
        _dev(risk, torch.float32, (self.B, self.Hkv, self.S // 16), "risk")
        kvc_int8_block_risk(self.h, ct, risk, stream)
        return risk

    def restore(self, blocks, k_full, v_full, stream=None):
        _dev(k_full, torch.bfloat16, (self.B, self.Hkv, self.S, self.d), "k_full")
        _dev(v_full, torch.bfloat16, (self.B, self.Hkv, self.S, self.d), "v_full")
        kvc_int8_restore(self.h, blocks, k_full, v_full, stream)

    def device_status(self, stream=None) -> int:
        return kvc_device_status(self.h, stream)

    def set_request_id(self, b, request_id, stream=None):
        kvc_set_request_id(self.h, b, request_id, stream)

    # prefix store
    def store_save(self, slot, b, n, stream=None):
        kvc_store_save(self.h, slot, b, n, stream)

    def store_load(self, slot, b, cut, stream=None):
        kvc_store_load(self.h, slot, b, cut, stream)

    def store_load_batch(self, slots, bs, cuts, stream=None):
        kvc_store_load_batch(self.h, slots, bs, cuts, stream)

    def save_prefix(self, store: PrefixStore, b, ids, scope: str, signature=b"", stream=None) -> int:
        """Records request b's prefill of ``ids`` in ``store`` and copies its rows to the slot."""
        slot = store.insert(ids, scope, signature)
        kvc_store_save(self.h, slot, b, len(_token_ids(ids)), stream)
        return slot

    def reuse_prefix(self, store: PrefixStore, b, ids, scope: str, signature=b"", stream=None) -> tuple:
        """Request b continues from the longest reusable stored prefix of ``ids``: (slot, cut)."""
        slot, cut = store.lookup(ids, scope, signature)
        kvc_store_load(self.h, slot, b, cut, stream)
        return slot, cut
