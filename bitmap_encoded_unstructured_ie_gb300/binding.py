"""Thin ctypes binding of libus (include/us.h) over torch tensors.

Argument marshalling only: every step of encode / SpMM / spMspV runs in the
CUDA library.  Torch supplies device memory and the current stream.  If the
library has not been built, the first call raises ``LibraryMissing``: there is
no CPU fallback.

Function names follow the C ABI: ``us_encode``, ``us_spmm_w4a4``,
``us_spmm_f16``, ``us_spmspv_f16``, ``us_colinfo``, ``us_spmspv_f16_ci``, ``us_quantize_x``,
``us_kv_write``, ``us_kv_read``, ``us_kv_commit``, ``us_attn_kv``, ``us_kv_reserve``, ``us_kv_slots``,
``us_norm_rope``, ``us_kv_append``, ``us_lat_write``, ``us_lat_read``, ``us_lat_commit``, ``us_attn_lat``,
``us_attn_rows``, ``us_workspace_bytes``, ``us_pick_split_k``,
``us_validate``, ``us_get_last_device_status``.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
import threading
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libus.so")

US_OK, US_ERR_INVALID_ARG, US_ERR_UNSUPPORTED, US_ERR_TOO_LARGE = 0, 1, 2, 3
US_ERR_WORKSPACE, US_ERR_CUDA, US_ERR_TIMEOUT, US_ERR_CORRUPT = 4, 5, 6, 7
US_F16, US_I4, US_I2, US_I8 = 0, 1, 2, 3          # US_I8: K/V cache only
US_ORDER_ROW, US_ORDER_COL = 0, 1
US_OP_ENCODE, US_OP_SPMM_W4A4, US_OP_SPMM_F16, US_OP_SPMSPV_F16 = 0, 1, 2, 3
US_BITMAP_STATIC = 1
US_ROPE_HALVES, US_ROPE_PAIRS = 0, 1

EXPORTED = ("us_encode_sizes", "us_encode", "us_spmm_w4a4", "us_spmm_f16", "us_spmm_f16_noalloc", "us_spmspv_f16",
            "us_colinfo", "us_spmspv_f16_ci", "us_quantize_x",
            "us_kv_write", "us_kv_read", "us_kv_commit", "us_attn_kv", "us_attn_kv_workspace_bytes",
            "us_kv_reserve", "us_kv_slots", "us_norm_rope", "us_kv_append", "us_lat_write", "us_lat_read", "us_lat_commit",
           "us_attn_lat", "us_attn_lat_workspace_bytes", "us_attn_rows", "us_attn_rows_workspace_bytes",
           "us_encode_ie_sizes", "us_encode_ie", "us_reorder_rows", "us_spmm_w4a4_ie", "us_workspace_bytes_ie",
            "us_pick_split_k_ie",
            "us_workspace_bytes", "us_pick_split_k", "us_validate", "us_get_last_device_status",
            "us_selftest_wait_timeout", "us_status_string", "us_version")


class LibraryMissing(RuntimeError):
    pass


class UsError(RuntimeError):
    def __init__(self, fn: str, code: int, text: str):
        super().__init__(f"{fn}: {text} ({code})")
        self.code = code


class us_bitmap(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int32), ("K", ctypes.c_int32), ("TM", ctypes.c_int32), ("TK", ctypes.c_int32),
                ("elem", ctypes.c_int32), ("order", ctypes.c_int32),
                ("bitmap", ctypes.c_void_p), ("tile_off", ctypes.c_void_p), ("values", ctypes.c_void_p),
                ("values_bytes", ctypes.c_uint64), ("flags", ctypes.c_uint32), ("reserved", ctypes.c_uint32)]


class us_bitmap_ie(ctypes.Structure):
    _fields_ = [("W", us_bitmap), ("RA", ctypes.c_int32), ("CA", ctypes.c_int32), ("perm", ctypes.c_void_p)]


class us_kv_cache(ctypes.Structure):
    _fields_ = [("elem", ctypes.c_int32), ("D", ctypes.c_int32), ("Hkv", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32), ("B", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p)]


class us_kv_pool(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("page_table", ctypes.c_void_p), ("held", ctypes.c_void_p),
                ("free_pages", ctypes.c_void_p), ("free_count", ctypes.c_void_p)]


class us_rope(ctypes.Structure):
    _fields_ = [("style", ctypes.c_int32), ("R", ctypes.c_int32), ("eps", ctypes.c_float), ("reserved", ctypes.c_int32),
                ("turns", ctypes.c_void_p)]


class us_heads(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("ld", ctypes.c_int64), ("hs", ctypes.c_int64), ("y", ctypes.c_void_p),
                ("ldy", ctypes.c_int64), ("hsy", ctypes.c_int64), ("w", ctypes.c_void_p), ("H", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class us_lat_cache(ctypes.Structure):
    _fields_ = [("Dc", ctypes.c_int32), ("Dr", ctypes.c_int32), ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("B", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("rows", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p)]


class us_attn_kv_rows(ctypes.Structure):
    _fields_ = [("Dn", ctypes.c_int32), ("Dr", ctypes.c_int32), ("Dv", ctypes.c_int32), ("H", ctypes.c_int32),
                ("K", ctypes.c_void_p), ("ldk", ctypes.c_int64), ("hsk", ctypes.c_int64), ("KR", ctypes.c_void_p),
                ("ldkr", ctypes.c_int64), ("V", ctypes.c_void_p), ("ldv", ctypes.c_int64), ("hsv", ctypes.c_int64),
                ("S", ctypes.c_int64)]


# The same as bytes, which the calls pass: a Structure takes three times as long to fill.
_pack_heads = struct.Struct("@PqqPqqPii").pack
_pack_rows = struct.Struct("@iiiiPqqPqPqqq").pack
assert struct.calcsize("@PqqPqqPii") == ctypes.sizeof(us_heads)
assert struct.calcsize("@iiiiPqqPqPqqq") == ctypes.sizeof(us_attn_kv_rows)

_lock = threading.Lock()
_lib = None


def load(path: str = LIB_PATH):
    """Load libus.so (once).  Raises LibraryMissing if it was not built."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise LibraryMissing(f"{path} not found: build it with __graft_entry__.build() "
                                 f"or python -m bitmap_encoded_unstructured_ie_gb300.build")
        lib = ctypes.CDLL(path)
        P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
        psz = ctypes.POINTER(ctypes.c_size_t)
        pbm = ctypes.POINTER(us_bitmap)
        lib.us_encode_sizes.argtypes = [i32, i32, i32, i32, i32, psz, psz, psz, psz]
        lib.us_encode.argtypes = [P, i64, i32, i32, i32, i32, i32, i32, P, P, P, sz, P, sz, P]
        lib.us_spmm_w4a4.argtypes = [pbm, P, P, P, i32, P, P, P, sz, i32, P]
        lib.us_spmm_f16.argtypes = [pbm, P, i32, P, P, sz, i32, P]
        lib.us_spmm_f16_noalloc.argtypes = [pbm, P, i32, P, i32, P]
        lib.us_spmspv_f16.argtypes = [pbm, P, ctypes.c_float, P, P, sz, P]
        lib.us_colinfo.argtypes = [pbm, P, P]
        pie = ctypes.POINTER(us_bitmap_ie)
        lib.us_encode_ie_sizes.argtypes = [i32, i32, i32, i32, i32, i32, i32, psz, psz, psz, psz]
        lib.us_encode_ie.argtypes = [P, i64, i32, i32, i32, i32, i32, i32, i32, P, P, P, P, sz, P, sz, P]
        lib.us_reorder_rows.argtypes = [P, i64, i32, i32, i32, i32, i32, i32, i32, P, i32]
        lib.us_spmm_w4a4_ie.argtypes = [pie, P, P, P, i32, P, P, P, sz, i32, P]
        lib.us_workspace_bytes_ie.argtypes = [pie, i32, i32, psz]
        lib.us_pick_split_k_ie.argtypes = [pie, i32, ctypes.POINTER(ctypes.c_int)]
        lib.us_spmspv_f16_ci.argtypes = [pbm, P, P, i32, ctypes.c_float, P, P, sz, P]
        lib.us_quantize_x.argtypes = [P, i32, i32, P, P, P]
        pkv = ctypes.POINTER(us_kv_cache)
        lib.us_kv_write.argtypes = [pkv, P, i64, P, i64, i32, P, P, i32, P]
        lib.us_kv_read.argtypes = [pkv, i32, P, P, i32, P, i64, P, i64, P]
        lib.us_kv_commit.argtypes = [pkv, i32, P, P, P, i32, P]
        lib.us_attn_kv.argtypes = [pkv, P, i64, i32, i32, P, P, P, i32, ctypes.c_float, P, i64, P, sz, P]
        lib.us_attn_kv_workspace_bytes.argtypes = [pkv, i32, i32, psz]
        f32, ppl = ctypes.c_float, ctypes.POINTER(us_kv_pool)
        prp, plt = ctypes.POINTER(us_rope), ctypes.POINTER(us_lat_cache)
        lib.us_kv_reserve.argtypes = [ppl, P, P]
        lib.us_kv_slots.argtypes = [ppl, i32, P, P, i32, P, P]
        lib.us_norm_rope.argtypes = [prp, i32, P, P, i32, i32, P, P, P, i32, P]
        lib.us_kv_append.argtypes = [pkv, prp, P, P, P, i64, i32, P, P, P, i32, P]
        lib.us_lat_write.argtypes = [plt, prp, P, i64, P, i32, P, P, P, i32, P]
        lib.us_lat_read.argtypes = [plt, i32, P, P, i32, P, i64, P]
        lib.us_lat_commit.argtypes = [plt, i32, P, P, P, i32, P]
        lib.us_attn_lat.argtypes = [plt, P, i64, i32, i32, P, P, P, i32, f32, P, i64, P, sz, P]
        lib.us_attn_lat_workspace_bytes.argtypes = [plt, i32, i32, psz]
        lib.us_attn_rows.argtypes = [P, P, i64, i32, i32, P, P, i32, f32, P, i64, P, sz, P]
        lib.us_attn_rows_workspace_bytes.argtypes = [P, i32, i32, psz]
        lib.us_workspace_bytes.argtypes = [i32, pbm, i32, i32, psz]
        lib.us_pick_split_k.argtypes = [i32, pbm, i32, ctypes.POINTER(ctypes.c_int)]
        lib.us_validate.argtypes = [pbm]
        lib.us_get_last_device_status.argtypes = [P]
        lib.us_selftest_wait_timeout.argtypes = [ctypes.c_uint64, P, P]
        lib.us_status_string.argtypes = [i32]
        lib.us_status_string.restype = ctypes.c_char_p
        lib.us_version.argtypes = []
        for name in EXPORTED:
            if name != "us_status_string":
                getattr(lib, name).restype = ctypes.c_int
        _lib = lib
        return lib


def status_string(code: int) -> str:
    return load().us_status_string(int(code)).decode()


def _check(fn: str, code: int):
    if code != US_OK:
        raise UsError(fn, code, status_string(code))


def _dptr(t: torch.Tensor | None):
    if t is None:
        return None
    assert t.is_cuda and t.is_contiguous(), "device tensors must be contiguous CUDA tensors"
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


@dataclass
class Encoded:
    """An encoded matrix: three device tensors plus its parameters."""
    M: int
    K: int
    TM: int
    TK: int
    elem: int
    order: int
    bitmap: torch.Tensor      # uint64 words (int64 storage)
    tile_off: torch.Tensor    # uint32 (int32 storage), nT + 1
    values: torch.Tensor      # uint8
    values_bytes: int
    flags: int = 0            # US_BITMAP_STATIC: not written by earlier work on the stream

    def desc(self) -> us_bitmap:
        return us_bitmap(self.M, self.K, self.TM, self.TK, self.elem, self.order,
                         self.bitmap.data_ptr(), self.tile_off.data_ptr(), self.values.data_ptr(),
                         self.values_bytes, self.flags, 0)

    def nbytes(self) -> int:
        return self.bitmap.numel() * 8 + self.tile_off.numel() * 4 + self.values_bytes


def encode_sizes(M, K, TM, TK, elem):
    b, o, v, w = (ctypes.c_size_t() for _ in range(4))
    _check("us_encode_sizes", load().us_encode_sizes(M, K, TM, TK, elem, ctypes.byref(b), ctypes.byref(o),
                                                     ctypes.byref(v), ctypes.byref(w)))
    return b.value, o.value, v.value, w.value


def us_encode(W: torch.Tensor, TM: int, TK: int, elem: int, order: int, stream=None, shrink: bool = True) -> Encoded:
    """Encode a dense CUDA matrix (fp16 for US_F16, int8 codes for US_I4)."""
    lib = load()
    M, K = W.shape
    dev = W.device
    assert W.is_cuda and W.stride(1) == 1, "W must be a CUDA matrix with unit column stride"
    bb, ob, vcap, wsb = encode_sizes(M, K, TM, TK, elem)
    bitmap = torch.empty(bb // 8, dtype=torch.int64, device=dev)
    tile_off = torch.empty(ob // 4, dtype=torch.int32, device=dev)
    values = torch.zeros(max(vcap, 16), dtype=torch.uint8, device=dev)
    ws = torch.zeros(max(wsb, 16), dtype=torch.uint8, device=dev)
    _check("us_encode", lib.us_encode(ctypes.c_void_p(W.data_ptr()), W.stride(0), M, K, TM, TK, elem, order, _dptr(bitmap),
                                      _dptr(tile_off), _dptr(values), values.numel(), _dptr(ws), ws.numel(),
                                      _stream(stream)))
    used_elems = int(tile_off[-1].item()) & 0xFFFFFFFF
    used = used_elems * {US_F16: 16, US_I4: 4, US_I2: 2}[elem] // 8
    if shrink:
        values = values[: max(used, 16)].clone()
    return Encoded(M, K, TM, TK, elem, order, bitmap, tile_off, values, used)


def us_encode_into(W: torch.Tensor, E: Encoded, ws: torch.Tensor, stream=None):
    """Re-encode W into E's existing buffers (no readback, no synchronisation).
    E.values must have the worst-case capacity (shrink=False)."""
    M, K = W.shape
    assert W.is_cuda and W.stride(1) == 1
    _check("us_encode", load().us_encode(ctypes.c_void_p(W.data_ptr()), W.stride(0), M, K, E.TM, E.TK, E.elem,
                                         E.order, _dptr(E.bitmap), _dptr(E.tile_off), _dptr(E.values),
                                         E.values.numel(), _dptr(ws), ws.numel(), _stream(stream)))


@dataclass
class EncodedIE:
    """IE-BME with RA x CA areas: an Encoded (ROW scan, union-mask bitmap) plus
    the area counts and the per-tile row permutation (device uint8, or None)."""
    E: Encoded
    RA: int
    CA: int
    perm: torch.Tensor | None = None

    def desc(self) -> us_bitmap_ie:
        return us_bitmap_ie(self.E.desc(), self.RA, self.CA, self.perm.data_ptr() if self.perm is not None else None)


def encode_ie_sizes(M, K, TM, TK, RA, CA, elem):
    b, o, v, w = (ctypes.c_size_t() for _ in range(4))
    _check("us_encode_ie_sizes", load().us_encode_ie_sizes(M, K, TM, TK, RA, CA, elem, ctypes.byref(b),
                                                           ctypes.byref(o), ctypes.byref(v), ctypes.byref(w)))
    return b.value, o.value, v.value, w.value


def us_encode_ie(W: torch.Tensor, TM: int, TK: int, RA: int, CA: int, elem: int, perm: torch.Tensor | None = None,
                 stream=None) -> EncodedIE:
    """Encode a dense CUDA matrix as IE-BME with RA x CA areas; perm: device
    uint8 tensor of TM bytes per tile (tile-major) or None."""
    lib = load()
    M, K = W.shape
    dev = W.device
    assert W.is_cuda and W.stride(1) == 1, "W must be a CUDA matrix with unit column stride"
    bb, ob, vcap, wsb = encode_ie_sizes(M, K, TM, TK, RA, CA, elem)
    bitmap = torch.empty(max(bb // 8, 2), dtype=torch.int64, device=dev)
    tile_off = torch.empty(ob // 4, dtype=torch.int32, device=dev)
    values = torch.zeros(max(vcap, 16), dtype=torch.uint8, device=dev)
    ws = torch.zeros(max(wsb, 16), dtype=torch.uint8, device=dev)
    _check("us_encode_ie", lib.us_encode_ie(ctypes.c_void_p(W.data_ptr()), W.stride(0), M, K, TM, TK, RA, CA, elem,
                                            _dptr(perm), _dptr(bitmap), _dptr(tile_off), _dptr(values),
                                            values.numel(), _dptr(ws), ws.numel(), _stream(stream)))
    used_elems = int(tile_off[-1].item()) & 0xFFFFFFFF
    used = used_elems * {US_F16: 16, US_I4: 4, US_I2: 2}[elem] // 8
    values = values[: max(used, 16)].clone()
    return EncodedIE(Encoded(M, K, TM, TK, elem, US_ORDER_ROW, bitmap, tile_off, values, used), RA, CA, perm)


def us_reorder_rows(W, TM: int, TK: int, RA: int, CA: int, elem: int, nthreads: int = 0):
    """Bitmap-aware row reordering on the host (offline): numpy W (fp16 or int8
    codes) -> numpy uint8 permutation, TM bytes per tile, tile-major."""
    import numpy as np
    Wh = np.ascontiguousarray(W)
    M, K = Wh.shape
    perm = np.zeros((M // TM) * (K // TK) * TM, np.uint8)
    n = nthreads or max(1, min(32, os.cpu_count() or 1))
    _check("us_reorder_rows", load().us_reorder_rows(Wh.ctypes.data, K, M, K, TM, TK, RA, CA, elem,
                                                     perm.ctypes.data, n))
    return perm


def us_workspace_bytes_ie(E: EncodedIE, N: int, split_k: int = 0) -> int:
    n = ctypes.c_size_t()
    d = E.desc()
    _check("us_workspace_bytes_ie", load().us_workspace_bytes_ie(ctypes.byref(d), N, split_k, ctypes.byref(n)))
    return n.value


def us_pick_split_k_ie(E: EncodedIE, N: int = 1) -> int:
    """0 when the balanced kernel serves us_spmm_w4a4_ie on E with N tokens."""
    s = ctypes.c_int()
    d = E.desc()
    _check("us_pick_split_k_ie", load().us_pick_split_k_ie(ctypes.byref(d), N, ctypes.byref(s)))
    return s.value


def workspace_ie(E: EncodedIE, N: int, split_k: int = 0) -> torch.Tensor:
    return torch.zeros(max(us_workspace_bytes_ie(E, N, split_k), 16), dtype=torch.uint8, device=E.E.bitmap.device)


def us_spmm_w4a4_ie(E: EncodedIE, Xq: torch.Tensor, s_w, s_x, N: int, Yacc: torch.Tensor, Y, ws: torch.Tensor,
                    split_k: int = 0, stream=None):
    d = E.desc()
    _check("us_spmm_w4a4_ie", load().us_spmm_w4a4_ie(ctypes.byref(d), _dptr(Xq), _dptr(s_w), _dptr(s_x), N,
                                                     _dptr(Yacc), _dptr(Y), _dptr(ws), ws.numel(), split_k,
                                                     _stream(stream)))


def from_host(bitmap, tile_off, values, M, K, TM, TK, elem, order, device="cuda") -> Encoded:
    """Wrap host numpy arrays of an encoded matrix as device tensors."""
    import numpy as np
    bm = torch.from_numpy(np.ascontiguousarray(bitmap).view(np.int64)).to(device)
    off = torch.from_numpy(np.ascontiguousarray(tile_off).view(np.int32)).to(device)
    v = np.ascontiguousarray(values, dtype=np.uint8)
    vb = v.size
    v = np.concatenate([v, np.zeros((-v.size) % 16 + (16 if v.size == 0 else 0), np.uint8)])
    return Encoded(M, K, TM, TK, elem, order, bm, off, torch.from_numpy(v).to(device), vb)


def us_workspace_bytes(op: int, E: Encoded, N: int = 1, split_k: int = 0) -> int:
    n = ctypes.c_size_t()
    d = E.desc()
    _check("us_workspace_bytes", load().us_workspace_bytes(op, ctypes.byref(d), N, split_k, ctypes.byref(n)))
    return n.value


def us_pick_split_k(op: int, E: Encoded, N: int = 1) -> int:
    s = ctypes.c_int()
    d = E.desc()
    _check("us_pick_split_k", load().us_pick_split_k(op, ctypes.byref(d), N, ctypes.byref(s)))
    return s.value


def workspace(op: int, E: Encoded, N: int = 1, split_k: int = 0) -> torch.Tensor:
    """A zero-filled workspace of the size the call needs."""
    return torch.zeros(max(us_workspace_bytes(op, E, N, split_k), 16), dtype=torch.uint8, device=E.bitmap.device)


def us_spmm_w4a4(E: Encoded, Xq: torch.Tensor, s_w: torch.Tensor, s_x: torch.Tensor, N: int,
                 Yacc: torch.Tensor, Y: torch.Tensor | None, ws: torch.Tensor, split_k: int = 0, stream=None):
    d = E.desc()
    _check("us_spmm_w4a4", load().us_spmm_w4a4(ctypes.byref(d), _dptr(Xq), _dptr(s_w), _dptr(s_x), N, _dptr(Yacc),
                                               _dptr(Y), _dptr(ws), ws.numel(), split_k, _stream(stream)))


def us_spmm_f16(E: Encoded, X: torch.Tensor, N: int, Y: torch.Tensor, ws: torch.Tensor, split_k: int = 0,
                stream=None):
    d = E.desc()
    _check("us_spmm_f16", load().us_spmm_f16(ctypes.byref(d), _dptr(X), N, _dptr(Y), _dptr(ws), ws.numel(),
                                             split_k, _stream(stream)))


def us_spmm_f16_noalloc(E: Encoded, X: torch.Tensor, N: int, Y: torch.Tensor, split_k: int = 0, stream=None):
    """fp16 SpMM whose split-K scratch lives inside the library (no workspace)."""
    d = E.desc()
    _check("us_spmm_f16_noalloc", load().us_spmm_f16_noalloc(ctypes.byref(d), _dptr(X), N, _dptr(Y), split_k,
                                                             _stream(stream)))


def us_spmspv_f16(E: Encoded, x: torch.Tensor, tau: float, y: torch.Tensor, ws: torch.Tensor, stream=None):
    d = E.desc()
    _check("us_spmspv_f16", load().us_spmspv_f16(ctypes.byref(d), _dptr(x), float(tau), _dptr(y), _dptr(ws),
                                                 ws.numel(), _stream(stream)))


def colinfo_words(E: Encoded) -> int:
    """Number of uint32 ColInfo words of a COL-order matrix (one per tile column)."""
    return (E.M // E.TM) * E.K


def us_colinfo(E: Encoded, colinfo: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """ColInfo of a COL-order matrix: int32 tensor (bit pattern of uint32) of
    (M / TM) * K words, tile-major, (offset << 16) | nnz per tile column."""
    if colinfo is None:
        colinfo = torch.empty(colinfo_words(E), dtype=torch.int32, device=E.bitmap.device)
    d = E.desc()
    _check("us_colinfo", load().us_colinfo(ctypes.byref(d), _dptr(colinfo), _stream(stream)))
    return colinfo


def us_spmspv_f16_ci(E: Encoded, colinfo: torch.Tensor, X: torch.Tensor, N: int, tau: float, Y: torch.Tensor,
                     ws: torch.Tensor | None = None, stream=None):
    """Batched spMspV through ColInfo: X N x K fp16 (bit pattern), Y N x M."""
    d = E.desc()
    _check("us_spmspv_f16_ci", load().us_spmspv_f16_ci(ctypes.byref(d), _dptr(colinfo), _dptr(X), N, float(tau),
                                                       _dptr(Y), _dptr(ws), ws.numel() if ws is not None else 0,
                                                       _stream(stream)))


def us_quantize_x(X: torch.Tensor, N: int, K: int, Xq: torch.Tensor, s_x: torch.Tensor, stream=None):
    """fp16 activations (N x K, token-major) -> packed int4 codes (N x K/2 bytes)
    and one fp16 scale per token."""
    _check("us_quantize_x", load().us_quantize_x(_dptr(X), N, K, _dptr(Xq), _dptr(s_x), _stream(stream)))


_F16, _I32 = torch.float16, torch.int32
_HALVES = frozenset((torch.float16, torch.int16, torch.uint16))     # fp16, or its bit pattern
_BYTES = frozenset((torch.uint8, torch.int8))
_WORDS = frozenset((torch.int64, torch.uint64))


@dataclass(frozen=True, eq=False)
class KVCache:
    """A paged, quantised key/value cache over device tensors: codes k and v
    (bytes, pages x Hkv x slots x row bytes), scales (fp16 or its bit pattern,
    pages x Hkv x slots x 2: K, then V) and the page table (int32, B x pages).
    The descriptor is made once, with the object; the tensors' contents may
    change, the tensors may not."""
    elem: int                 # US_I8 or US_I4
    D: int
    k: torch.Tensor
    v: torch.Tensor
    scale: torch.Tensor
    page_table: torch.Tensor

    def __post_init__(self):
        num_pages, Hkv, page_size, row = self.k.shape
        B, max_pages = self.page_table.shape
        assert row * 8 == self.D * (8 if self.elem == US_I8 else 4), "k: rows of D codes"
        assert self.v.shape == self.k.shape and tuple(self.scale.shape) == (num_pages, Hkv, page_size, 2)
        assert self.k.dtype in _BYTES and self.v.dtype in _BYTES, "k, v: bytes"
        assert self.scale.dtype in _HALVES, "scale: fp16 or its bit pattern"
        assert self.page_table.dtype == torch.int32
        device = self.k.get_device()
        assert all(t.get_device() == device for t in (self.v, self.scale, self.page_table)), "tensors of one device"
        d = us_kv_cache(self.elem, self.D, Hkv, page_size, num_pages, B, max_pages, 0, _dptr(self.k), _dptr(self.v),
                        _dptr(self.scale), _dptr(self.page_table))
        for name, value in (("B", B), ("Hkv", Hkv), ("page_size", page_size), ("device", device),
                            ("_desc", d), ("_ref", ctypes.byref(d))):
            object.__setattr__(self, name, value)


def kv_cache(elem: int, D: int, Hkv: int, page_size: int, num_pages: int, page_table: torch.Tensor) -> KVCache:
    """An empty cache of num_pages pages on the page table's device."""
    dev, row = page_table.device, D * (8 if elem == US_I8 else 4) // 8
    k, v = (torch.zeros(num_pages, Hkv, page_size, row, dtype=torch.uint8, device=dev) for _ in range(2))
    return KVCache(elem, D, k, v, torch.ones(num_pages, Hkv, page_size, 2, dtype=torch.float16, device=dev), page_table)


# The cache's calls are short (a decode step appends and attends in a few
# microseconds on the GPU), so their marshalling passes plain integers.
def _rows(x: torch.Tensor, H: int, C: KVCache):
    """Rows, pointer and row distance of T x H x D fp16 rows whose heads are contiguous."""
    T, h, d = x.shape
    ld, sh, sd = x.stride()
    t = x.dtype
    assert (t is _F16 or t in _HALVES) and h == H and d == C.D and sd == 1 and (sh == d or H == 1), \
        "rows must be T x H x D CUDA fp16 with contiguous heads"
    assert x.get_device() == C.device, "rows must be on the cache's device"
    return T, x.data_ptr(), (ld if T > 1 else H * d)


def _i32(x: torch.Tensor, n: int, C: KVCache) -> int:
    assert x.dtype is _I32 and x.numel() == n and x.is_contiguous(), "int32 CUDA array of n entries"
    assert x.get_device() == C.device, "arrays must be on the cache's device"
    return x.data_ptr()


# current_stream() builds an object (2.9 us on the GPU machine's host, of a call's 9); the raw handle does not (0.1 us).
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _raw_stream(stream, C: KVCache) -> int:
    # (the library launches on the current device)
    assert _current_device() == C.device, "the cache's device must be the current one"
    if stream is not None:
        assert stream.device_index == C.device, "the stream must be of the cache's device"
        return stream.cuda_stream
    return torch.cuda.current_stream().cuda_stream if _current_raw_stream is None else _current_raw_stream(C.device)


def us_kv_write(C: KVCache, K: torch.Tensor, V: torch.Tensor, tok_off: torch.Tensor, pos: torch.Tensor, max_n: int,
                stream=None):
    """Quantise T x Hkv x D rows of K and V into the cache at positions pos[b] .. ."""
    T, kp, ldk = _rows(K, C.Hkv, C)
    Tv, vp, ldv = _rows(V, C.Hkv, C)
    assert T == Tv
    _check("us_kv_write", (_lib or load()).us_kv_write(C._ref, kp, ldk, vp, ldv, T, _i32(tok_off, C.B + 1, C),
                                                       _i32(pos, C.B, C), max_n, _raw_stream(stream, C)))


def us_kv_read(C: KVCache, tok_off: torch.Tensor, pos: torch.Tensor, max_n: int, K: torch.Tensor, V: torch.Tensor,
               stream=None):
    """Read positions pos[b] .. back as fp16 rows (T x Hkv x D) of K and V."""
    T, kp, ldk = _rows(K, C.Hkv, C)
    Tv, vp, ldv = _rows(V, C.Hkv, C)
    assert T == Tv
    _check("us_kv_read", (_lib or load()).us_kv_read(C._ref, T, _i32(tok_off, C.B + 1, C), _i32(pos, C.B, C), max_n, kp, ldk,
                                                     vp, ldv, _raw_stream(stream, C)))


def us_kv_commit(C: KVCache, acc_off: torch.Tensor, acc: torch.Tensor, pos: torch.Tensor, max_n: int, stream=None):
    """Move the accepted drafted tokens' entries, pos[b] + acc[i], to pos[b] + i."""
    T = acc.numel()
    _check("us_kv_commit", (_lib or load()).us_kv_commit(C._ref, T, _i32(acc_off, C.B + 1, C), _i32(acc, T, C),
                                                         _i32(pos, C.B, C), max_n, _raw_stream(stream, C)))


def us_attn_kv_workspace_bytes(C: KVCache, Hq: int, max_n: int) -> int:
    n = ctypes.c_size_t()
    _check("us_attn_kv_workspace_bytes", load().us_attn_kv_workspace_bytes(C._ref, Hq, max_n, ctypes.byref(n)))
    return n.value


def workspace_attn_kv(C: KVCache, Hq: int, max_n: int) -> torch.Tensor:
    """A zero-filled workspace of the size us_attn_kv needs."""
    return torch.zeros(max(us_attn_kv_workspace_bytes(C, Hq, max_n), 16), dtype=torch.uint8, device=C.k.device)


def us_attn_kv(C: KVCache, Q: torch.Tensor, tok_off: torch.Tensor, pos: torch.Tensor, mask: torch.Tensor | None,
               max_n: int, scale: float, O: torch.Tensor, ws: torch.Tensor, stream=None):
    """Attention of T x Hq x D query rows over the cache; mask: one 64-bit word
    per row (a tree of drafted tokens), or None (a chain)."""
    Hq = Q.shape[1]
    T, qp, ldq = _rows(Q, Hq, C)
    To, op, ldo = _rows(O, Hq, C)
    assert T == To and ws.is_contiguous() and ws.get_device() == C.device, "ws must be contiguous, on the cache's device"
    if mask is not None:
        assert mask.dtype in _WORDS and mask.numel() == T and mask.is_contiguous(), "mask must be T CUDA 64-bit words"
        assert mask.get_device() == C.device, "mask must be on the cache's device"
    _check("us_attn_kv", (_lib or load()).us_attn_kv(C._ref, qp, ldq, Hq, T, _i32(tok_off, C.B + 1, C), _i32(pos, C.B, C),
                                                     None if mask is None else mask.data_ptr(), max_n, scale, op, ldo,
                                                     ws.data_ptr(), ws.numel() * ws.element_size(),
                                                     _raw_stream(stream, C)))


# ---- page tables from request lengths
@dataclass(frozen=True, eq=False)
class KVPool:
    """The pages that requests hold and those that are free, all int32 on the device:
    the page table (B x max_pages, as in KVCache; the same tensor may serve caches),
    how many pages each request holds (B), the stack of free pages (num_pages) and how
    many of it are free (1).  us_kv_reserve changes their contents."""
    page_size: int
    page_table: torch.Tensor
    held: torch.Tensor
    free_pages: torch.Tensor
    free_count: torch.Tensor

    def __post_init__(self):
        B, max_pages = self.page_table.shape
        parts = (self.page_table, self.held, self.free_pages, self.free_count)
        assert all(t.dtype is _I32 for t in parts), "a pool's tensors are int32"
        assert self.held.numel() == B and self.free_count.numel() == 1
        device = self.page_table.get_device()
        assert all(t.get_device() == device for t in parts), "tensors of one device"
        d = us_kv_pool(B, self.page_size, self.free_pages.numel(), max_pages, *(_dptr(t) for t in parts))
        for name, value in (("B", B), ("num_pages", self.free_pages.numel()), ("device", device), ("_desc", d),
                            ("_ref", ctypes.byref(d))):
            object.__setattr__(self, name, value)


def kv_pool(page_size: int, num_pages: int, B: int, max_pages: int, device="cuda") -> KVPool:
    """A pool of which all pages are free (page 0 is taken first)."""
    return KVPool(page_size, torch.full((B, max_pages), -1, dtype=_I32, device=device),
                  torch.zeros(B, dtype=_I32, device=device),
                  torch.arange(num_pages - 1, -1, -1, dtype=_I32, device=device),
                  torch.full((1,), num_pages, dtype=_I32, device=device))


def us_kv_reserve(P: KVPool, length: torch.Tensor, stream=None):
    """Request b comes to hold the pages of length[b] positions: gives back, then takes."""
    _check("us_kv_reserve", (_lib or load()).us_kv_reserve(P._ref, _i32(length, P.B, P), _raw_stream(stream, P)))


def us_kv_slots(P: KVPool, tok_off: torch.Tensor, pos: torch.Tensor, max_n: int, slots: torch.Tensor, stream=None):
    """slots[t]: the row of a pool of pages where token t's entry lies (int64; -1: nowhere)."""
    assert slots.dtype is torch.int64 and slots.is_contiguous() and slots.get_device() == P.device, \
        "slots must be contiguous int64 on the pool's device"
    _check("us_kv_slots", (_lib or load()).us_kv_slots(P._ref, slots.numel(), _i32(tok_off, P.B + 1, P), _i32(pos, P.B, P),
                                                       max_n, slots.data_ptr(), _raw_stream(stream, P)))


# ---- norm and rotation of queries and keys
def rope_freq(freq: torch.Tensor) -> torch.Tensor:
    """Frequencies in radians a position -> the 64-bit fractions of a turn that Rope takes
    (int64, the bits of uint64), on the same device."""
    turns = [int(math.ldexp(math.fmod(f / (2 * math.pi), 1.0) % 1.0, 64)) & (1 << 64) - 1 for f in freq.double().reshape(-1).tolist()]
    return torch.tensor([t - (1 << 64) if t >> 63 else t for t in turns], dtype=torch.int64, device=freq.device)


@dataclass(frozen=True, eq=False)
class Rope:
    """A rotation by position and the eps of the norm before it.  turns: R/2 frequencies
    (rope_freq) on the device; an empty tensor: no rotation."""
    style: int                # US_ROPE_HALVES or US_ROPE_PAIRS
    turns: torch.Tensor
    eps: float = 1e-6

    def __post_init__(self):
        assert self.turns.dtype in _WORDS, "turns: 64-bit words (rope_freq)"
        d = us_rope(self.style, 2 * self.turns.numel(), self.eps, 0, _dptr(self.turns))
        for name, value in (("R", 2 * self.turns.numel()), ("device", self.turns.get_device()), ("_desc", d),
                            ("_ref", ctypes.byref(d))):
            object.__setattr__(self, name, value)


def _apart(x: torch.Tensor, D: int, device: int):
    """Rows, heads, pointer and distances of T x H x D fp16 heads."""
    T, H, d = x.shape
    ld, hs, sd = x.stride()
    assert x.dtype in _HALVES and d == D and sd == 1, "heads must be T x H x D CUDA fp16 with contiguous values"
    assert x.get_device() == device, "tensors must be on one device"
    if H == 1:
        hs = D
    return T, H, x.data_ptr(), (ld if T > 1 else H * hs), hs


def _heads(x, w, y, D: int, device: int, T: int):
    """us_heads as bytes; None for no heads."""
    if x is None:
        return None
    Tx, H, xp, ld, hs = _apart(x, D, device)
    assert Tx == T, "as many rows of queries as of keys"
    yp = ldy = hsy = 0
    if y is not None:
        Ty, Hy, yp, ldy, hsy = _apart(y, D, device)
        assert Ty == T and Hy == H, "results have the shape of their inputs"
    return _pack_heads(xp, ld, hs, yp, ldy, hsy, _weight(w, D, device), H, 0)


def _weight(w, D: int, device: int) -> int:
    if w is None:
        return 0
    assert w.dtype in _HALVES and w.numel() == D and w.is_contiguous(), "weights: D contiguous CUDA fp16 values"
    assert w.get_device() == device, "tensors must be on one device"
    return w.data_ptr()


def us_norm_rope(rope: Rope, Q, wq, Qo, K, wk, Ko, tok_off: torch.Tensor, pos: torch.Tensor, depth, max_n: int, stream=None):
    """Norm (weights wq, wk of D values, or None) and rotation of T x H x D query and key
    heads (either may be None) into Qo and Ko, which may be Q and K themselves."""
    T, _, D = (Q if Q is not None else K).shape
    dev = rope.device
    _check("us_norm_rope", (_lib or load()).us_norm_rope(
        rope._ref, D, _heads(Q, wq, Qo, D, dev, T), _heads(K, wk, Ko, D, dev, T), pos.numel(), T,
        _i32(tok_off, pos.numel() + 1, rope), _i32(pos, pos.numel(), rope), None if depth is None else _i32(depth, T, rope), max_n,
        _raw_stream(stream, rope)))


def us_kv_append(C: KVCache, rope: Rope, Q, wq, Qo, K: torch.Tensor, wk, V: torch.Tensor, tok_off: torch.Tensor,
                 pos: torch.Tensor, depth, max_n: int, Ko=None, stream=None):
    """us_norm_rope of Q (or None) and K, then us_kv_write of the keys it gives and of V, in one pass."""
    T, vp, ldv = _rows(V, C.Hkv, C)
    assert K.shape[1] == C.Hkv and rope.device == C.device
    dev, D = C.device, C.D
    _check("us_kv_append", (_lib or load()).us_kv_append(
        C._ref, rope._ref, _heads(Q, wq, Qo, D, dev, T), _heads(K, wk, Ko, D, dev, T), vp, ldv, T, _i32(tok_off, C.B + 1, C),
        _i32(pos, C.B, C), None if depth is None else _i32(depth, T, C), max_n, _raw_stream(stream, C)))


# ---- the cache of latent rows, and attention over it
@dataclass(frozen=True, eq=False)
class LatCache:
    """A paged cache of latent rows over device tensors: rows (fp16, pages x slots x
    (Dc + Dr)) and the page table (int32, B x pages).  The tensors' contents may change,
    the tensors may not."""
    Dc: int
    Dr: int
    rows: torch.Tensor
    page_table: torch.Tensor

    def __post_init__(self):
        num_pages, page_size, W = self.rows.shape
        B, max_pages = self.page_table.shape
        assert W == self.Dc + self.Dr, "rows of Dc + Dr values"
        assert self.rows.dtype in _HALVES, "rows: fp16 or its bit pattern"
        assert self.page_table.dtype is _I32
        device = self.rows.get_device()
        assert self.page_table.get_device() == device, "tensors of one device"
        d = us_lat_cache(self.Dc, self.Dr, page_size, num_pages, B, max_pages, _dptr(self.rows), _dptr(self.page_table))
        for name, value in (("B", B), ("W", W), ("page_size", page_size), ("device", device), ("_desc", d),
                            ("_ref", ctypes.byref(d))):
            object.__setattr__(self, name, value)


def lat_cache(Dc: int, Dr: int, page_size: int, num_pages: int, page_table: torch.Tensor) -> LatCache:
    """An empty cache of num_pages pages on the page table's device."""
    return LatCache(Dc, Dr, torch.zeros(num_pages, page_size, Dc + Dr, dtype=_F16, device=page_table.device), page_table)


def _row2(X: torch.Tensor, W: int, device: int):
    """Rows, pointer and row distance of T x W fp16 rows."""
    T, w = X.shape
    ld, sd = X.stride()
    assert X.dtype in _HALVES and w == W and sd == 1, "rows must be T x W CUDA fp16 with contiguous values"
    assert X.get_device() == device, "tensors must be on one device"
    return T, X.data_ptr(), (ld if T > 1 else W)


def us_lat_write(C: LatCache, rope: Rope, X: torch.Tensor, w, tok_off: torch.Tensor, pos: torch.Tensor, depth, max_n: int,
                 stream=None):
    """Append rows X (T x (Dc + Dr)): latent values normed (weights w of Dc values, or None), the key rotated."""
    T, xp, ldx = _row2(X, C.W, C.device)
    assert rope.device == C.device, "tensors must be on one device"
    _check("us_lat_write", (_lib or load()).us_lat_write(
        C._ref, rope._ref, xp, ldx, _weight(w, C.Dc, C.device) or None, T, _i32(tok_off, C.B + 1, C), _i32(pos, C.B, C),
        None if depth is None else _i32(depth, T, C), max_n, _raw_stream(stream, C)))


def us_lat_read(C: LatCache, tok_off: torch.Tensor, pos: torch.Tensor, max_n: int, X: torch.Tensor, stream=None):
    """Read positions pos[b] .. back as rows (T x (Dc + Dr))."""
    T, xp, ldx = _row2(X, C.W, C.device)
    _check("us_lat_read", (_lib or load()).us_lat_read(C._ref, T, _i32(tok_off, C.B + 1, C), _i32(pos, C.B, C), max_n, xp, ldx,
                                                       _raw_stream(stream, C)))


def us_lat_commit(C: LatCache, acc_off: torch.Tensor, acc: torch.Tensor, pos: torch.Tensor, max_n: int, stream=None):
    """Move the accepted drafted tokens' rows, pos[b] + acc[i], to pos[b] + i."""
    T = acc.numel()
    _check("us_lat_commit", (_lib or load()).us_lat_commit(C._ref, T, _i32(acc_off, C.B + 1, C), _i32(acc, T, C),
                                                           _i32(pos, C.B, C), max_n, _raw_stream(stream, C)))


def us_attn_lat_workspace_bytes(C: LatCache, Hq: int, max_n: int) -> int:
    n = ctypes.c_size_t()
    _check("us_attn_lat_workspace_bytes", load().us_attn_lat_workspace_bytes(C._ref, Hq, max_n, ctypes.byref(n)))
    return n.value


def workspace_attn_lat(C: LatCache, Hq: int, max_n: int) -> torch.Tensor:
    """A zero-filled workspace of the size us_attn_lat needs."""
    return torch.zeros(max(us_attn_lat_workspace_bytes(C, Hq, max_n), 16), dtype=torch.uint8, device=C.rows.device)


def _packed(x: torch.Tensor, H: int, D: int, device: int):
    """Rows, pointer and row distance of T x H x D fp16 rows whose heads are side by side."""
    T, h, d = x.shape
    ld, sh, sd = x.stride()
    assert x.dtype in _HALVES and h == H and d == D and sd == 1 and (sh == d or H == 1), \
        "rows must be T x H x D CUDA fp16 with contiguous heads"
    assert x.get_device() == device, "tensors must be on one device"
    return T, x.data_ptr(), (ld if T > 1 else H * D)


def _space(ws: torch.Tensor, device: int) -> int:
    assert ws.is_contiguous() and ws.get_device() == device, "ws must be contiguous, on the call's device"
    return ws.numel() * ws.element_size()


def us_attn_lat(C: LatCache, Q: torch.Tensor, tok_off: torch.Tensor, pos: torch.Tensor, mask, max_n: int, scale: float,
                O: torch.Tensor, ws: torch.Tensor, stream=None):
    """Attention of T x Hq x (Dc + Dr) query rows over the latent rows, to T x Hq x Dc; mask as in us_attn_kv."""
    Hq, dev = Q.shape[1], C.device
    T, qp, ldq = _packed(Q, Hq, C.W, dev)
    To, op, ldo = _packed(O, Hq, C.Dc, dev)
    assert T == To
    if mask is not None:
        assert mask.dtype in _WORDS and mask.numel() == T and mask.is_contiguous(), "mask must be T CUDA 64-bit words"
        assert mask.get_device() == dev, "mask must be on the cache's device"
    _check("us_attn_lat", (_lib or load()).us_attn_lat(C._ref, qp, ldq, Hq, T, _i32(tok_off, C.B + 1, C), _i32(pos, C.B, C),
                                                       None if mask is None else mask.data_ptr(), max_n, scale, op, ldo,
                                                       ws.data_ptr(), _space(ws, dev), _raw_stream(stream, C)))


def us_attn_rows_workspace_bytes(Dn: int, Dr: int, Dv: int, H: int, B: int, max_n: int) -> int:
    n = ctypes.c_size_t()
    a = _pack_rows(Dn, Dr, Dv, H, 0, 0, 0, 0, 0, 0, 0, 0, 0)
    _check("us_attn_rows_workspace_bytes", load().us_attn_rows_workspace_bytes(a, B, max_n, ctypes.byref(n)))
    return n.value


def workspace_attn_rows(Dn: int, Dr: int, Dv: int, H: int, B: int, max_n: int, device="cuda") -> torch.Tensor:
    """A zero-filled workspace of the size us_attn_rows needs."""
    return torch.zeros(max(us_attn_rows_workspace_bytes(Dn, Dr, Dv, H, B, max_n), 16), dtype=torch.uint8, device=device)


class _On:
    """A device, where a call has no object that names it."""
    __slots__ = ("device",)

    def __init__(self, device):
        self.device = device


def us_attn_rows(Q: torch.Tensor, K: torch.Tensor, KR: torch.Tensor, V: torch.Tensor, tok_off: torch.Tensor,
                 kv_off: torch.Tensor, max_n: int, scale: float, O: torch.Tensor, ws: torch.Tensor, stream=None):
    """Causal attention of T x H x (Dn + Dr) query rows, the last of their requests' key
    rows, over S x H x Dn keys K, the S x Dr key part KR that all heads share and
    S x H x Dv values V, to T x H x Dv."""
    on = _On(Q.get_device())
    dev, H, S = on.device, Q.shape[1], K.shape[0]
    Dn, Dr, Dv = K.shape[2], KR.shape[1], V.shape[2]
    T, qp, ldq = _packed(Q, H, Dn + Dr, dev)
    To, op, ldo = _packed(O, H, Dv, dev)
    Sk, Hk, kp, ldk, hsk = _apart(K, Dn, dev)
    Sv, Hv, vp, ldv, hsv = _apart(V, Dv, dev)
    Sr, rp, ldkr = _row2(KR, Dr, dev)
    assert T == To and Sv == S and Sr == S and Hk == H and Hv == H, "K, KR and V have the same rows, K and V Q's heads"
    B = tok_off.numel() - 1
    a = _pack_rows(Dn, Dr, Dv, H, kp, ldk, hsk, rp, ldkr, vp, ldv, hsv, S)
    _check("us_attn_rows", (_lib or load()).us_attn_rows(a, qp, ldq, B, T, _i32(tok_off, B + 1, on), _i32(kv_off, B + 1, on), max_n,
                                                         scale, op, ldo, ws.data_ptr(), _space(ws, dev), _raw_stream(stream, on)))


def us_validate_host(bitmap, tile_off, values, M, K, TM, TK, elem, order) -> int:
    """us_validate on host numpy arrays; returns the status code."""
    import numpy as np
    bm = np.ascontiguousarray(bitmap, dtype=np.uint64)
    off = np.ascontiguousarray(tile_off, dtype=np.uint32)
    v = np.ascontiguousarray(values, dtype=np.uint8)
    d = us_bitmap(M, K, TM, TK, elem, order, bm.ctypes.data, off.ctypes.data,
                  v.ctypes.data if v.size else None, v.size, 0, 0)
    return int(load().us_validate(ctypes.byref(d)))


def us_selftest_wait_timeout(limit_ns: int, elapsed: torch.Tensor | None = None, stream=None):
    """Run the bounded-wait self-test: one device wait that nothing completes,
    given up after limit_ns (elapsed: optional int64 device tensor of one element)."""
    _check("us_selftest_wait_timeout", load().us_selftest_wait_timeout(int(limit_ns), _dptr(elapsed),
                                                                       _stream(stream)))


def us_get_last_device_status(stream=None) -> int:
    return int(load().us_get_last_device_status(_stream(stream)))
