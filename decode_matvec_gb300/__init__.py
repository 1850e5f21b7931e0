"""Python binding of ``libqmoe.so``: the GB300 fused decode-and-multiply library.

Argument marshalling only: every step of the hot path runs in the library's
CUDA kernels (``include/qmoe.h`` documents each call).  PyTorch supplies device
memory and streams.  Importing this package fails loudly when the library has
not been built (``python decode_matvec_gb300/build.py``); there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqmoe.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python decode_matvec_gb300/build.py` "
                      "(or __graft_entry__.build()); there is no non-CUDA fallback")
_lib = ctypes.CDLL(LIB_PATH)

QMOE_OK, QMOE_EINVAL, QMOE_ECAPACITY, QMOE_ECUDA, QMOE_EFORMAT, QMOE_ETIMEOUT, QMOE_EUNSUPPORTED = 0, -1, -2, -3, -4, -5, -6
STATUS_NAMES = {0: "QMOE_OK", -1: "QMOE_EINVAL", -2: "QMOE_ECAPACITY", -3: "QMOE_ECUDA", -4: "QMOE_EFORMAT",
                -5: "QMOE_ETIMEOUT", -6: "QMOE_EUNSUPPORTED"}
DICT_ENTRIES = 65536
DICT_WORDS = 2 * DICT_ENTRIES
COMPACT_BYTES = 7 * DICT_ENTRIES
QMOE_VQ_RVQ, QMOE_VQ_E8P = 0, 1      # code formats of an RVQ matrix set

EXPORTED = [
    "qmoe_encode_dictionary", "qmoe_pack", "qmoe_dict_compact", "qmoe_expert_matvec", "qmoe_route",
    "qmoe_bucketise", "qmoe_moe_layer_ws_size", "qmoe_moe_layer", "rvq_expert_matmul_ws_size",
    "rvq_expert_matmul", "rvq_moe_layer_ws_size", "rvq_moe_layer", "rvq_pack", "qmoe_check_status",
    "qmoe_last_error", "qmoe_decode_dense", "rvq_decode_dense", "qmoe_set_phase_events",
    "qmoe_moe_layer_noalloc", "qmoe_pack_device_ws_size", "qmoe_pack_device", "rvq_pack_stages",
    "rvq_stage_allocation", "e8p_base_table", "e8p_pack", "e8p_nearest", "qmoe_offsets_compact",
    "qmoe_moe_layer_kernels", "kv4_block_tables", "qk_norm_rope", "kv4_append", "kv4_gather",
    "kv4_attention_ws_size", "kv4_attention", "kv4_block_tables_bounded", "add_rms_norm", "qmoe_route_scored",
    "kv4_block_bounds", "kv4_select_blocks_ws_size", "kv4_select_blocks", "kv4_attention_blocks_ws_size",
    "kv4_attention_blocks",
]


class QmoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        msg = _lib.qmoe_last_error().decode()
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


def _check(status: int, where: str) -> None:
    if status != QMOE_OK:
        raise QmoeError(status, where)


# ------------------------------------------------------------------ C structs
class CDict(ctypes.Structure):
    _fields_ = [("words", ctypes.c_void_p), ("compact", ctypes.c_void_p)]


class CMatrixSet(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("code_base", ctypes.c_void_p), ("row_off", ctypes.c_void_p),
                ("blk_len", ctypes.c_void_p),
                ("scale_f16", ctypes.c_void_p), ("count", ctypes.c_int), ("rows", ctypes.c_int),
                ("cols", ctypes.c_int), ("block", ctypes.c_int)]


class CRvqSet(ctypes.Structure):
    _fields_ = [("idx", ctypes.c_void_p), ("codebooks", ctypes.c_void_p), ("scale_f16", ctypes.c_void_p),
                ("sign_out", ctypes.c_void_p), ("sign_in", ctypes.c_void_p), ("count", ctypes.c_int),
                ("rows", ctypes.c_int), ("cols", ctypes.c_int), ("stages", ctypes.c_void_p),
                ("idx_base", ctypes.c_void_p), ("n_stages", ctypes.c_int), ("format", ctypes.c_int)]


class CKv4Cache(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_void_p), ("n_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("n_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int)]


class CKv4Bounds(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("steps", ctypes.c_void_p), ("n_pages", ctypes.c_int),
                ("page_size", ctypes.c_int), ("n_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int)]


_vp, _i, _sz, _d = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_double
_i64, _f = ctypes.c_int64, ctypes.c_float
_sig = {
    "qmoe_encode_dictionary": [_vp, _sz, _d, _vp, _vp],
    "qmoe_pack": [_vp, _i, _i, _i, _vp, _vp, _sz, _vp, _vp],
    "qmoe_dict_compact": [_vp, _vp],
    "qmoe_expert_matvec": [_vp, _vp, _vp, _i, _vp, _i, _vp],
    "qmoe_route": [_vp, _i, _i, _i, _vp, _vp, _vp],
    "qmoe_bucketise": [_vp, _i, _i, _i, _vp, _vp, _vp, _vp],
    "qmoe_moe_layer_ws_size": [_i, _i, _i, _i, _i, _vp],
    "qmoe_moe_layer_kernels": [_i, _i, _i, _i, _i, _vp, _vp, _vp],
    "qmoe_moe_layer": [_vp, _vp, _vp, _vp, _i, _i, _vp, _vp, _vp, _i, _vp, _sz, _vp],
    "rvq_expert_matmul_ws_size": [_i, _i, _i, _vp],
    "rvq_expert_matmul": [_vp, _vp, _i, _vp, _i, _vp, _sz, _vp],
    "rvq_moe_layer_ws_size": [_i, _i, _i, _i, _i, _vp],
    "rvq_moe_layer": [_vp, _vp, _vp, _vp, _i, _i, _vp, _vp, _vp, _i, _vp, _sz, _vp],
    "rvq_pack": [_vp, _i, _i, _vp, _vp, _vp, _vp, _vp],
    "qmoe_check_status": [_vp],
    "qmoe_decode_dense": [_vp, _vp, _vp, _vp],
    "rvq_decode_dense": [_vp, _vp, _vp],
    "qmoe_set_phase_events": [_vp, _i],
    "qmoe_moe_layer_noalloc": [_vp, _vp, _vp, _vp, _i, _i, _vp, _vp, _vp, _i, _vp],
    "qmoe_pack_device_ws_size": [_i, _i, _i, _vp],
    "qmoe_pack_device": [_vp, _vp, _i, _i, _i, _vp, _sz, _vp, _vp, _sz, _vp],
    "rvq_pack_stages": [_vp, _i, _i, _vp, _vp, _vp, _i, _vp, _vp],
    "rvq_stage_allocation": [_vp, _i, _i, _vp],
    "e8p_base_table": [_vp],
    "e8p_pack": [_vp, _i, _i, _vp, _vp, _vp, _vp],
    "e8p_nearest": [_vp, _sz, _vp],
    "qmoe_offsets_compact": [_vp, _i, _i, _vp, _vp],
    "kv4_block_tables": [_vp, _vp, _i, _vp, _vp, _i, _vp, _i, _vp, _vp, _vp, _vp, _i, _vp, _vp],
    "kv4_block_tables_bounded": [_vp, _vp, _i, _vp, _i, _vp, _i, _vp, _i, _vp, _vp, _vp, _vp, _i, _vp, _vp],
    "qk_norm_rope": [_vp, _i64, _i, _i, _i, _i, _vp, _vp, _f, _vp, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp],
    "kv4_append": [_vp, _vp, _i64, _vp, _i64, _i, _vp, _vp],
    "kv4_gather": [_vp, _vp, _i, _vp, _vp, _vp],
    "kv4_attention_ws_size": [_i, _i, _i, _i, _i, _i, _i, _vp],
    "kv4_attention": [_vp, _vp, _i, _i, _vp, _vp, _i, _vp, _i, _i, _i, _f, _i, _i, _vp, _vp, _sz, _vp],
    "add_rms_norm": [_vp, _i, _i64, _vp, _i64, _vp, _i64, _vp, _i, _i, _f, _vp, _i64, _vp, _vp, _i, _vp],
    "qmoe_route_scored": [_vp, _i, _i64, _i, _i, _i, _i, _vp, _i, _i, _i, _i, _f, _vp, _vp, _vp],
    "kv4_block_bounds": [_vp, _vp, _vp, _i, _vp],
    "kv4_select_blocks_ws_size": [_i, _i, _i, _i, _vp],
    "kv4_select_blocks": [_vp, _vp, _i, _i, _vp, _vp, _i, _vp, _i, _i, _i, _i, _i, _vp, _vp, _sz, _vp],
    "kv4_attention_blocks_ws_size": [_i, _i, _i, _i, _i, _i, _vp],
    "kv4_attention_blocks": [_vp, _vp, _i, _i, _vp, _vp, _i, _vp, _i, _vp, _i, _f, _vp, _vp, _sz, _vp],
}
for _name, _args in _sig.items():
    _f = getattr(_lib, _name)
    _f.argtypes = _args
    _f.restype = ctypes.c_int
_lib.qmoe_last_error.argtypes = []
_lib.qmoe_last_error.restype = ctypes.c_char_p


def lib() -> ctypes.CDLL:
    return _lib


def _np_ptr(a: np.ndarray) -> int:
    return a.ctypes.data if a is not None else None


_raw_stream = None      # (index of the current device, handle of a device's current stream), looked up on first use


def _raw():
    # (private names of torch: the public torch.cuda.current_stream() makes a Stream object, 3 us a call against 0.2)
    global _raw_stream
    if _raw_stream is None:
        import torch
        torch.cuda.init()
        _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
    return _raw_stream


def _stream_ptr(stream) -> int:
    if stream is not None:
        return int(stream.cuda_stream)
    device, current = _raw_stream or _raw()
    return current(device())


def _dptr(t) -> int | None:
    return None if t is None else int(t.data_ptr())


# ================================================================ host codec
def qmoe_encode_dictionary(p0: float | None = None, symbols: np.ndarray | None = None):
    """Algorithm 1 dictionary as uint32[2*65536], plus the p0 it was built for."""
    words = np.zeros(DICT_WORDS, dtype=np.uint32)
    used = ctypes.c_double(0.0)
    sym = None if symbols is None else np.ascontiguousarray(symbols, dtype=np.int8)
    _check(_lib.qmoe_encode_dictionary(_np_ptr(sym), 0 if sym is None else sym.size,
                                       float(p0 if p0 is not None else 0.0), _np_ptr(words), ctypes.byref(used)),
           "qmoe_encode_dictionary")
    return words, used.value


def qmoe_pack(tern: np.ndarray, dict_words: np.ndarray, block: int = 256):
    """Greedy longest-match codewords (uint16) and per-block offsets (uint32) of a ternary matrix."""
    tern = np.ascontiguousarray(tern, dtype=np.int8)
    rows, cols = tern.shape
    words = np.ascontiguousarray(dict_words, dtype=np.uint32)
    n = ctypes.c_size_t(0)
    _check(_lib.qmoe_pack(_np_ptr(tern), rows, cols, block, _np_ptr(words), None, 0, ctypes.byref(n), None),
           "qmoe_pack(count)")
    nb = (cols + block - 1) // block
    codes = np.zeros(max(n.value, 1), dtype=np.uint16)
    off = np.zeros(rows * nb + 1, dtype=np.uint32)
    _check(_lib.qmoe_pack(_np_ptr(tern), rows, cols, block, _np_ptr(words), _np_ptr(codes), codes.size,
                          ctypes.byref(n), _np_ptr(off)), "qmoe_pack")
    return codes[:n.value], off


def qmoe_pack_into(tern: np.ndarray, dict_words: np.ndarray, block: int, codes_out: np.ndarray,
                   off_out: np.ndarray) -> int:
    """Pack into caller buffers (views); returns the codeword count.  Releases the GIL while packing."""
    tern = np.ascontiguousarray(tern, dtype=np.int8)
    rows, cols = tern.shape
    n = ctypes.c_size_t(0)
    _check(_lib.qmoe_pack(_np_ptr(tern), rows, cols, block, _np_ptr(dict_words), _np_ptr(codes_out),
                          codes_out.size, ctypes.byref(n), _np_ptr(off_out)), "qmoe_pack")
    return n.value


def qmoe_dict_compact(dict_words: np.ndarray) -> np.ndarray:
    words = np.ascontiguousarray(dict_words, dtype=np.uint32)
    out = np.zeros(COMPACT_BYTES, dtype=np.uint8)
    _check(_lib.qmoe_dict_compact(_np_ptr(words), _np_ptr(out)), "qmoe_dict_compact")
    return out


def rvq_pack(w: np.ndarray, sign_out: np.ndarray, sign_in: np.ndarray, codebooks_f16: np.ndarray,
             stages: int | None = None):
    """Host RVQ encoder: (idx uint8 [rows, cols/8, S], scale fp16 bits [rows]); S = stages, by default
    the number of codebooks given ([S_max, 256, 8] fp16 bits; the first S are used)."""
    w = np.ascontiguousarray(w, dtype=np.float64)
    rows, cols = w.shape
    so = np.ascontiguousarray(sign_out, dtype=np.int8)
    si = np.ascontiguousarray(sign_in, dtype=np.int8)
    cb = np.ascontiguousarray(codebooks_f16, dtype=np.uint16)
    n_st = cb.shape[0] if stages is None else int(stages)
    if not 1 <= n_st <= cb.shape[0]:
        raise ValueError("stage count outside 1 .. number of codebooks")
    idx = np.zeros((rows, cols // 8, n_st), dtype=np.uint8)
    sc = np.zeros(rows, dtype=np.uint16)
    _check(_lib.rvq_pack_stages(_np_ptr(w), rows, cols, _np_ptr(so), _np_ptr(si), _np_ptr(cb), n_st, _np_ptr(idx),
                                _np_ptr(sc)), "rvq_pack_stages")
    return idx, sc


def rvq_stage_allocation(popularity: np.ndarray, s_bar: int = 2) -> np.ndarray:
    """Stages per expert by popularity thirds (s_bar + 1 / s_bar / s_bar - 1), uint8 [E]."""
    pop = np.ascontiguousarray(popularity, dtype=np.float64)
    out = np.zeros(pop.shape[0], dtype=np.uint8)
    _check(_lib.rvq_stage_allocation(_np_ptr(pop), pop.shape[0], int(s_bar), _np_ptr(out)), "rvq_stage_allocation")
    return out


def e8p_base_table() -> np.ndarray:
    """The E8P base table: uint32 [256], nibble j of entry p = 2|a_j| of absolute pattern p."""
    out = np.zeros(256, dtype=np.uint32)
    _check(_lib.e8p_base_table(_np_ptr(out)), "e8p_base_table")
    return out


def e8p_pack(w: np.ndarray, sign_out: np.ndarray, sign_in: np.ndarray):
    """Host E8P encoder: (code words uint16 [rows, cols/8], scale fp16 bits [rows])."""
    w = np.ascontiguousarray(w, dtype=np.float64)
    rows, cols = w.shape
    so = np.ascontiguousarray(sign_out, dtype=np.int8)
    si = np.ascontiguousarray(sign_in, dtype=np.int8)
    codes = np.zeros((rows, cols // 8), dtype=np.uint16)
    sc = np.zeros(rows, dtype=np.uint16)
    _check(_lib.e8p_pack(_np_ptr(w), rows, cols, _np_ptr(so), _np_ptr(si), _np_ptr(codes), _np_ptr(sc)), "e8p_pack")
    return codes, sc


def e8p_nearest(u: np.ndarray) -> np.ndarray:
    """Code words (uint16 [n]) of the E8P codewords nearest to the rows of u [n, 8]."""
    u = np.ascontiguousarray(u, dtype=np.float64).reshape(-1, 8)
    out = np.zeros(u.shape[0], dtype=np.uint16)
    _check(_lib.e8p_nearest(_np_ptr(u), u.shape[0], _np_ptr(out)), "e8p_nearest")
    return out


def qmoe_last_error() -> str:
    return _lib.qmoe_last_error().decode()


def qmoe_check_status(stream=None) -> int:
    return _lib.qmoe_check_status(_stream_ptr(stream))


# ================================================================ device objects
class Dictionary:
    """Canonical words and the derived compact table, resident on the device."""

    def __init__(self, words: np.ndarray, device="cuda"):
        import torch
        w = np.ascontiguousarray(words, dtype=np.uint32)
        compact = qmoe_dict_compact(w)
        self.words_host = w
        self.words = torch.from_numpy(w.view(np.int32)).to(device)
        self.compact = torch.from_numpy(compact).to(device)
        self.c = CDict(_dptr(self.words), _dptr(self.compact))


class MatrixSet:
    """`count` dictionary-coded matrices of one shape, resident on the device, with compact offsets:
    row_off uint32 [count][rows + 1] and blk_len uint8 [count][rows][nb - 1] (qmoe_offsets_compact)."""

    def __init__(self, codes, code_base, row_off, blk_len, scale_f16, count, rows, cols, block=256):
        self.codes, self.code_base, self.row_off, self.blk_len, self.scale = codes, code_base, row_off, blk_len, scale_f16
        self.count, self.rows, self.cols, self.block = count, rows, cols, block
        self.c = CMatrixSet(_dptr(codes), _dptr(code_base), _dptr(row_off), _dptr(blk_len), _dptr(scale_f16), count,
                            rows, cols, block)

    @property
    def nb(self) -> int:
        return (self.cols + self.block - 1) // self.block

    @classmethod
    def from_host(cls, codes: np.ndarray, blk_off: np.ndarray, scale_f16: np.ndarray, rows, cols, block=256,
                  code_base: np.ndarray | None = None, count: int = 1, device="cuda"):
        """From qmoe_pack's output (uint32 block offsets [count][rows*nb + 1]), re-encoded compactly."""
        import torch
        codes = np.ascontiguousarray(codes, dtype=np.uint16)
        padded = np.zeros((codes.size + 15) // 8 * 8, dtype=np.uint16)     # whole 16-byte chunks, plus one
        padded[:codes.size] = codes
        c = torch.from_numpy(padded.view(np.int16)).to(device)
        row_off, blk_len = qmoe_offsets_compact(blk_off, rows, (cols + block - 1) // block, count)
        o = torch.from_numpy(row_off.view(np.int32).copy()).to(device)
        bl = torch.from_numpy(blk_len.copy()).to(device) if blk_len.size else None
        s = torch.from_numpy(np.ascontiguousarray(scale_f16, dtype=np.uint16).view(np.int16).copy()).to(device)
        b = None
        if code_base is not None:
            b = torch.from_numpy(np.ascontiguousarray(code_base, dtype=np.uint64).view(np.int64).copy()).to(device)
        return cls(c, b, o, bl, s, count, rows, cols, block)

    def expert(self, e: int, code_base_host=None) -> "MatrixSet":
        """A one-matrix set for matrix e (views into the same device buffers); code_base_host: the host copy
        of the set's code bases (needed when count > 1)."""
        base = int(code_base_host[e]) if self.count > 1 else 0
        nb1 = self.nb - 1
        return MatrixSet(self.codes[base:], None, self.row_off[e * (self.rows + 1):(e + 1) * (self.rows + 1)],
                         self.blk_len[e * self.rows * nb1:(e + 1) * self.rows * nb1] if nb1 else None,
                         self.scale[e * self.rows:(e + 1) * self.rows], 1, self.rows, self.cols, self.block)


def qmoe_offsets_compact(blk_off: np.ndarray, rows: int, nb: int, count: int = 1):
    """Compact offsets of `count` matrices from their uint32 block offsets [count][rows*nb + 1]:
    (row_off uint32 [count*(rows + 1)], blk_len uint8 [count*rows*(nb - 1)])."""
    bo = np.ascontiguousarray(blk_off, dtype=np.uint32).reshape(count, rows * nb + 1)
    row_off = np.zeros((count, rows + 1), dtype=np.uint32)
    blk_len = np.zeros((count, rows * (nb - 1)), dtype=np.uint8)
    for e in range(count):
        _check(_lib.qmoe_offsets_compact(_np_ptr(bo[e]), rows, nb, _np_ptr(row_off[e]),
                                         _np_ptr(blk_len[e]) if nb > 1 else None), "qmoe_offsets_compact")
    return row_off.reshape(-1), blk_len.reshape(-1)


class RvqMatrixSet:
    """`count` RVQ-coded matrices of one shape, resident on the device.  With `stages` (device uint8 per
    matrix) and `idx_base` (device int64 byte offsets), matrices may have 1 .. n_stages stages each."""

    def __init__(self, idx, codebooks, scale_f16, sign_out, sign_in, count, rows, cols, stages=None, idx_base=None,
                 n_stages=0, fmt=QMOE_VQ_RVQ):
        self.idx, self.codebooks, self.scale, self.sign_out, self.sign_in = idx, codebooks, scale_f16, sign_out, sign_in
        self.count, self.rows, self.cols = count, rows, cols
        self.stages, self.idx_base, self.n_stages, self.fmt = stages, idx_base, n_stages, fmt
        self.c = CRvqSet(_dptr(idx), _dptr(codebooks), _dptr(scale_f16), _dptr(sign_out), _dptr(sign_in), count,
                         rows, cols, _dptr(stages), _dptr(idx_base), n_stages, fmt)

    @classmethod
    def e8p_from_host(cls, codes, scale_f16, sign_out, sign_in, count, rows, cols, device="cuda"):
        """E8P set: codes uint16 [count, rows, cols/8]; the base table comes from e8p_base_table."""
        import torch

        def up(a, dt, view):
            return torch.from_numpy(np.ascontiguousarray(a, dtype=dt).view(view).copy()).to(device)
        return cls(up(codes, np.uint16, np.int16), up(e8p_base_table(), np.uint32, np.int32),
                   up(scale_f16, np.uint16, np.int16), up(sign_out, np.int8, np.int8), up(sign_in, np.int8, np.int8),
                   count, rows, cols, fmt=QMOE_VQ_E8P)

    @classmethod
    def from_host(cls, idx, codebooks_f16, scale_f16, sign_out, sign_in, count, rows, cols, device="cuda"):
        """idx: uint8 [count, rows, cols/8, 2] (two stages each), or a list of count arrays
        [rows, cols/8, S_e] with per-matrix stage counts (each matrix's codes start 16-byte aligned)."""
        import torch

        def up(a, dt, view):
            return torch.from_numpy(np.ascontiguousarray(a, dtype=dt).view(view).copy()).to(device)
        cb = np.ascontiguousarray(codebooks_f16, dtype=np.uint16)
        if isinstance(idx, (list, tuple)):
            st = np.array([a.shape[2] for a in idx], dtype=np.uint8)
            sizes = [a.size for a in idx]
            base = np.zeros(count, dtype=np.int64)
            off = 0
            for e, n in enumerate(sizes):
                base[e] = off
                off += (n + 15) // 16 * 16
            flat = np.zeros(max(off, 16), dtype=np.uint8)
            for e, a in enumerate(idx):
                flat[base[e]:base[e] + sizes[e]] = np.ascontiguousarray(a, dtype=np.uint8).reshape(-1)
            return cls(up(flat, np.uint8, np.uint8), up(cb, np.uint16, np.int16), up(scale_f16, np.uint16, np.int16),
                       up(sign_out, np.int8, np.int8), up(sign_in, np.int8, np.int8), count, rows, cols,
                       stages=up(st, np.uint8, np.uint8), idx_base=up(base, np.int64, np.int64), n_stages=cb.shape[0])
        return cls(up(idx, np.uint8, np.uint8), up(cb, np.uint16, np.int16),
                   up(scale_f16, np.uint16, np.int16), up(sign_out, np.int8, np.int8), up(sign_in, np.int8, np.int8),
                   count, rows, cols, n_stages=cb.shape[0])


# ================================================================ device calls
def qmoe_expert_matvec(d: Dictionary, m: MatrixSet, x, y, y_is_f32: bool = True, stream=None):
    """y[T, rows] = x[T, cols] W^T (x: int16-viewed bf16 tensor on the device)."""
    T = int(x.shape[0]) if x.dim() == 2 else 1
    _check(_lib.qmoe_expert_matvec(ctypes.byref(d.c), ctypes.byref(m.c), _dptr(x), T, _dptr(y), int(bool(y_is_f32)),
                                   _stream_ptr(stream)), "qmoe_expert_matvec")
    return y


def qmoe_decode_dense(d: Dictionary, m: MatrixSet, w_out, stream=None):
    _check(_lib.qmoe_decode_dense(ctypes.byref(d.c), ctypes.byref(m.c), _dptr(w_out), _stream_ptr(stream)),
           "qmoe_decode_dense")
    return w_out


def qmoe_route(logits, k: int, ids, gates, stream=None):
    T, E = logits.shape
    _check(_lib.qmoe_route(_dptr(logits), T, E, k, _dptr(ids), _dptr(gates), _stream_ptr(stream)), "qmoe_route")
    return ids, gates


def qmoe_bucketise(ids, E: int, counts, offsets, perm, stream=None):
    T, k = ids.shape
    _check(_lib.qmoe_bucketise(_dptr(ids), T, k, E, _dptr(counts), _dptr(offsets), _dptr(perm), _stream_ptr(stream)),
           "qmoe_bucketise")


def qmoe_pack_device_ws_size(rows: int, cols: int, block: int = 256) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.qmoe_pack_device_ws_size(rows, cols, block, ctypes.byref(n)), "qmoe_pack_device_ws_size")
    return n.value


def qmoe_pack_device(d: Dictionary, tern, codes, blk_off, workspace, block: int = 256, stream=None):
    """Device encoder: codewords and block offsets of the int8 ternary matrix `tern` (device tensor
    [rows, cols]) into `codes` (int16-viewed uint16) and `blk_off` (int32-viewed uint32, rows*nb + 1).
    The codeword count is blk_off[-1] once the stream has reached the end of the call."""
    rows, cols = tern.shape
    _check(_lib.qmoe_pack_device(ctypes.byref(d.c), _dptr(tern), rows, cols, block, _dptr(codes),
                                 int(codes.numel()), _dptr(blk_off), _dptr(workspace), int(workspace.numel()),
                                 _stream_ptr(stream)), "qmoe_pack_device")
    return codes, blk_off


def qmoe_moe_layer_ws_size(E, d_model, d_ff, T, k) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.qmoe_moe_layer_ws_size(E, d_model, d_ff, T, k, ctypes.byref(n)), "qmoe_moe_layer_ws_size")
    return n.value


QMOE_KERNEL_FLAT, QMOE_KERNEL_ROWS, QMOE_KERNEL_FLAT_L2 = 0, 1, 2
KERNEL_NAMES = {QMOE_KERNEL_FLAT: "dict_gemm_kernel", QMOE_KERNEL_ROWS: "dict_rows_kernel",
                QMOE_KERNEL_FLAT_L2: "dict_gemm_kernel"}


def qmoe_moe_layer_kernels(E, d_model, d_ff, T, k):
    """(wi kernel, wo kernel, tensor-core launch) of a qmoe_moe_layer call with these shapes."""
    wi, wo, tc = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0)
    _check(_lib.qmoe_moe_layer_kernels(E, d_model, d_ff, T, k, ctypes.byref(wi), ctypes.byref(wo), ctypes.byref(tc)),
           "qmoe_moe_layer_kernels")
    return wi.value, wo.value, bool(tc.value)


def qmoe_moe_layer(d: Dictionary, wi: MatrixSet, wo: MatrixSet, x, ids, gates, y, workspace, y_is_f32=True,
                   stream=None):
    T, k = ids.shape
    _check(_lib.qmoe_moe_layer(ctypes.byref(d.c), ctypes.byref(wi.c), ctypes.byref(wo.c), _dptr(x), T, k, _dptr(ids),
                               _dptr(gates), _dptr(y), int(bool(y_is_f32)), _dptr(workspace),
                               workspace.numel() * workspace.element_size(), _stream_ptr(stream)), "qmoe_moe_layer")
    return y


def qmoe_moe_layer_noalloc(d: Dictionary, wi: MatrixSet, wo: MatrixSet, x, ids, gates, y, y_is_f32=True,
                           stream=None):
    """qmoe_moe_layer with its scratch in the library's static device buffer (no workspace)."""
    T, k = ids.shape
    _check(_lib.qmoe_moe_layer_noalloc(ctypes.byref(d.c), ctypes.byref(wi.c), ctypes.byref(wo.c), _dptr(x), T, k,
                                       _dptr(ids), _dptr(gates), _dptr(y), int(bool(y_is_f32)), _stream_ptr(stream)),
           "qmoe_moe_layer_noalloc")
    return y


def rvq_expert_matmul_ws_size(rows, cols, T) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.rvq_expert_matmul_ws_size(rows, cols, T, ctypes.byref(n)), "rvq_expert_matmul_ws_size")
    return n.value


def rvq_expert_matmul(m: RvqMatrixSet, x, y, workspace, y_is_f32=True, stream=None):
    T = int(x.shape[0])
    _check(_lib.rvq_expert_matmul(ctypes.byref(m.c), _dptr(x), T, _dptr(y), int(bool(y_is_f32)), _dptr(workspace),
                                  workspace.numel() * workspace.element_size(), _stream_ptr(stream)),
           "rvq_expert_matmul")
    return y


def rvq_moe_layer_ws_size(E, d_model, d_ff, T, k) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.rvq_moe_layer_ws_size(E, d_model, d_ff, T, k, ctypes.byref(n)), "rvq_moe_layer_ws_size")
    return n.value


def rvq_moe_layer(gate: RvqMatrixSet, up: RvqMatrixSet, down: RvqMatrixSet, x, ids, gates, y, workspace,
                  y_is_f32=True, stream=None):
    T, k = ids.shape
    _check(_lib.rvq_moe_layer(ctypes.byref(gate.c), ctypes.byref(up.c), ctypes.byref(down.c), _dptr(x), T, k,
                              _dptr(ids), _dptr(gates), _dptr(y), int(bool(y_is_f32)), _dptr(workspace),
                              workspace.numel() * workspace.element_size(), _stream_ptr(stream)), "rvq_moe_layer")
    return y


def rvq_decode_dense(m: RvqMatrixSet, w_out, stream=None):
    _check(_lib.rvq_decode_dense(ctypes.byref(m.c), _dptr(w_out), _stream_ptr(stream)), "rvq_decode_dense")
    return w_out


def qmoe_set_phase_events(events) -> None:
    """Install (list of torch.cuda.Event, 6..8 of them) or clear (None) the phase-event hook."""
    if not events:
        _check(_lib.qmoe_set_phase_events(None, 0), "qmoe_set_phase_events")
        return
    arr = (ctypes.c_void_p * len(events))(*[int(e.cuda_event) for e in events])
    _check(_lib.qmoe_set_phase_events(arr, len(events)), "qmoe_set_phase_events")


# ================================================================ attention over the 4-bit cache
class Kv4Cache:
    """One layer's keys and values in 4 bits: a handle on `pages`, a contiguous uint8 device tensor
    [n_pages, page_bytes] (``kv4_cache`` in qmoe.h documents the layout)."""

    def __init__(self, pages, page_size: int, n_kv_heads: int, head_dim: int):
        import torch
        nbytes = self.page_bytes(page_size, n_kv_heads, head_dim)
        if pages.dtype != torch.uint8 or pages.dim() != 2 or pages.shape[1] != nbytes or not pages.is_contiguous():
            raise ValueError(f"pages must be a contiguous uint8 tensor [n_pages, {nbytes}]")
        if not pages.is_cuda:
            raise ValueError("pages must be on a CUDA device")
        self.pages, self.page_size, self.n_kv_heads, self.head_dim = pages, page_size, n_kv_heads, head_dim
        self.device = pages.get_device()
        self.n_pages = int(pages.shape[0])
        self.c = CKv4Cache(_dptr(pages), self.n_pages, page_size, n_kv_heads, head_dim)
        self.ref = ctypes.byref(self.c)

    @staticmethod
    def page_bytes(page_size: int, n_kv_heads: int, head_dim: int) -> int:
        return n_kv_heads * page_size * (head_dim + 8)

    @classmethod
    def empty(cls, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int, device="cuda") -> "Kv4Cache":
        import torch
        pages = torch.zeros((n_pages, cls.page_bytes(page_size, n_kv_heads, head_dim)), dtype=torch.uint8, device=device)
        return cls(pages, page_size, n_kv_heads, head_dim)


def _refuse(what: str):
    raise ValueError(what)


# The calls below are made once per layer and decode step: each tensor is looked at once (type, device, layout, then
# pointer), in as few Python calls as that takes.
_int32 = _f32 = None
_bits16 = ()         # bf16, and its bits as 16-bit integers


def _call_on(t, name: str, stream):
    """(device index, stream handle) of a call: the current device, which t has to be on (and the other tensors where t
    is), and its current stream where none is given."""
    global _int32, _f32, _bits16
    if not _bits16:
        import torch
        _int32, _f32, _bits16 = torch.int32, torch.float32, (torch.bfloat16, torch.int16, torch.uint16)
    dev = t.get_device()
    if dev < 0:
        _refuse(f"{name}: a tensor on the current CUDA device")
    device, current = _raw_stream or _raw()
    if dev != device():
        _refuse(f"{name}: a tensor on the current CUDA device")
    return dev, current(dev) if stream is None else int(stream.cuda_stream)


def _i32(t, n: int, name: str, dev: int) -> int:
    """Device pointer of a contiguous int32 tensor of at least n elements."""
    if t.dtype is not _int32 or t.get_device() != dev or not t.is_contiguous() or t.numel() < n:
        _refuse(f"{name}: a contiguous int32 tensor of {n} elements or more on cuda:{dev}")
    return t.data_ptr()


def _b16(t, n: int, name: str, dev: int) -> int:
    """Device pointer of a contiguous bf16 tensor of n elements."""
    if t.dtype not in _bits16 or t.get_device() != dev or not t.is_contiguous() or t.numel() != n:
        _refuse(f"{name}: a contiguous bf16 tensor of {n} elements on cuda:{dev}")
    return t.data_ptr()


def kv4_block_tables(cached, new_tokens, free_pages, n_free, page_size: int, table, q_start, kv_len, slots, positions,
                     n_free_out, stream=None):
    """Block tables and slot maps of a batch from its requests' lengths (all int32 device tensors): takes the
    new pages from the stack free_pages[:n_free] (an n_free past free_pages is an error on the device), writes their entries of table [B, max_blocks], and gives
    q_start [B + 1], kv_len [B], and the slot and position of each new token."""
    B, n = new_tokens.numel(), slots.numel()
    rows, width = table.shape
    if rows != B:
        _refuse("table: [B, max_blocks]")
    dev, handle = _call_on(new_tokens, "new_tokens", stream)
    st = _lib.kv4_block_tables_bounded(_i32(cached, B, "cached", dev), _i32(new_tokens, B, "new_tokens", dev), B,
                                       _i32(free_pages, 0, "free_pages", dev), free_pages.numel(),
                                       _i32(n_free, 1, "n_free", dev), page_size, _i32(table, 0, "table", dev), width,
                                       _i32(q_start, B + 1, "q_start", dev), _i32(kv_len, B, "kv_len", dev),
                                       _i32(slots, n, "slots", dev), _i32(positions, n, "positions", dev), n,
                                       _i32(n_free_out, 1, "n_free_out", dev), handle)
    if st:
        _check(st, "kv4_block_tables")


def qk_norm_rope(qkv, n_q_heads: int, n_kv_heads: int, head_dim: int, q_weight, k_weight, eps: float, cos_sin, positions,
                 q_out, k_out=None, interleaved: bool = False, cache: Kv4Cache | None = None, slots=None, stream=None):
    """Per-head RMS norms of queries and keys (weights None: no norm) and their rotation (cos_sin None: none) from
    the rows of qkv [T, >= heads * head_dim] (bf16) into q_out [T, n_q_heads, head_dim] and k_out; with a cache,
    keys and values are also written to it at slots."""
    T, width = qkv.shape
    row, one = qkv.stride()
    dev, handle = _call_on(qkv, "qkv", stream)
    if one != 1 or qkv.dtype not in _bits16 or width < (n_q_heads + n_kv_heads * (1 if cache is None else 2)) * head_dim:
        _refuse("qkv: bf16 [T, heads * head_dim], rows contiguous")
    n_pos = rot = cs = pos = None
    if cos_sin is not None:
        n_pos, rot = cos_sin.shape
        if cos_sin.dtype is not _f32 or cos_sin.get_device() != dev or not cos_sin.is_contiguous():
            _refuse(f"cos_sin: a contiguous float32 tensor [n_pos, rot_dim] on cuda:{dev}")
        cs, pos = cos_sin.data_ptr(), _i32(positions, T, "positions", dev)
    if cache is not None and cache.device != dev:
        _refuse(f"cache: on cuda:{dev}")
    st = _lib.qk_norm_rope(qkv.data_ptr(), row, T, n_q_heads, n_kv_heads, head_dim,
                           None if q_weight is None else _b16(q_weight, head_dim, "q_weight", dev),
                           None if k_weight is None else _b16(k_weight, head_dim, "k_weight", dev), eps, cs, rot or 0,
                           interleaved, n_pos or 0, pos,
                           _b16(q_out, T * n_q_heads * head_dim, "q_out", dev) if n_q_heads else None,
                           None if k_out is None else _b16(k_out, T * n_kv_heads * head_dim, "k_out", dev),
                           None if cache is None else cache.ref, None if slots is None else _i32(slots, T, "slots", dev),
                           handle)
    if st:
        _check(st, "qk_norm_rope")
    return q_out, k_out


def _heads(x, T: int, cache: Kv4Cache) -> int:
    """Token stride of x [T, n_kv_heads, head_dim] (bf16, a token's heads contiguous)."""
    s0, s1, s2 = x.stride()
    if x.shape != (T, cache.n_kv_heads, cache.head_dim) or x.dtype not in _bits16 or x.get_device() != cache.device or s2 != 1 or (s1 != cache.head_dim and cache.n_kv_heads > 1):
        _refuse("k, v: bf16 [T, n_kv_heads, head_dim] where the cache is, a token's heads contiguous")
    return s0


def kv4_append(cache: Kv4Cache, k, v, slots, stream=None):
    """Quantise keys and values [T, n_kv_heads, head_dim] (bf16; any token stride) into the cache at slots."""
    T = k.shape[0]
    dev, handle = _call_on(cache.pages, "cache", stream)
    st = _lib.kv4_append(cache.ref, k.data_ptr(), _heads(k, T, cache), v.data_ptr(), _heads(v, T, cache), T,
                         _i32(slots, T, "slots", dev), handle)
    if st:
        _check(st, "kv4_append")


def kv4_gather(cache: Kv4Cache, slots, k_out, v_out, stream=None):
    """The keys and values that the cache holds at slots, as bf16 [n, n_kv_heads, head_dim]."""
    n = slots.numel()
    size = n * cache.n_kv_heads * cache.head_dim
    dev, handle = _call_on(cache.pages, "cache", stream)
    st = _lib.kv4_gather(cache.ref, _i32(slots, n, "slots", dev), n, _b16(k_out, size, "k_out", dev),
                         _b16(v_out, size, "v_out", dev), handle)
    if st:
        _check(st, "kv4_gather")
    return k_out, v_out


def kv4_attention_ws_size(B: int, n_q_heads: int, n_kv_heads: int, head_dim: int, n_q_tokens: int, max_q: int,
                          max_kv: int) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.kv4_attention_ws_size(B, n_q_heads, n_kv_heads, head_dim, n_q_tokens, max_q, max_kv, ctypes.byref(n)),
           "kv4_attention_ws_size")
    return n.value


def kv4_attention(cache: Kv4Cache, q, q_start, kv_len, table, out, workspace, max_q: int, max_kv: int, scale: float,
                  causal: bool = True, window: int = 0, stream=None):
    """Softmax attention of a ragged batch over the cache: q, out [n_q_tokens, n_q_heads, head_dim] (bf16), request b's
    queries being rows q_start[b] .. q_start[b + 1] - 1 and the last tokens of its kv_len[b]."""
    n, hq, D = q.shape
    rows, width = table.shape
    B = kv_len.numel()
    if D != cache.head_dim or rows != B:
        _refuse("q: [n, n_q_heads, head_dim] of the cache's head_dim; table: [B, max_blocks]")
    dev, handle = _call_on(cache.pages, "cache", stream)
    if workspace.get_device() != dev or not workspace.is_contiguous():
        _refuse(f"workspace: a contiguous tensor on cuda:{dev}")
    st = _lib.kv4_attention(cache.ref, _b16(q, n * hq * D, "q", dev), n, hq, _i32(q_start, B + 1, "q_start", dev),
                            _i32(kv_len, B, "kv_len", dev), B, _i32(table, 0, "table", dev), width, max_q, max_kv, scale,
                            causal, window, _b16(out, n * hq * D, "out", dev), workspace.data_ptr(), workspace.nbytes,
                            handle)
    if st:
        _check(st, "kv4_attention")
    return out


# ================================================================ around attention and experts
def _rows(t, T: int, n: int, types, name: str, dev: int) -> int:
    """Row stride of t [T, n] (values of a row contiguous)."""
    if t.dtype in types and t.get_device() == dev:
        if t.is_contiguous() and t.numel() == T * n:
            return n
        if t.shape == (T, n):
            s0, s1 = t.stride()
            if s1 == 1 or n == 1:
                return s0
    _refuse(f"{name}: [{T}, {n}] of {' or '.join(str(x) for x in types)} on cuda:{dev}, the values of a row contiguous")


_bits8 = ()          # e4m3, and its bits as 8-bit integers


def add_rms_norm(x, weight, eps: float, y=None, residual=None, residual_out=None, codes=None, scales=None, stream=None):
    """y = norm(x + residual) * weight for rows of x [T, n] (bf16 or float32; any row stride); residual_out (bf16; None:
    residual itself) gets x + residual.  codes [T, n] (float8_e4m3fn or uint8) get y / scale with scales [T, 1] (a scale a
    row) or [T, ceil(n / 128)] (one for each 128 values)."""
    global _bits8
    T, n = x.shape
    dev, handle = _call_on(x, "x", stream)
    f32 = x.dtype is _f32
    xs = _rows(x, T, n, _bits16 if not f32 else (_f32,), "x", dev)
    rs = ros = ys = 0
    rp = rop = yp = cp = sp = None
    group = 0
    if residual is not None:
        rs, rp = _rows(residual, T, n, _bits16, "residual", dev), residual.data_ptr()
        if residual_out is None:
            ros, rop = rs, rp
        else:
            ros, rop = _rows(residual_out, T, n, _bits16, "residual_out", dev), residual_out.data_ptr()
    elif residual_out is not None:
        _refuse("residual_out: needs a residual")
    if y is not None:
        ys, yp = _rows(y, T, n, _bits16, "y", dev), y.data_ptr()
    if codes is not None:
        if not _bits8:
            import torch
            _bits8 = (torch.float8_e4m3fn, torch.uint8)
        if codes.dtype not in _bits8 or codes.shape != (T, n) or codes.get_device() != dev or not codes.is_contiguous():
            _refuse(f"codes: a contiguous float8_e4m3fn tensor [{T}, {n}] on cuda:{dev}")
        groups = (n + 127) >> 7
        if (scales is None or scales.dtype is not _f32 or scales.get_device() != dev or not scales.is_contiguous()
                or scales.dim() != 2 or scales.shape[0] != T or scales.shape[1] not in (1, groups)):
            _refuse(f"scales: a contiguous float32 tensor [{T}, 1] or [{T}, {groups}] on cuda:{dev}")
        group = 0 if scales.shape[1] == 1 else 128
        cp, sp = codes.data_ptr(), scales.data_ptr()
    elif scales is not None:
        _refuse("scales: need codes")
    st = _lib.add_rms_norm(x.data_ptr(), f32, xs, rp, rs, rop, ros, None if weight is None else _b16(weight, n, "weight", dev), T, n,
                           eps, yp, ys, cp, sp, group, handle)
    if st:
        _check(st, "add_rms_norm")
    return y


def qmoe_route_scored(logits, k: int, ids, gates, sigmoid: bool = False, bias=None, n_groups: int = 1, top_groups: int = 1,
                      group_best: int = 1, renormalise: bool = False, scale: float = 1.0, stream=None):
    """Experts ids [T, k] (int32) and gates [T, k] (float32) from logits [T, E] (float32 or bf16; any row stride): softmax or
    sigmoid scores, chosen by score + bias (float32 [E]) among the top_groups best of n_groups groups."""
    T, E = logits.shape
    dev, handle = _call_on(logits, "logits", stream)
    f32 = logits.dtype is _f32
    stride = _rows(logits, T, E, _bits16 if not f32 else (_f32,), "logits", dev)
    bp = None
    if bias is not None:
        if bias.dtype is not _f32 or bias.get_device() != dev or not bias.is_contiguous() or bias.numel() != E:
            _refuse(f"bias: a contiguous float32 tensor of {E} elements on cuda:{dev}")
        bp = bias.data_ptr()
    if gates.dtype is not _f32 or gates.get_device() != dev or not gates.is_contiguous() or gates.numel() != T * k:
        _refuse(f"gates: a contiguous float32 tensor [{T}, {k}] on cuda:{dev}")
    if ids.numel() != T * k:
        _refuse(f"ids: a contiguous int32 tensor [{T}, {k}] on cuda:{dev}")
    st = _lib.qmoe_route_scored(logits.data_ptr(), f32, stride, T, E, k, sigmoid, bp, n_groups, top_groups, group_best, renormalise,
                                scale, _i32(ids, T * k, "ids", dev), gates.data_ptr(), handle)
    if st:
        _check(st, "qmoe_route_scored")
    return ids, gates


# ================================================================ attention over chosen blocks
class Kv4Bounds:
    """Bounds of each block's keys beside a Kv4Cache: codes int8 [n_pages, n_kv_heads, 2, head_dim] and steps float32
    [n_pages, n_kv_heads] (``kv4_bounds`` in qmoe.h)."""

    def __init__(self, codes, steps, page_size: int):
        import torch
        if codes.dtype != torch.int8 or codes.dim() != 4 or codes.shape[2] != 2 or not codes.is_contiguous():
            raise ValueError("codes must be a contiguous int8 tensor [n_pages, n_kv_heads, 2, head_dim]")
        if steps.dtype != torch.float32 or steps.shape != codes.shape[:2] or not steps.is_contiguous():
            raise ValueError("steps must be a contiguous float32 tensor [n_pages, n_kv_heads]")
        if not codes.is_cuda or steps.get_device() != codes.get_device():
            raise ValueError("codes and steps must be on one CUDA device")
        self.codes, self.steps, self.page_size = codes, steps, page_size
        self.n_pages, self.n_kv_heads, _, self.head_dim = codes.shape
        self.device = codes.get_device()
        self.c = CKv4Bounds(_dptr(codes), _dptr(steps), self.n_pages, page_size, self.n_kv_heads, self.head_dim)
        self.ref = ctypes.byref(self.c)

    @classmethod
    def empty(cls, cache: Kv4Cache) -> "Kv4Bounds":
        import torch
        where = cache.pages.device
        return cls(torch.zeros((cache.n_pages, cache.n_kv_heads, 2, cache.head_dim), dtype=torch.int8, device=where),
                   torch.zeros((cache.n_pages, cache.n_kv_heads), dtype=torch.float32, device=where), cache.page_size)


def kv4_block_bounds(cache: Kv4Cache, bounds: Kv4Bounds, slots, stream=None):
    """Bring the bounds of the blocks that tokens were written to at slots (int32) up to date."""
    dev, handle = _call_on(cache.pages, "cache", stream)
    if bounds.device != dev:
        _refuse(f"bounds: on cuda:{dev}")
    n = slots.numel()
    st = _lib.kv4_block_bounds(cache.ref, bounds.ref, _i32(slots, n, "slots", dev), n, handle)
    if st:
        _check(st, "kv4_block_bounds")


def kv4_select_blocks_ws_size(n_q_tokens: int, n_kv_heads: int, page_size: int, max_kv: int) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.kv4_select_blocks_ws_size(n_q_tokens, n_kv_heads, page_size, max_kv, ctypes.byref(n)), "kv4_select_blocks_ws_size")
    return n.value


def kv4_select_blocks(bounds: Kv4Bounds, q, q_start, kv_len, table, sel, workspace, max_kv: int, first: int = 1, last: int = 1,
                      stream=None):
    """Fill sel [n_q_tokens, n_kv_heads, top] (int32) with the blocks that each query of q [n_q_tokens, n_q_heads, head_dim]
    (bf16) attends to: the first and last ones and those whose bounds give the largest scores, ascending, then -1."""
    n, hq, D = q.shape
    rows, width = table.shape
    B = kv_len.numel()
    n_sel, heads, top = sel.shape
    if D != bounds.head_dim or rows != B or n_sel != n or heads != bounds.n_kv_heads:
        _refuse("q: [n, n_q_heads, head_dim] of the bounds' head_dim; table: [B, max_blocks]; sel: [n, n_kv_heads, top]")
    dev, handle = _call_on(bounds.codes, "bounds", stream)
    if workspace.get_device() != dev or not workspace.is_contiguous():
        _refuse(f"workspace: a contiguous tensor on cuda:{dev}")
    st = _lib.kv4_select_blocks(bounds.ref, _b16(q, n * hq * D, "q", dev), n, hq, _i32(q_start, B + 1, "q_start", dev),
                                _i32(kv_len, B, "kv_len", dev), B, _i32(table, 0, "table", dev), width, max_kv, top, first, last,
                                _i32(sel, 0, "sel", dev), workspace.data_ptr(), workspace.nbytes, handle)
    if st:
        _check(st, "kv4_select_blocks")
    return sel


def kv4_attention_blocks_ws_size(n_q_tokens: int, n_q_heads: int, n_kv_heads: int, head_dim: int, page_size: int, top: int) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.kv4_attention_blocks_ws_size(n_q_tokens, n_q_heads, n_kv_heads, head_dim, page_size, top, ctypes.byref(n)),
           "kv4_attention_blocks_ws_size")
    return n.value


def kv4_attention_blocks(cache: Kv4Cache, q, q_start, kv_len, table, sel, out, workspace, scale: float, stream=None):
    """kv4_attention (causal) where each query token and kv head sees the blocks of its list sel [n_q_tokens, n_kv_heads,
    top] only."""
    n, hq, D = q.shape
    rows, width = table.shape
    B = kv_len.numel()
    n_sel, heads, top = sel.shape
    if D != cache.head_dim or rows != B or n_sel != n or heads != cache.n_kv_heads:
        _refuse("q: [n, n_q_heads, head_dim] of the cache's head_dim; table: [B, max_blocks]; sel: [n, n_kv_heads, top]")
    dev, handle = _call_on(cache.pages, "cache", stream)
    if workspace.get_device() != dev or not workspace.is_contiguous():
        _refuse(f"workspace: a contiguous tensor on cuda:{dev}")
    st = _lib.kv4_attention_blocks(cache.ref, _b16(q, n * hq * D, "q", dev), n, hq, _i32(q_start, B + 1, "q_start", dev),
                                   _i32(kv_len, B, "kv_len", dev), B, _i32(table, 0, "table", dev), width, _i32(sel, 0, "sel", dev), top,
                                   scale, _b16(out, n * hq * D, "out", dev), workspace.data_ptr(), workspace.nbytes, handle)
    if st:
        _check(st, "kv4_attention_blocks")
    return out
