"""The paged low-bit key/value cache: the Python binding of ``include/gptq_cache.h``.

``gptq_cache_write`` and ``gptq_cache_read`` mirror the C calls (argument marshalling and
checks only); ``KVCache`` holds a cache's arrays and forwards to them.  The sizes come
from the tensors: K and V are (rows, heads, dim) with any strides and unit stride along
dim; ``codes`` int32 (pages, page_size, heads, words); ``grids`` float32 (pages, page_size,
heads, groups, 2) holding (scale, zero), or uint8 (pages, page_size, heads, blocks) for
microscaled blocks; ``table`` int32 (seqs, width), ``cu`` int32 (seqs + 1) and ``start``
int32 (seqs) say which position of which sequence each row is.

There is no CPU fallback, work runs on `stream` (default: the current stream of the
tensors' device) and nothing is synchronised; out-of-range positions and pages and
non-finite groups are reported in `status`, as the header says.
"""
from __future__ import annotations

import ctypes
import struct
from dataclasses import dataclass

import torch

from . import gptq as G
from .mx import _WORDS, _call, _status_ptr, mx_words

GPTQ_CACHE_GRID, GPTQ_CACHE_MX = 0, 1

# every symbol include/gptq_cache.h declares
EXPORTS = ("gptq_cache_words", "gptq_cache_grid_bytes", "gptq_cache_write", "gptq_cache_read")


class gptq_cache_config(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("bits", ctypes.c_int), ("group_size", ctypes.c_int),
                ("sym", ctypes.c_int)]


# struct gptq_cache and struct gptq_cache_rows of the header, packed per call (a ctypes.Structure
# costs the host three times as much to make)
_CACHE = struct.Struct("@4P4q")
_ROWS = struct.Struct("@PqqPPq")

_lib = None


def load_library() -> ctypes.CDLL:
    """libgptq.so with the signatures of include/gptq_cache.h declared."""
    global _lib
    if _lib is None:
        lib = G.load_library()
        vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        cfg, cache, rows = ctypes.POINTER(gptq_cache_config), ctypes.c_char_p, ctypes.c_char_p
        for name in ("gptq_cache_words", "gptq_cache_grid_bytes"):
            getattr(lib, name).argtypes = [cfg, i64]
            getattr(lib, name).restype = ctypes.c_size_t
        lib.gptq_cache_write.argtypes = [vp, vp, i32, i64, i64, i64, i64, i64, cfg, cache, rows, vp, vp]
        lib.gptq_cache_write.restype = i32
        lib.gptq_cache_read.argtypes = [cfg, cache, rows, vp, vp, i32, i64, i64, i64, i64, i64, vp, vp]
        lib.gptq_cache_read.restype = i32
        _lib = lib
    return _lib


_KINDS = {"grid": GPTQ_CACHE_GRID, "mx": GPTQ_CACHE_MX}


def make_cache_config(kind="grid", bits=4, group_size=0, sym=False) -> gptq_cache_config:
    """kind "grid" (min-max integer grids, 4 or 8 bits) or "mx" (microscaled 4-bit blocks)."""
    if kind not in _KINDS:
        raise ValueError(f'kind must be "grid" or "mx", got {kind!r}')
    return gptq_cache_config(_KINDS[kind], int(bits), int(group_size), int(bool(sym)))


def gptq_cache_words(cfg: gptq_cache_config, dim: int) -> int:
    return int(load_library().gptq_cache_words(ctypes.byref(cfg), dim))


def gptq_cache_grid_bytes(cfg: gptq_cache_config, dim: int) -> int:
    return int(load_library().gptq_cache_grid_bytes(ctypes.byref(cfg), dim))


def _grid_shape(cfg, pages, page_size, heads, dim):
    if cfg.kind == GPTQ_CACHE_MX:
        return (pages, page_size, heads, (dim + 31) // 32), torch.uint8
    return (pages, page_size, heads, G.n_groups(dim, cfg.group_size), 2), torch.float32


def _words(cfg, dim):
    return mx_words(dim) if cfg.kind == GPTQ_CACHE_MX else G.packed_words(dim, cfg.bits)


def _expect_rows_of(t, name):
    if t.dim() != 3 or (t.stride(2) != 1 and t.shape[2] > 1):
        raise ValueError(f"{name} must be 3-D (rows, heads, dim) with unit stride along dim")
    if t.dtype not in G._DT:
        raise ValueError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}")


def _no_overlap(t, name):
    """Written tensors: no two (row, head) pairs may share memory."""
    if t.is_contiguous():
        return
    n, h, d = t.shape
    (a, sa), (b, sb) = sorted(((n, t.stride(0)), (h, t.stride(1))), key=lambda x: x[1])
    if (a > 1 and sa < d) or (b > 1 and sb < (sa * (a - 1) + d if a > 1 else d)):
        raise ValueError(f"the rows of {name} must not overlap")


def _explain(K, V, cfg, k_codes, k_grids, v_codes, v_grids, table, cu, start, written):
    """Raise for the first tensor of a call that does not fit."""
    _expect_rows_of(K, "K")
    _expect_rows_of(V, "V")
    if V.shape != K.shape or V.dtype != K.dtype:
        raise ValueError("V must have the shape and dtype of K")
    if written:
        _no_overlap(K, "K")
        _no_overlap(V, "V")
    if k_codes.dim() != 4:
        raise ValueError("k_codes must be 4-D (pages, page_size, heads, words)")
    pages, page_size = k_codes.shape[:2]
    _, H, D = K.shape
    shape = (pages, page_size, H, _words(cfg, D))
    G._expect(k_codes, "k_codes", shape, _WORDS)
    G._expect(v_codes, "v_codes", shape, _WORDS)
    shape, dtype = _grid_shape(cfg, pages, page_size, H, D)
    G._expect(k_grids, "k_grids", shape, (dtype,))
    G._expect(v_grids, "v_grids", shape, (dtype,))
    if table.dim() != 2 or table.dtype != torch.int32 or (table.shape[1] > 1 and table.stride(1) != 1):
        raise ValueError("table must be an int32 (seqs, width) tensor with unit column stride")
    S, width = table.shape
    if S > 1 and table.stride(0) < width:
        raise ValueError("the rows of table must not overlap")
    G._expect(cu, "cu", (S + 1,), (torch.int32,))
    G._expect(start, "start", (S,), (torch.int32,))


_I32 = torch.int32


def _marshal(K, V, cfg, k_codes, k_grids, v_codes, v_grids, table, cu, start, status,
             written=False):
    """Check a call's tensors; the arguments of the C call that both directions share.  One
    expression passes what fits; _explain says what does not."""
    fits = False
    if K.dim() == 3 and k_codes.dim() == 4 and table.dim() == 2 and V.shape == K.shape:
        T, H, D = K.shape
        (kt, kh, k1), (vt, vh, v1) = K.stride(), V.stride()
        pages, page_size, _, _ = k_codes.shape
        (S, width), (ld, one) = table.shape, table.stride()
        codes = (pages, page_size, H, _words(cfg, D))
        grids, gtype = _grid_shape(cfg, pages, page_size, H, D)
        if S <= 1:
            ld = width
        fits = (k_codes.shape == codes and v_codes.shape == codes and k_grids.shape == grids
                and v_grids.shape == grids and k_codes.dtype in _WORDS and v_codes.dtype in _WORDS
                and k_grids.dtype is gtype and v_grids.dtype is gtype and k_codes.is_contiguous()
                and v_codes.is_contiguous() and k_grids.is_contiguous() and v_grids.is_contiguous()
                and (k1 == v1 == 1 or D == 1) and V.dtype is K.dtype and K.dtype in G._DT
                and table.dtype is _I32 and (one == 1 or width <= 1) and ld >= width
                and cu.shape == (S + 1,) and start.shape == (S,) and cu.dtype is _I32
                and start.dtype is _I32 and cu.is_contiguous() and start.is_contiguous()
                and not (written and not (K.is_contiguous() and V.is_contiguous())))
    if not fits:
        _explain(K, V, cfg, k_codes, k_grids, v_codes, v_grids, table, cu, start, written)
    st = _status_ptr(status)
    dev = K.get_device()
    if dev < 0 or st is not None or not (
            dev == V.get_device() == k_codes.get_device() == k_grids.get_device()
            == v_codes.get_device() == v_grids.get_device() == table.get_device()
            == cu.get_device() == start.get_device()):
        G._need_cuda(K, V, k_codes, k_grids, v_codes, v_grids, table, cu, start, status)
    where = (ctypes.byref(cfg),
             _CACHE.pack(k_codes.data_ptr(), k_grids.data_ptr(), v_codes.data_ptr(),
                         v_grids.data_ptr(), pages, page_size, H, D),
             _ROWS.pack(table.data_ptr(), ld, width, cu.data_ptr(), start.data_ptr(), S))
    data = (K.data_ptr(), V.data_ptr(), G._DT[K.dtype], T, kt, kh, vt, vh)
    return dev, where, data, st


def gptq_cache_write(K, V, cfg, k_codes, k_grids, v_codes, v_grids, table, cu, start, status=None,
                     stream=None) -> None:
    """Quantise the rows of K and V (rows, heads, dim) into their slots of the cache."""
    dev, where, data, st = _marshal(K, V, cfg, k_codes, k_grids, v_codes, v_grids, table, cu,
                                    start, status)
    _call(load_library().gptq_cache_write, "gptq_cache_write", dev, stream, *data, *where, st)


def gptq_cache_read(cfg, k_codes, k_grids, v_codes, v_grids, table, cu, start, K, V, status=None,
                    stream=None) -> None:
    """The rows' values out of their slots of the cache into K and V (rows, heads, dim)."""
    dev, where, data, st = _marshal(K, V, cfg, k_codes, k_grids, v_codes, v_grids, table, cu,
                                    start, status, written=True)
    _call(load_library().gptq_cache_read, "gptq_cache_read", dev, stream, *where, *data, st)


# --------------------------------------------------------------------------- one cache
@dataclass
class KVCache:
    """The arrays of one layer's cache: `pages` pages of `page_size` tokens."""
    cfg: gptq_cache_config
    k_codes: torch.Tensor
    k_grids: torch.Tensor
    v_codes: torch.Tensor
    v_grids: torch.Tensor
    heads: int
    dim: int

    @classmethod
    def alloc(cls, cfg, pages, page_size, heads, dim, device="cuda") -> "KVCache":
        """A zeroed cache (a slot that was never written reads back as zeros)."""
        if gptq_cache_words(cfg, dim) == 0:
            raise G.GPTQError(G.GPTQ_ERR_UNSUPPORTED, "KVCache.alloc")
        shape, dtype = _grid_shape(cfg, pages, page_size, heads, dim)
        codes = (pages, page_size, heads, _words(cfg, dim))
        t = [torch.zeros(s, dtype=d, device=device) for _ in range(2)
             for s, d in ((codes, torch.int32), (shape, dtype))]
        return cls(cfg, *t, heads, dim)

    @property
    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in
                   (self.k_codes, self.k_grids, self.v_codes, self.v_grids))

    def write(self, K, V, table, cu, start, status=None, stream=None) -> None:
        gptq_cache_write(K, V, self.cfg, self.k_codes, self.k_grids, self.v_codes, self.v_grids,
                         table, cu, start, status, stream)

    def read(self, table, cu, start, rows: int, dtype=torch.float16, status=None, stream=None):
        """(K, V) of `rows` rows, each (rows, heads, dim)."""
        with G._on(stream):
            K, V = (torch.zeros(rows, self.heads, self.dim, dtype=dtype,
                                device=self.k_codes.device) for _ in range(2))
            gptq_cache_read(self.cfg, self.k_codes, self.k_grids, self.v_codes, self.v_grids,
                            table, cu, start, K, V, status, stream)
        return K, V
