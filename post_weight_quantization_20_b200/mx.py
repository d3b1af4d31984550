"""Microscaled 4-bit rows: the Python binding of ``include/gptq_mx.h``.

The functions named ``gptq_mx_*`` mirror the C calls (argument marshalling and checks
only); ``mx_quantize``, ``mx_dequantize``, ``mx_matmul`` and ``mx_linear`` allocate their
results.  A matrix's stored form is a pair of tensors:

* ``codes``  int32 (rows, mx_words(cols)): eight 4-bit codes per word;
* ``scales`` uint8 mx_scale_shape(rows, cols): one byte per 32 columns, in 128 x 4 tiles.

As in ``gptq``, there is no CPU fallback, work runs on `stream` (default: the current
stream of the tensors' device) and nothing is synchronised.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import gptq as G

# every symbol include/gptq_mx.h declares
EXPORTS = ("gptq_mx_scale_bytes", "gptq_mx_quantize", "gptq_mx_dequantize", "gptq_mx_matmul",
           "gptq_mx_debug_give_up")

_lib = None


def load_library() -> ctypes.CDLL:
    """libgptq.so with the signatures of include/gptq_mx.h declared."""
    global _lib
    if _lib is None:
        lib = G.load_library()
        vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        lib.gptq_mx_scale_bytes.argtypes = [i64, i64]
        lib.gptq_mx_scale_bytes.restype = ctypes.c_size_t
        lib.gptq_mx_quantize.argtypes = [vp, i32, i64, i64, i64, vp, vp, vp, vp]
        lib.gptq_mx_quantize.restype = i32
        lib.gptq_mx_dequantize.argtypes = [vp, vp, i64, i64, vp, i32, i64, vp]
        lib.gptq_mx_dequantize.restype = i32
        lib.gptq_mx_matmul.argtypes = [vp, vp, i64, vp, vp, i64, i64, vp, i32, i64, vp, vp]
        lib.gptq_mx_matmul.restype = i32
        lib.gptq_mx_debug_give_up.argtypes = [ctypes.c_int32]
        lib.gptq_mx_debug_give_up.restype = ctypes.c_int32
        _lib = lib
    return _lib


def mx_words(cols: int) -> int:
    """32-bit words of a row's codes."""
    return (cols + 31) // 32 * 4


def mx_scale_shape(rows: int, cols: int) -> tuple:
    return ((rows + 127) // 128, (cols + 127) // 128, 32, 16)


def gptq_mx_scale_bytes(rows: int, cols: int) -> int:
    return int(load_library().gptq_mx_scale_bytes(rows, cols))


_WORDS = (torch.int32, torch.uint32)


def _call(f, name, dev, stream, *args):
    """Call the library's `f` on `stream` (default: the current one) of device `dev`, which is
    made the current one: a launch and its stream belong to it."""
    if dev == torch._C._cuda_getDevice():
        code = f(*args, torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)
    else:
        with torch.cuda.device(dev):
            code = f(*args, torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)
    if code:
        G._check(code, name)


def _expect_stored(codes, scales, rows, cols, name=""):
    """Raise unless codes and scales are the stored form of a rows x cols matrix."""
    words, shape = (rows, (cols + 31) // 32 * 4), mx_scale_shape(rows, cols)
    if not (codes.shape == words and scales.shape == shape and codes.dtype in _WORDS
            and scales.dtype is torch.uint8 and codes.is_contiguous() and scales.is_contiguous()):
        G._expect(codes, name + "codes", words, _WORDS)
        G._expect(scales, name + "scales", shape, (torch.uint8,))


def _expect_matrix(t, name):
    """Rows and columns of a matrix, its type and the distance of its rows."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D with unit column stride")
    (R, C), (ld, one) = t.shape, t.stride()
    if one != 1 and C > 1:
        raise ValueError(f"{name} must be 2-D with unit column stride")
    dt = G._DT.get(t.dtype)
    if dt is None:
        raise ValueError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}")
    if R <= 1:
        ld = C
    elif ld < C:
        raise ValueError(f"the rows of {name} must not overlap")
    return R, C, dt, ld


def _status_ptr(status):
    if status is None:
        return None
    G._expect_status(status)
    return status.data_ptr()


def gptq_mx_quantize(X, codes, scales, status=None, stream=None) -> None:
    """The stored form of X (rows x cols, unit column stride) into codes and scales."""
    R, C, dt, ld = _expect_matrix(X, "X")
    _expect_stored(codes, scales, R, C)
    st = _status_ptr(status)
    dev = X.get_device()
    if dev < 0 or codes.get_device() != dev or scales.get_device() != dev or st is not None:
        G._need_cuda(X, codes, scales, status)
    _call(load_library().gptq_mx_quantize, "gptq_mx_quantize", dev, stream, X.data_ptr(), dt, R, C,
          ld, codes.data_ptr(), scales.data_ptr(), st)


def gptq_mx_dequantize(codes, scales, Y, stream=None) -> None:
    """Y (rows x cols) = the values the stored form stands for."""
    R, C, dt, ld = _expect_matrix(Y, "Y")
    _expect_stored(codes, scales, R, C)
    dev = Y.get_device()
    if dev < 0 or codes.get_device() != dev or scales.get_device() != dev:
        G._need_cuda(codes, scales, Y)
    _call(load_library().gptq_mx_dequantize, "gptq_mx_dequantize", dev, stream, codes.data_ptr(),
          scales.data_ptr(), R, C, Y.data_ptr(), dt, ld)


def gptq_mx_matmul(x_codes, x_scales, w_codes, w_scales, cols, Y, status=None,
                   stream=None) -> None:
    """Y (tokens x rows) = X W^T of two stored forms with `cols` columns each."""
    M, R, dt, ld = _expect_matrix(Y, "Y")
    cols = int(cols)
    _expect_stored(x_codes, x_scales, M, cols, "x_")
    _expect_stored(w_codes, w_scales, R, cols, "w_")
    st = _status_ptr(status)
    dev = Y.get_device()
    if dev < 0 or st is not None or not (dev == x_codes.get_device() == x_scales.get_device()
                                         == w_codes.get_device() == w_scales.get_device()):
        G._need_cuda(x_codes, x_scales, w_codes, w_scales, Y, status)
    _call(load_library().gptq_mx_matmul, "gptq_mx_matmul", dev, stream, x_codes.data_ptr(),
          x_scales.data_ptr(), M, w_codes.data_ptr(), w_scales.data_ptr(), R, cols, Y.data_ptr(),
          dt, ld, st)


def gptq_mx_debug_give_up(stages: int) -> int:
    """Stage of a tile at which the products' last MMA issuer gives up (-1: none); returns the
    previous one.  For tests of the timeout path."""
    return int(load_library().gptq_mx_debug_give_up(int(stages)))


# --------------------------------------------------------------------------- whole matrices
@dataclass
class MXMatrix:
    """A rows x cols matrix in its stored form."""
    codes: torch.Tensor
    scales: torch.Tensor
    rows: int
    cols: int

    @property
    def nbytes(self) -> int:
        return self.codes.numel() * 4 + self.scales.numel()


def mx_quantize(X: torch.Tensor, status=None, stream=None) -> MXMatrix:
    """The stored form of X (rows x cols)."""
    _expect_matrix(X, "X")
    R, C = X.shape
    with G._on(stream):
        q = MXMatrix(torch.empty(R, mx_words(C), dtype=torch.int32, device=X.device),
                     torch.empty(mx_scale_shape(R, C), dtype=torch.uint8, device=X.device), R, C)
        gptq_mx_quantize(X, q.codes, q.scales, status, stream)
    return q


def mx_dequantize(q: MXMatrix, dtype=torch.float32, stream=None) -> torch.Tensor:
    with G._on(stream):
        Y = torch.empty(q.rows, q.cols, dtype=dtype, device=q.codes.device)
        gptq_mx_dequantize(q.codes, q.scales, Y, stream)
    return Y


def mx_matmul(x: MXMatrix, w: MXMatrix, dtype=torch.float32, status=None,
              stream=None) -> torch.Tensor:
    """x W^T (x.rows x w.rows)."""
    if x.cols != w.cols:
        raise ValueError(f"both matrices need the same cols, got {x.cols} and {w.cols}")
    with G._on(stream):
        Y = torch.empty(x.rows, w.rows, dtype=dtype, device=w.codes.device)
        gptq_mx_matmul(x.codes, x.scales, w.codes, w.scales, w.cols, Y, status, stream)
    return Y


def mx_linear(X: torch.Tensor, w: MXMatrix, dtype=None, status=None, stream=None) -> torch.Tensor:
    """X W^T with the activations X (tokens x cols) quantised to the same 4-bit blocks first."""
    return mx_matmul(mx_quantize(X, status, stream), w, dtype or X.dtype, status, stream)
