"""Microscaled 4-bit matrices: rows quantised and read back, and the product of
two such matrices on the 4-bit tensor cores.

Argument marshalling over the C ABI declared in include/ft_fp4.h, which says
what each call computes; errors raise FtError.  Dense tensors may be strided
views (columns contiguous); calls enqueue on the current stream (or `stream`).

    w = Fp4Matrix(FT_FP4_NVFP4, N, K)      # a projection's weights, quantised once
    fp4_quantize(weight, w)
    xq = Fp4Matrix(FT_FP4_NVFP4, T, K)
    # every step:
    fp4_quantize(x, xq)
    fp4_matmul(xq, w, out, add=residual)   # out = x weight^T + residual
"""

from __future__ import annotations

import ctypes

import torch

from . import FT_NVFP4, FtError, block_bytes, load
from .attention import _DT, _bad, _need, _status, _stream

FT_FP4_NVFP4, FT_FP4_MXFP4 = 0, 1
FT_FP4_TILES, FT_FP4_ROWS = 0, 1

_V, _I32, _I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
_SIGS = {
    "ft_fp4_scale_bytes": (ctypes.c_uint64, [_I32, _I32, _I64, _I64]),
    "ft_fp4_quantize": (_I32, [_V, _I64, _I32, _V, _I32, _V]),
    "ft_fp4_values": (_I32, [_V, _V, _I64, _I32, _V]),
    "ft_fp4_matmul": (_I32, [_V, _V, _V, _I64, _I32, _V, _I64, _V, _V]),
}
_lib = None


class FtFp4Matrix(ctypes.Structure):
    _fields_ = [("fmt", _I32), ("order", _I32), ("rows", _I64), ("K", _I64), ("pitch", _I64), ("codes", _V),
                ("scales", _V), ("scale", _V), ("scale_stride", _I64)]


def _bind():
    global _lib
    if _lib is None:
        lib = load()
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def _check(status, elsewhere=False):
    if status:
        more = " (for the tensors are not all on one GPU)" if elsewhere else ""
        raise FtError(status, _lib.ft_last_error().decode() + more)


def fp4_scale_bytes(fmt: int, order: int, rows: int, K: int) -> int:
    return int(_bind().ft_fp4_scale_bytes(fmt, order, rows, K))


class Fp4Matrix:
    """A matrix [rows, K] of 4-bit values: codes [rows, bytes of a row], block scales, and (NVFP4) fp32 scales of the
    rows or one of the matrix.  `Fp4Matrix.over` describes arrays that the caller has."""

    def __init__(self, fmt: int, rows: int, K: int, order: int = FT_FP4_TILES, device="cuda"):
        n = fp4_scale_bytes(fmt, order, max(rows, 1), K)
        _need(n > 0, f"Fp4Matrix: format {fmt}, order {order}, [{rows}, {K}]")
        codes = torch.zeros(rows, -(-K // 32) * 16, dtype=torch.uint8, device=device)
        scales = torch.zeros(n, dtype=torch.uint8, device=device)
        scale = torch.ones(rows, dtype=torch.float32, device=device) if fmt == FT_FP4_NVFP4 else None
        self._describe(fmt, K, codes, scales, scale, order)

    @classmethod
    def over(cls, fmt: int, K: int, codes, scales, scale=None, order: int = FT_FP4_TILES) -> "Fp4Matrix":
        self = cls.__new__(cls)
        self._describe(fmt, K, codes, scales, scale, order)
        return self

    def _describe(self, fmt, K, codes, scales, scale, order):
        _need(codes.dim() == 2 and codes.element_size() == 1, f"Fp4Matrix: codes {tuple(codes.shape)} {codes.dtype}")
        _need(not codes.dtype.is_floating_point or codes.dtype is torch.float4_e2m1fn_x2, f"Fp4Matrix: codes {codes.dtype}")
        rows, wide = codes.shape
        _need(K > 0 and 2 * wide >= K, f"Fp4Matrix: rows of {wide} bytes do not hold {K} values")
        _need(codes.stride(1) == 1 or wide == 1, "Fp4Matrix: a row's codes must be contiguous")
        _need(scales.element_size() == 1 and scales.is_contiguous(), "Fp4Matrix: scales must be contiguous bytes")
        own = torch.float8_e4m3fn if fmt == FT_FP4_NVFP4 else torch.float8_e8m0fnu
        _need(not scales.dtype.is_floating_point or scales.dtype is own, f"Fp4Matrix: scales {scales.dtype}")
        n = fp4_scale_bytes(fmt, order, rows, K)
        _need(rows == 0 or n > 0, f"Fp4Matrix: format {fmt}, order {order}, [{rows}, {K}]")
        _need(scales.numel() >= n, f"Fp4Matrix: {scales.numel()} bytes of scales, [{rows}, {K}] needs {n}")
        stride = 0
        if scale is not None:
            _need(scale.dtype is torch.float32 and scale.dim() <= 1 and scale.numel() in (1, rows),
                  f"Fp4Matrix: scale {tuple(scale.shape)} {scale.dtype}")
            stride = scale.stride(0) if scale.dim() == 1 and scale.numel() == rows and rows > 1 else 0
        self.fmt, self.order, self.rows, self.K = fmt, order, rows, K
        self.codes, self.scales, self.scale = codes, scales, scale
        self.dev = codes.get_device()
        _need(scales.get_device() == self.dev and (scale is None or scale.get_device() == self.dev),
              "Fp4Matrix: codes and scales are on different devices")
        # a matrix of one row may carry any stride
        pitch = codes.stride(0) if rows > 1 else -(-max(wide, codes.stride(0)) // 16) * 16
        self.desc = FtFp4Matrix(fmt, order, rows, K, pitch, codes.data_ptr(), scales.data_ptr(),
                                None if scale is None else scale.data_ptr(), stride)
        self._ref = ctypes.addressof(self.desc)


def expert_matrices(block, H: int, I: int, scales):
    """The gate, up and down matrices of one NVFP4 expert block (ft_moe.h; `block` its bytes, `scales` its three tensor
    scales [3] fp32), to be quantised into with given=True."""
    total, off = block_bytes(FT_NVFP4, H, I, 16)
    _need(total > 0, f"expert_matrices: no NVFP4 blocks of {H} x {I}")
    _need(block.dtype is torch.uint8 and block.dim() == 1 and block.is_contiguous() and block.numel() >= total,
          f"expert_matrices: a block has {total} contiguous bytes")
    _need(scales.dtype is torch.float32 and scales.shape == (3,), "expert_matrices: scales must be a float32 [3]")
    out = []
    for i, (rows, K) in enumerate(((I, H), (I, H), (H, I))):
        codes = block[off[i]:off[i] + rows * K // 2].view(rows, K // 2)
        out.append(Fp4Matrix.over(FT_FP4_NVFP4, K, codes, block[off[3 + i]:off[3 + i] + rows * K // 16],
                                  scale=scales[i:i + 1], order=FT_FP4_ROWS))
    return out


def _dense(t, name, rows, K):
    if t.shape != (rows, K):
        _bad(f"{name}: shape {tuple(t.shape)}, expected {(rows, K)}")
    if t.stride(1) != 1 and K > 1:
        _bad(f"{name}: columns must be contiguous")
    return t.stride(0) if rows > 1 else 0  # a matrix of one row may carry any stride


def fp4_quantize(x, m: Fp4Matrix, given: bool = False, stream=None):
    """m = x [rows, K], quantised (ft_fp4_quantize): NVFP4 rows with a scale that is found and written to m.scale, or
    with `given` the one that stands there."""
    lib = _lib or _bind()
    stride, dev = _dense(x, "x", m.rows, m.K), m.dev
    elsewhere = dev < 0 or x.get_device() != dev
    status = lib.ft_fp4_quantize(None if elsewhere else x.data_ptr(), stride, _DT.get(x.dtype, -1), m._ref, int(given),
                                 _stream(dev, stream))
    if status:
        _check(status, elsewhere)


def fp4_values(m: Fp4Matrix, out, stream=None):
    """out [rows, K] = the values that m stands for (ft_fp4_values)."""
    lib = _lib or _bind()
    stride, dev = _dense(out, "out", m.rows, m.K), m.dev
    elsewhere = dev < 0 or out.get_device() != dev
    status = lib.ft_fp4_values(m._ref, None if elsewhere else out.data_ptr(), stride, _DT.get(out.dtype, -1),
                               _stream(dev, stream))
    if status:
        _check(status, elsewhere)


def fp4_matmul(x: Fp4Matrix, w: Fp4Matrix, out, add=None, dev_status=None, stream=None):
    """out [T, N] = x [T, K] w [N, K]^T (+ add [T, N], which may be out) (ft_fp4_matmul)."""
    lib = _lib or _bind()
    dev = x.dev
    stride = _dense(out, "out", x.rows, w.rows)
    more = 0
    if add is not None:
        more = _dense(add, "add", x.rows, w.rows)
        if add.dtype is not out.dtype:
            _bad(f"add: dtype {add.dtype}, expected {out.dtype}")
    elsewhere = (dev < 0 or w.dev != dev or out.get_device() != dev or (add is not None and add.get_device() != dev)
                 or (dev_status is not None and dev_status.get_device() != dev))
    status = lib.ft_fp4_matmul(x._ref, w._ref, None if elsewhere else out.data_ptr(), stride, _DT.get(out.dtype, -1),
                               None if add is None else add.data_ptr(), more, _status(dev_status), _stream(dev, stream))
    if status:
        _check(status, elsewhere)
