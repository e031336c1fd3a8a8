"""Attention operators next to the expert layer: rotary positions, the paged
key-value cache (16-, 8- and 4-bit rows) and the attention of one new token a
row over it.

Argument marshalling over the C ABI declared in include/ft_attn.h, which says
what each call computes; errors raise FtError.  Tensors may be strided views
(channels contiguous); calls enqueue on the current stream (or `stream`).

    cache = KvCache(FT_KV_E4M3, Hkv=8, D=128, page_size=64, n_pages=4096)
    spin = Rope(128, base=5e5)
    ws = torch.zeros(attn_decode_workspace(T, Hq, 8, 128), dtype=torch.uint8, device="cuda")
    # every step, for T sequences: pos[t] = tokens already cached, lens[t] = pos[t] + 1
    kv_append(cache, k, v, pages, pos, rope=spin, q=q, q_out=q)
    attn_decode(cache, q, pages, lens, out, ws)
"""

from __future__ import annotations

import ctypes
import struct

import torch

from . import FT_ERR_INVALID, FT_OK, FtError, load

FT_KV_BF16, FT_KV_F16, FT_KV_E4M3, FT_KV_NVFP4 = range(4)
FT_DT_BF16, FT_DT_F16, FT_DT_F32 = range(3)
(FT_ROPE_PLAIN, FT_ROPE_LINEAR, FT_ROPE_BASE, FT_ROPE_PARTS_BY_TURNS, FT_ROPE_PARTS_BY_INDEX) = range(5)

_DT = {torch.bfloat16: FT_DT_BF16, torch.float16: FT_DT_F16, torch.float32: FT_DT_F32}

_V, _I32, _F, _D, _SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_double, ctypes.c_size_t
_SIGS = {
    "ft_rope_freqs": (_I32, [_I32, _D, _I32, _D, _D, _D, _I32, _V]),
    "ft_rope": (_I32, [_V, _I32, _I32, _I32, _I32, _V, _V, _V, _V]),
    "ft_rope_sections": (_I32, [_I32, _V, _I32, _I32, _V]),
    "ft_rope_by_axes": (_I32, [_V, _I32, _I32, _I32, _I32, _V, _V, _V, _V, _V]),
    "ft_kv_row_bytes": (ctypes.c_uint64, [_I32, _I32]),
    "ft_kv_append": (_I32, [_V, _V, _V, _I32, _I32, _V, _V, _V, _V, _V, _V, _I32, _V, _V, _V]),
    "ft_kv_append_by_axes": (_I32, [_V, _V, _V, _I32, _I32, _V, _V, _V, _V, _V, _V, _V, _I32, _V, _V, _V]),
    "ft_kv_gather": (_I32, [_V, _V, _V, _V, _I32, _V, _V, _I32, _V, _V]),
    "ft_attn_decode_workspace": (_SZ, [_I32, _I32, _I32, _I32]),
    "ft_attn_decode": (_I32, [_V, _V, _I32, _I32, _I32, _V, _V, _V, _F, _I32, _V, _I32, _V, _V, _SZ, _V, _V]),
}
_lib = None

# The descriptors of ft_attn.h as packed bytes (cheaper to build for each call than ctypes structures).
_ROWS = struct.Struct("=Qqq")
_TABLE = struct.Struct("=Qqii")
_AXES = struct.Struct("=Qiiq")


class FtKvCache(ctypes.Structure):
    _fields_ = [("fmt", _I32), ("Hkv", _I32), ("D", _I32), ("page_size", _I32), ("n_pages", ctypes.c_int64),
                ("page_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64), ("slot_stride", ctypes.c_int64),
                ("k", _V), ("v", _V), ("k_scale", _V), ("v_scale", _V), ("k_block", _V), ("v_block", _V)]


class FtRopeTable(ctypes.Structure):
    _fields_ = [("freqs", _V), ("rot_dim", _I32), ("interleaved", _I32), ("mscale", _F)]


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


def _need(ok, message):
    if not ok:
        raise FtError(FT_ERR_INVALID, message)


def _bad(message):
    raise FtError(FT_ERR_INVALID, message)


def _check(status, elsewhere=False):
    if status != FT_OK:
        more = " (for the tensors are not all on one GPU)" if elsewhere else ""
        raise FtError(status, _lib.ft_last_error().decode() + more)


def _stream(dev, stream):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev) if dev >= 0 else 0
    return stream if isinstance(stream, int) else stream.cuda_stream


# The checks below build their messages only when they fail: a decode step calls these functions once a layer, and
# formatting them costs more than the launch.  Where the tensors are not all on one GPU, a kernel may not use their
# addresses: the call is made without its positions (or lengths) then, which the library refuses after its own checks.
def _rows(t, name, shape, dtype):
    """A tensor of this [T, heads, D] and type as an ft_rows."""
    if t.shape != shape:
        _bad(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype is not dtype:
        _bad(f"{name}: dtype {t.dtype}, expected {dtype}")
    return _rows_of(t, name, shape)


def _rows_of(t, name, shape):
    """The same of a tensor whose shape and type have been looked at."""
    s0, s1, s2 = t.stride()
    if s2 != 1:
        _bad(f"{name}: channels must be contiguous")
    # a dimension of one place may carry any stride
    return _ROWS.pack(t.data_ptr(), s0 if shape[0] > 1 else 0, s1 if shape[1] > 1 else 0)


def _ints(t, name, T):
    if t is None:
        return None
    if t.dtype is not torch.int32 or t.numel() != T or not t.is_contiguous():
        _bad(f"{name}: a contiguous int32 [{T}] is needed")
    return t.data_ptr()


def _table(pages):
    if pages.dim() != 2 or pages.dtype is not torch.int32:
        _bad("pages: an int32 [sequences, pages] is needed")
    (s0, s1), (n, most) = pages.stride(), pages.shape
    if s1 != 1 and most > 1:  # a dimension of one place may carry any stride
        _bad("pages: a sequence's pages must be contiguous")
    return _TABLE.pack(pages.data_ptr(), s0, most, n)


def _status(t):
    if t is None:
        return None
    if t.dtype is not torch.int32 or t.numel() < 1:
        _bad("dev_status: an int32 tensor is needed")
    return t.data_ptr()


def _ptr(t):
    return None if t is None else t.data_ptr()


def kv_row_bytes(fmt: int, D: int) -> int:
    return int(_bind().ft_kv_row_bytes(fmt, D))


class KvCache:
    """One layer's paged cache: rows [n_pages, Hkv, page_size] of D values.

    Arrays: k, v (16-bit values; float8_e4m3fn codes; uint8 pairs of E2M1
    codes), k_scale, v_scale (uint8 exponents + 127), k_block, v_block (uint8
    E4M3 block scales).  `KvCache.over` describes arrays that the caller has,
    in any order of pages, heads and slots (the rows' last dimension contiguous
    and the same row strides for all arrays)."""

    def __init__(self, fmt: int, Hkv: int, D: int, page_size: int, n_pages: int, device="cuda"):
        shape, z = (n_pages, Hkv, page_size), dict(device=device)
        arrays = {}
        for n in ("k", "v"):
            if fmt in (FT_KV_BF16, FT_KV_F16):
                arrays[n] = torch.zeros(*shape, D, dtype=torch.bfloat16 if fmt == FT_KV_BF16 else torch.float16, **z)
                continue
            if fmt == FT_KV_E4M3:
                arrays[n] = torch.zeros(*shape, D, dtype=torch.float8_e4m3fn, **z)
            else:
                arrays[n] = torch.zeros(*shape, D // 2, dtype=torch.uint8, **z)
                arrays[n + "_block"] = torch.zeros(*shape, D // 16, dtype=torch.uint8, **z)
            arrays[n + "_scale"] = torch.full(shape, 127, dtype=torch.uint8, **z)
        self._describe(fmt, D, arrays)

    @classmethod
    def over(cls, fmt: int, D: int, k, v, k_scale=None, v_scale=None, k_block=None, v_block=None) -> "KvCache":
        self = cls.__new__(cls)
        self._describe(fmt, D, dict(k=k, v=v, k_scale=k_scale, v_scale=v_scale, k_block=k_block, v_block=v_block))
        return self

    def _describe(self, fmt, D, arrays):
        width = {FT_KV_BF16: D, FT_KV_F16: D, FT_KV_E4M3: D, FT_KV_NVFP4: D // 2}.get(fmt)
        _need(width is not None, f"cache format {fmt}")
        k = arrays["k"]
        _need(k.dim() == 4, "cache arrays are [pages, heads, slots, ...]")
        self.dev = k.get_device()
        n_pages, Hkv, page_size = k.shape[:3]
        # each array's own floating type; integers of its size are taken for its bits
        own = {"": {FT_KV_BF16: torch.bfloat16, FT_KV_F16: torch.float16, FT_KV_E4M3: torch.float8_e4m3fn,
                    FT_KV_NVFP4: torch.float4_e2m1fn_x2}[fmt], "_scale": torch.float8_e8m0fnu, "_block": torch.float8_e4m3fn}
        strides = None
        for name in ("k", "v", "k_scale", "v_scale", "k_block", "v_block"):
            t = arrays.get(name)
            setattr(self, name, t)
            if t is None:
                continue
            w = width if name in ("k", "v") else D // 16 if name.endswith("_block") else 1
            shape = (n_pages, Hkv, page_size) + (() if name.endswith("_scale") else (w,))
            size = 2 if fmt in (FT_KV_BF16, FT_KV_F16) and name in ("k", "v") else 1
            _need(tuple(t.shape) == shape and t.element_size() == size, f"cache {name}: {tuple(t.shape)} {t.dtype}")
            _need(not t.dtype.is_floating_point or t.dtype is own[name[1:]], f"cache {name}: {t.dtype}")
            _need(t.get_device() == self.dev, f"cache {name}: on {t.device}, the keys are on {k.device}")
            _need(t.dim() == 3 or t.stride(3) == 1, f"cache {name}: rows must be contiguous")
            _need(all(s % w == 0 for s in t.stride()[:3]), f"cache {name}: strides must be whole rows")
            # a dimension of one place has no stride of its own
            rows = [s // w if n > 1 else 0 for s, n in zip(t.stride()[:3], shape)]
            _need(strides is None or rows == strides, f"cache {name}: row strides {rows}, the keys' are {strides}")
            strides = rows
        self.fmt, self.Hkv, self.D, self.page_size, self.n_pages = fmt, Hkv, D, page_size, n_pages
        self.desc = FtKvCache(fmt, Hkv, D, page_size, n_pages, *strides, *(
            _ptr(arrays.get(n)) for n in ("k", "v", "k_scale", "v_scale", "k_block", "v_block")))
        self._ref = ctypes.addressof(self.desc)


class Rope:
    """A rotary table (ft_rope_freqs on the host, kept on the device).

    sections: how many channel pairs turn by each of several axes (time, height, width), in runs or, with `weave`,
    taking turns (ft_rope_sections).  Positions are then [axes, T]."""

    def __init__(self, rot_dim: int, base: float = 10000.0, interleaved: bool = False, scaling: int = FT_ROPE_PLAIN,
                 factor: float = 1.0, low: float = 1.0, high: float = 32.0, orig_len: int = 8192,
                 mscale: float = 1.0, device="cuda", sections=None, weave: bool = False):
        host = torch.empty(max(rot_dim, 0) // 2, dtype=torch.int64)
        lib = _bind()
        _check(lib.ft_rope_freqs(rot_dim, base, scaling, factor, low, high, orig_len, host.data_ptr()))
        self.rot_dim, self.interleaved, self.mscale = rot_dim, bool(interleaved), float(mscale)
        self.freqs = host.to(device)
        self.dev = self.freqs.get_device()
        self.desc = FtRopeTable(self.freqs.data_ptr(), rot_dim, int(self.interleaved), self.mscale)
        self._ref = ctypes.addressof(self.desc)
        self.n_axes, self.axis = 1, None
        if sections is None:
            _need(not weave, "Rope: weave is for sections")
            return
        counts = torch.tensor(list(sections), dtype=torch.int32)
        axis = torch.empty(rot_dim // 2, dtype=torch.uint8)
        _check(lib.ft_rope_sections(rot_dim, counts.data_ptr(), counts.numel(), int(weave), axis.data_ptr()))
        self.n_axes, self.axis = counts.numel(), axis.to(device)

    def _positions(self, pos, name, T):
        """(address of the positions, an ft_rope_axes or None)."""
        if self.axis is None:
            return _ints(pos, name, T), None
        n = self.n_axes
        if pos.dtype is not torch.int32 or pos.shape != (n, T):
            _bad(f"{name}: an int32 [{n}, {T}] is needed, a row for each axis")
        stride, step = pos.stride()
        if step != 1 and T > 1:
            _bad(f"{name}: an axis's positions must be contiguous")
        return pos.data_ptr(), _AXES.pack(self.axis.data_ptr(), n, 0, stride if n > 1 else T)


def _shape3(t, name, heads, D):
    """t's [T, heads, D] with these heads and channels (None: any)."""
    shape = t.shape
    if len(shape) != 3 or (heads is not None and shape[1] != heads) or (D is not None and shape[2] != D):
        _bad(f"{name}: shape {tuple(shape)}, expected [T, {'*' if heads is None else heads}, {'*' if D is None else D}]")
    return shape


def rope(x, pos, table: Rope, out, stream=None):
    """out[t, h] = x[t, h] rotated to pos[t], or by several axes to pos[:, t] (ft_rope, ft_rope_by_axes); out may be x."""
    lib = _lib or _bind()
    dtype, dev = x.dtype, x.get_device()
    T, heads, D = shape = _shape3(x, "x", None, None)
    at, axes = table._positions(pos, "pos", T)
    elsewhere = dev < 0 or table.dev != dev or (at is not None and pos.get_device() != dev) or out.get_device() != dev
    if axes is None:
        status = lib.ft_rope(_rows_of(x, "x", shape), T, heads, D, _DT.get(dtype, -1), None if elsewhere else at,
                             table._ref, _rows(out, "out", shape, dtype), _stream(dev, stream))
    else:
        status = lib.ft_rope_by_axes(_rows_of(x, "x", shape), T, heads, D, _DT.get(dtype, -1), None if elsewhere else at,
                                     table._ref, axes, _rows(out, "out", shape, dtype), _stream(dev, stream))
    if status:
        _check(status, elsewhere)


def kv_append(cache: KvCache, k, v, pages, pos, seq=None, rope: Rope | None = None, rope_pos=None, q=None, q_out=None,
              dev_status=None, stream=None):
    """Write k and v [T, Hkv, D] to position pos[t] of sequence seq[t] (default t); with `rope`, k is rotated first
    and q into q_out in the same launch (ft_kv_append).  Of several axes, rope_pos [axes, T] has to be given
    (ft_kv_append_by_axes)."""
    lib = _lib or _bind()
    dtype, dev = k.dtype, k.get_device()
    shape = _shape3(k, "k", cache.Hkv, cache.D)
    T = shape[0]
    at = _ints(pos, "pos", T)
    elsewhere = (dev < 0 or cache.dev != dev or v.get_device() != dev or pages.get_device() != dev
                 or (at is not None and pos.get_device() != dev) or (seq is not None and seq.get_device() != dev)
                 or (dev_status is not None and dev_status.get_device() != dev)
                 or (rope is not None and (rope.dev != dev or (rope_pos is not None and rope_pos.get_device() != dev))))
    Hq, q_rows, q_out_rows = 0, None, None
    if q is not None:
        q_shape = _shape3(q, "q", None, cache.D)
        Hq = q_shape[1]
        if q_shape[0] != T or q_out is None:
            _bad("kv_append: q has k's tokens, and needs q_out")
        if q.dtype is not dtype:
            _bad(f"q: dtype {q.dtype}, expected {dtype}")
        q_rows, q_out_rows = _rows_of(q, "q", q_shape), _rows(q_out, "q_out", q_shape, dtype)
        elsewhere = elsewhere or q.get_device() != dev or q_out.get_device() != dev
    if rope is None or rope.axis is None:
        status = lib.ft_kv_append(
            cache._ref, _rows_of(k, "k", shape), _rows(v, "v", shape, dtype), T, _DT.get(dtype, -1), _table(pages),
            None if seq is None else _ints(seq, "seq", T), None if elsewhere else at, None if rope is None else rope._ref,
            None if rope_pos is None else _ints(rope_pos, "rope_pos", T), q_rows, Hq, q_out_rows, _status(dev_status),
            _stream(dev, stream))
    else:
        if rope_pos is None:
            _bad("kv_append: several axes need rope_pos")
        turns, axes = rope._positions(rope_pos, "rope_pos", T)
        status = lib.ft_kv_append_by_axes(
            cache._ref, _rows_of(k, "k", shape), _rows(v, "v", shape, dtype), T, _DT.get(dtype, -1), _table(pages),
            None if seq is None else _ints(seq, "seq", T), None if elsewhere else at, rope._ref, axes, turns, q_rows, Hq,
            q_out_rows, _status(dev_status), _stream(dev, stream))
    if status:
        _check(status, elsewhere)


def kv_gather(cache: KvCache, pages, pos, k_out, v_out, seq=None, dev_status=None, stream=None):
    """k_out, v_out [T, Hkv, D] (either may be None) = the cached rows of position pos[t] of sequence seq[t]
    (ft_kv_gather)."""
    lib = _lib or _bind()
    some = k_out if k_out is not None else v_out
    if some is None:
        _bad("kv_gather: no output")
    dtype, dev = some.dtype, some.get_device()
    shape = _shape3(some, "output", cache.Hkv, cache.D)
    T = shape[0]
    at = _ints(pos, "pos", T)
    elsewhere = (dev < 0 or cache.dev != dev or (v_out is not None and v_out.get_device() != dev)
                 or pages.get_device() != dev or (at is not None and pos.get_device() != dev)
                 or (seq is not None and seq.get_device() != dev)
                 or (dev_status is not None and dev_status.get_device() != dev))
    status = lib.ft_kv_gather(
        cache._ref, _table(pages), None if seq is None else _ints(seq, "seq", T), None if elsewhere else at, T,
        None if k_out is None else _rows_of(k_out, "k_out", shape),
        None if v_out is None else _rows(v_out, "v_out", shape, dtype), _DT.get(dtype, -1), _status(dev_status),
        _stream(dev, stream))
    if status:
        _check(status, elsewhere)


def attn_decode_workspace(T: int, Hq: int, Hkv: int, D: int) -> int:
    return int(_bind().ft_attn_decode_workspace(T, Hq, Hkv, D))


def attn_decode(cache: KvCache, q, pages, lens, out, ws, seq=None, scale: float | None = None, window: int = 0,
                lse=None, dev_status=None, stream=None):
    """out [T, Hq, D] = attention of q [T, Hq, D] over the first lens[t] (with `window`: the last `window` of them)
    cached tokens of sequence seq[t] (ft_attn_decode).  scale defaults to 1 / sqrt(D)."""
    lib = _lib or _bind()
    T, Hq, D = shape = _shape3(q, "q", None, cache.D)
    dtype, out_dtype, dev = q.dtype, out.dtype, q.get_device()
    if lse is not None and (lse.dtype is not torch.float32 or lse.shape != (T, Hq) or not lse.is_contiguous()):
        _bad("attn_decode: lse must be a contiguous float32 [T, Hq]")
    if not ws.is_contiguous():
        _bad("attn_decode: ws must be contiguous")
    at = _ints(lens, "lens", T)
    elsewhere = (dev < 0 or cache.dev != dev or out.get_device() != dev or pages.get_device() != dev
                 or (at is not None and lens.get_device() != dev) or ws.get_device() != dev
                 or (seq is not None and seq.get_device() != dev) or (lse is not None and lse.get_device() != dev)
                 or (dev_status is not None and dev_status.get_device() != dev))
    status = lib.ft_attn_decode(
        cache._ref, _rows_of(q, "q", shape), T, Hq, _DT.get(dtype, -1), _table(pages),
        None if seq is None else _ints(seq, "seq", T), None if elsewhere else at, D ** -0.5 if scale is None else scale,
        window, _rows(out, "out", shape, out_dtype), _DT.get(out_dtype, -1), None if lse is None else lse.data_ptr(),
        ws.data_ptr(), ws.nbytes, _status(dev_status), _stream(dev, stream))
    if status:
        _check(status, elsewhere)
