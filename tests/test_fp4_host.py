"""4-bit matrices and rotations by several axes without a GPU: exported symbols,
sizes, sections, and what is refused before a kernel could see it."""

import ctypes
import os
import re

import pytest
import torch

from conftest import ROOT

HEADER = os.path.join(ROOT, "include", "ft_fp4.h")


@pytest.fixture(scope="module")
def fp4():
    from quantized_expert_ffn_router_gb300 import build as b

    b.build()
    from quantized_expert_ffn_router_gb300 import fp4

    fp4._bind()
    return fp4


@pytest.fixture(scope="module")
def att(fp4):
    from quantized_expert_ffn_router_gb300 import attention

    attention._bind()
    return attention


def refused(call, *a, status=1, **kw):
    with pytest.raises(Exception) as e:
        call(*a, **kw)
    assert getattr(e.value, "status", None) == status, e.value
    return str(e.value)


def test_every_declared_symbol_is_bound(fp4):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    assert set(re.findall(r"\b(ft_\w+)\s*\(", text)) == set(fp4._SIGS)


def test_scale_bytes(fp4):
    n = fp4.fp4_scale_bytes
    assert n(0, 0, 1, 16) == n(0, 0, 128, 64) == 512 and n(0, 0, 129, 64) == 1024 and n(0, 0, 128, 80) == 1024
    assert n(1, 0, 128, 128) == 512 and n(1, 0, 300, 160) == 3 * 2 * 512
    assert n(0, 1, 5, 48) == 15 and n(1, 1, 5, 64) == 10
    assert n(0, 0, 2 ** 31 - 1, 2 ** 31 - 16) == 2 ** 24 * 2 ** 25 * 512
    for bad in ((2, 0, 4, 64), (0, 2, 4, 64), (0, 0, 0, 64), (0, 0, 4, 0), (0, 0, 4, 24), (1, 0, 4, 48), (0, 0, 2 ** 31, 64),
                (0, 0, 4, 2 ** 31)):
        assert n(*bad) == 0


def matrix(fp4, fmt=0, rows=4, K=64, order=0):
    return fp4.Fp4Matrix(fmt, rows, K, order, device="cpu")


def test_matrices_that_do_not_fit_are_refused(fp4):
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    over = lambda fmt=0, K=64, codes=u8(4, 32), scales=u8(512), **kw: fp4.Fp4Matrix.over(fmt, K, codes, scales, **kw)
    over()
    over(scales=u8(512).view(torch.float8_e4m3fn))
    over(fmt=1, scales=u8(512).view(torch.float8_e8m0fnu))
    over(scale=torch.ones(()))
    over(codes=u8(4, 64)[:, :32], scale=torch.ones(1))
    for bad in (dict(K=80), dict(K=24), dict(K=0), dict(fmt=3), dict(order=2), dict(scales=u8(511)), dict(codes=u8(4, 32, 1)),
                dict(codes=u8(4, 64)[:, ::2]), dict(scales=u8(1024)[::2]), dict(codes=torch.zeros(4, 32)),
                dict(scales=u8(512).view(torch.float8_e8m0fnu)), dict(scale=torch.ones(3)), dict(scale=torch.ones(4).double()),
                dict(scale=torch.ones(4, 1)), dict(fmt=1, K=48)):
        refused(over, **bad)
    refused(fp4.Fp4Matrix, 0, 4, 24, device="cpu")


@pytest.mark.parametrize("stream", [None, 0])
def test_tensors_that_are_not_on_a_gpu_are_refused(fp4, stream):
    m, w, x, out = matrix(fp4), matrix(fp4, rows=6), torch.zeros(4, 64), torch.zeros(4, 6)
    refused(fp4.fp4_quantize, x, m, stream=stream)
    refused(fp4.fp4_values, m, x, stream=stream)
    refused(fp4.fp4_matmul, m, w, out, stream=stream)
    none = matrix(fp4, rows=0)  # a call of no rows reads nothing
    fp4.fp4_quantize(torch.zeros(0, 64), none, stream=stream)
    fp4.fp4_values(none, torch.zeros(0, 64), stream=stream)
    fp4.fp4_matmul(none, w, torch.zeros(0, 6), stream=stream)


def test_arguments_that_do_not_fit_are_refused(fp4):
    m, w = matrix(fp4), matrix(fp4, rows=6)
    for bad in (torch.zeros(4, 80), torch.zeros(5, 64), torch.zeros(4, 128)[:, ::2], torch.zeros(64)):
        refused(fp4.fp4_quantize, bad, m)
        refused(fp4.fp4_values, m, bad)
    out = torch.zeros(4, 6)
    refused(fp4.fp4_matmul, m, w, torch.zeros(4, 7))
    refused(fp4.fp4_matmul, m, w, torch.zeros(4, 12)[:, ::2])
    refused(fp4.fp4_matmul, m, w, out, add=torch.zeros(4, 5))
    refused(fp4.fp4_matmul, m, w, out, add=torch.zeros(4, 6, dtype=torch.bfloat16))
    refused(fp4.fp4_matmul, m, w, out, dev_status=torch.zeros(1))


class C:
    """Calls with addresses that nothing is read from: what the library refuses by itself."""

    def __init__(self, fp4):
        self.fp4, self.lib = fp4, fp4._bind()

    def m(self, **kw):
        a = dict(fmt=0, order=0, rows=4, K=64, pitch=32, codes=1 << 20, scales=1 << 21, scale=1 << 22, scale_stride=1)
        return self.fp4.FtFp4Matrix(**{**a, **kw})

    def quantize(self, m, x=1 << 16, stride=64, dtype=0, given=0):
        return self.lib.ft_fp4_quantize(x, stride, dtype, ctypes.byref(m) if m else None, given, None)

    def matmul(self, x, w, out=1 << 16, stride=8, dtype=0, add=None, add_stride=8):
        return self.lib.ft_fp4_matmul(ctypes.byref(x), ctypes.byref(w), out, stride, dtype, add, add_stride, None, None)


def test_the_library_refuses(fp4):
    c = C(fp4)
    assert c.quantize(None) == 1
    for want, bad in ((2, dict(fmt=2)), (2, dict(order=5)), (1, dict(K=0)), (1, dict(K=72)), (2, dict(rows=1 << 31)),
                      (1, dict(rows=-1)), (1, dict(codes=None)), (1, dict(scales=None)), (1, dict(codes=(1 << 20) + 8)),
                      (1, dict(scales=(1 << 21) + 4)), (1, dict(pitch=24)), (1, dict(pitch=16)), (1, dict(scale=(1 << 22) + 2)),
                      (1, dict(scale_stride=-1)), (1, dict(fmt=1)), (1, dict(fmt=1, K=48, scale=None))):
        assert c.quantize(c.m(**bad)) == want, bad
        assert c.matmul(c.m(**bad), c.m()) == want and c.matmul(c.m(), c.m(**bad)) == want, bad
    # the scale of the rows has to have a place when it is found
    for bad in (dict(scale=None), dict(scale_stride=0)):
        assert c.quantize(c.m(**bad)) == 1
    for bad in (dict(x=None), dict(x=(1 << 16) + 8), dict(stride=60), dict(stride=-64), dict(dtype=3), dict(dtype=-1)):
        assert c.quantize(c.m(), **bad) == 1, bad
    # products
    assert c.matmul(c.m(), c.m(fmt=1, scale=None)) == 1 and c.matmul(c.m(), c.m(K=128, pitch=64)) == 1
    assert c.matmul(c.m(order=1), c.m()) == 2 and c.matmul(c.m(), c.m(order=1)) == 2
    for bad in (dict(out=None), dict(out=(1 << 16) + 1), dict(stride=-8), dict(dtype=4), dict(add=(1 << 17) + 1),
                dict(add=1 << 17, add_stride=-1), dict(add=1 << 16, add_stride=16), dict(stride=3), dict(stride=0)):
        assert c.matmul(c.m(), c.m(), **bad) == 1, bad
    for rows in ((1 << 31) - 1, (1 << 31) - 1023):
        assert c.matmul(c.m(rows=rows), c.m()) == 2 and c.matmul(c.m(), c.m(rows=rows)) == 2
    assert c.quantize(c.m(rows=0)) == c.matmul(c.m(rows=0), c.m()) == c.matmul(c.m(), c.m(rows=0)) == 0


# ------------------------------------------------------------ several axes ---
def axes(att, rot, sections, weave):
    return att.Rope(rot, device="cpu", sections=sections, weave=weave).axis.tolist()


def test_sections(att):
    assert axes(att, 16, (2, 3, 3), False) == [0, 0, 1, 1, 1, 2, 2, 2]
    assert axes(att, 16, (0, 8), False) == [1] * 8
    assert axes(att, 16, (4, 2, 2), True) == [0, 1, 2, 0, 1, 2, 0, 0]
    assert axes(att, 14, (3, 2, 2), True) == [0, 1, 2, 0, 1, 2, 0]
    assert axes(att, 8, (4,), True) == [0] * 4
    assert axes(att, 16, (8, 0, 0), True) == [0] * 8
    from test_gpu_rope_axes import CASES, axis_of

    for _, rot, sections, weave in CASES:
        got = axes(att, rot, sections, weave)
        assert got == axis_of(sections, weave).tolist() and [got.count(a) for a in range(len(sections))] == list(sections)


def test_sections_that_do_not_fit_are_refused(att):
    for rot, sections, weave in ((16, (2, 3, 2), False), (16, (9, -1), False), (16, (), False), (18, (1,) * 9, False),
                                 (16, (2, 3, 3, 1), False), (16, (1, 4, 3), True), (16, (2, 3, 3), True), (15, (7,), False)):
        refused(att.Rope, rot, device="cpu", sections=sections, weave=weave)
    refused(att.Rope, 16, device="cpu", weave=True)


def test_positions_of_axes_that_do_not_fit_are_refused(att):
    T, D = 3, 32
    x = torch.zeros(T, 2, D, dtype=torch.bfloat16)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    two, one = att.Rope(D, device="cpu", sections=(8, 8)), att.Rope(D, device="cpu")
    for pos in (i(T), i(3, T), i(2, T + 1), torch.zeros(2, T), i(2, 2 * T)[:, ::2]):
        message = refused(att.rope, x, pos, two, x)
        assert "GPU" not in message
    refused(att.rope, x, i(2, T), one, x)
    assert "GPU" in refused(att.rope, x, i(2, T), two, x)
    cache = att.KvCache(att.FT_KV_BF16, 2, D, 16, 4, device="cpu")
    assert "rope_pos" in refused(att.kv_append, cache, x, x, i(T, 1), i(T), rope=two, q=x, q_out=x)
    assert "GPU" in refused(att.kv_append, cache, x, x, i(T, 1), i(T), rope=two, rope_pos=i(2, T), q=x, q_out=x)
    # positions of one axis behind the other's
    lib = att._bind()
    rows = att._ROWS.pack(1 << 16, 64, 32)
    table = att.FtRopeTable(1 << 17, D, 0, 1.0)
    call = lambda axis, n, stride: lib.ft_rope_by_axes(rows, T, 2, D, 0, 1 << 18, ctypes.addressof(table),
                                                       att._AXES.pack(axis, n, 0, stride), rows, None)
    for bad in ((0, 2, T), (1 << 19, 0, T), (1 << 19, 9, T), (1 << 19, 2, T - 1)):
        assert call(*bad) == 1, bad
    assert lib.ft_rope_by_axes(rows, T, 2, D, 0, 1 << 18, ctypes.addressof(table), None, rows, None) == 1
