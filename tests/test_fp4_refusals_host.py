"""Calls of the 4-bit matrices and of rotations by several axes that are taken or
refused at the edge of what the headers say, without a GPU: a call that is taken
comes as far as the launch, which fails here."""

import ctypes

import pytest
import torch

from test_fp4_host import C, att, fp4, refused  # noqa: F401

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are nobody's")
INVALID = 1


def test_rows_of_values_that_overlap_are_refused(fp4):  # noqa: F811
    c = C(fp4)
    values = lambda m, stride, dtype=0: c.lib.ft_fp4_values(ctypes.byref(m), 1 << 16, stride, dtype, None)
    for stride in (0, 8, 56):
        assert values(c.m(), stride) == INVALID and "overlap" in c.lib.ft_last_error().decode()
        assert values(c.m(rows=1), stride) != INVALID  # one row may carry any stride
        assert c.quantize(c.m(), stride=stride) != INVALID  # rows that are read may be one row
    assert values(c.m(), 60, 2) == INVALID
    assert values(c.m(), 64) != INVALID and values(c.m(), 72) != INVALID


def test_positions_may_be_the_same_on_every_axis(att):  # noqa: F811
    T, D = 3, 32
    rows, table = att._ROWS.pack(1 << 16, 64, 32), att.FtRopeTable(1 << 17, D, 0, 1.0)
    lib = att._bind()
    call = lambda stride, T=T: lib.ft_rope_by_axes(rows, T, 2, D, 0, 1 << 18, ctypes.addressof(table),
                                                   att._AXES.pack(1 << 19, 2, 0, stride), rows, None)
    assert call(0) != INVALID and call(T) != INVALID
    assert call(T - 1) == call(1) == call(-T) == call(-1) == INVALID


def test_positions_of_a_rotation_that_is_not_there_are_refused(att):  # noqa: F811
    from quantized_expert_ffn_router_gb300 import pipeline

    T, Hq, D = 2, 4, 32
    cache = att.KvCache(att.FT_KV_BF16, 2, D, 16, 4, device="cpu")
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    qkv = torch.zeros(T, (Hq + 4) * D, dtype=torch.bfloat16)
    plain = pipeline.DecodeAttention(cache, Hq, T, device="cpu")
    message = refused(plain, qkv, i(T, 1), i(T), rope_pos=i(T))
    assert "rope" in message and "GPU" not in message
    assert "GPU" in refused(plain, qkv, i(T, 1), i(T))  # without them it is a call of tensors that are on none


def test_one_row_in_place_may_carry_any_strides(fp4):  # noqa: F811
    c = C(fp4)
    assert c.matmul(c.m(rows=1), c.m(), stride=8, add=1 << 16, add_stride=16) != INVALID
    assert c.matmul(c.m(rows=2), c.m(), stride=8, add=1 << 16, add_stride=16) == INVALID
