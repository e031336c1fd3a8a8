"""Rotary positions with several axes, alone and on the way into the cache:
against the formula in 64 bits, and each axis's channels against the rotation by
that axis alone, bit for bit."""

import math

import numpy as np
import pytest
import torch

from attn_helpers import DT, FMT, f64, quantised, random_table, rotated
from test_gpu_kv import i32, rope_bound, rows

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def att(cuda_lib):
    from quantized_expert_ffn_router_gb300 import attention

    return attention


def axis_of(sections, weave):
    """Each pair's axis, one pair after the other."""
    left, out = list(sections), []
    for i in range(sum(sections)):
        a = i % len(sections) if weave else next(j for j, n in enumerate(left) if n)
        if weave and i // len(sections) >= sections[a]:
            a = 0
        left[a] -= 1
        out.append(a)
    return np.array(out)


def turned(x, pos, spin, sections, weave, layout, mscale):
    """Rows [T, h, D] turned by pos [axes, T], in 64 bits: a pair at a time."""
    freqs = spin.freqs.cpu().numpy().astype(np.float64) * (2 * math.pi / 2.0 ** 64)
    y = np.array(x, np.float64)
    for i, a in enumerate(axis_of(sections, weave)):
        one = np.where(np.arange(len(freqs)) == i, freqs, 0.0)
        at = (2 * i, 2 * i + 1) if layout == "pairs" else (i, i + len(freqs))
        y[..., at] = rotated(x, pos[a], one, layout, mscale)[..., at]
    return y


CASES = [  # D, rot, sections, weave
    (128, 128, (24, 20, 20), True), (128, 128, (16, 24, 24), False), (128, 64, (8, 12, 12), False), (64, 64, (32,), False),
    (256, 64, (11, 11, 10), True), (80, 80, (13, 20, 7), False), (96, 32, (0, 16), False), (72, 24, (4, 4, 4), True),
    (8, 8, (1, 1, 1, 1), True), (128, 20, (3, 0, 7), False), (128, 2, (1,), True), (192, 96, (6, 6, 6, 6, 6, 6, 6, 6), False),
    (256, 254, (100, 27), True)]


def positions(n, T, seed):
    p = np.random.default_rng(seed).integers(0, 1 << 20, (n, T))
    p[:, 0], p[-1, -1] = 0, 2 ** 31 - 1
    return p


@pytest.mark.parametrize("D,rot,sections,weave", CASES)
@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_rope_axes(att, D, rot, sections, weave, layout, dtype):
    T, h, n = 7, 3, len(sections)
    x = rows(T, h, D, dtype, D + rot)
    kw = dict(base=5e5, interleaved=layout == "pairs", mscale=1.25)
    spin = att.Rope(rot, sections=sections, weave=weave, **kw)
    one = att.Rope(rot, **kw)
    pos = positions(n, T, D)
    wide = torch.full((n, T + 5), -7, dtype=torch.int32, device=DEV)  # rows of positions further apart
    wide[:, :T] = i32(pos)
    out = torch.full((T, h, D), float("nan"), dtype=DT[dtype], device=DEV)
    att.rope(x, wide[:, :T], spin, out)
    want = turned(f64(x), pos, spin, sections, weave, layout, 1.25)
    assert (np.abs(f64(out) - want) <= rope_bound(x, spin, dtype, want)).all()
    assert torch.equal(out[..., rot:], x[..., rot:])
    for a in range(n):
        alone = torch.empty_like(out)
        att.rope(x, i32(pos[a]), one, alone)
        at = np.flatnonzero(axis_of(sections, weave) == a)
        ch = np.concatenate([2 * at, 2 * at + 1]) if layout == "pairs" else np.concatenate([at, at + rot // 2])
        assert torch.equal(out[..., ch], alone[..., ch])
    att.rope(x, wide[:, :T], spin, x)  # in place
    assert torch.equal(x, out)


@pytest.mark.parametrize("T,Hkv,D,page,rot,sections,weave", [
    (1, 1, 64, 16, 64, (12, 10, 10), True), (33, 3, 128, 24, 64, (16, 8, 8), False), (70, 8, 64, 1, 32, (5, 11), False),
    (300, 4, 128, 32, 128, (24, 20, 20), True), (17, 5, 96, 48, 96, (16, 16, 16), True)])
@pytest.mark.parametrize("fmt,dtype", [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "bf16"), ("e4m3", "f16"), ("nvfp4", "bf16")])
@pytest.mark.parametrize("layout", ["half", "pairs"])
def test_append_axes(att, T, Hkv, D, page, rot, sections, weave, fmt, dtype, layout):
    n = [T - T // 3, T // 3] if T > 2 else [T]
    pages = sum(-(-x // page) for x in n) + 1
    table = i32(random_table(n, page, pages, T))
    seq = np.repeat(np.arange(len(n)), n)
    at = np.concatenate([np.arange(a) for a in n])
    cache = att.KvCache(FMT[fmt], Hkv, D, page, pages)
    k, v, q = (rows(T, h, D, dtype, s) for h, s in ((Hkv, 1), (Hkv, 2), (2 * Hkv, 3)))
    q_out = torch.zeros(T, 2 * Hkv, D, dtype=DT[dtype], device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    spin = att.Rope(rot, base=1e4, interleaved=layout == "pairs", mscale=1.125, sections=sections, weave=weave)
    pos = positions(len(sections), T, T)
    skip = T // 2 if T > 2 else -1  # a padding token: not written, its query rotated all the same
    places = np.where(np.arange(T) == skip, -1, at)
    att.kv_append(cache, k, v, table, i32(places), seq=i32(seq), rope=spin, rope_pos=i32(pos), q=q, q_out=q_out, dev_status=status)
    ko, vo = (torch.full((T, Hkv, D), float("nan"), device=DEV) for _ in "kv")
    att.kv_gather(cache, table, i32(places), ko, vo, seq=i32(seq), dev_status=status)
    assert int(status.item()) == 0
    kept = np.arange(T) != skip
    turn = lambda x: turned(f64(x), pos, spin, sections, weave, layout, 1.125)
    assert (f64(vo)[kept] == quantised(fmt, f64(v))[kept]).all() and (f64(vo)[~kept] == 0).all()
    want = turn(k)
    if fmt in ("bf16", "f16"):
        assert (np.abs(f64(ko) - want) <= rope_bound(k, spin, dtype, want))[kept].all()
    else:
        assert (f64(ko) == quantised(fmt, want))[kept].all()
    wq = turn(q)
    assert (np.abs(f64(q_out) - wq) <= rope_bound(q, spin, dtype, wq)).all()


def test_no_tokens(att):
    spin = att.Rope(64, sections=(16, 16))
    z = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    att.rope(z, torch.zeros(2, 0, dtype=torch.int32, device=DEV), spin, z)


@pytest.mark.parametrize("T", [1, 33])
@pytest.mark.parametrize("weave", [False, True])
def test_the_same_position_on_every_axis(att, T, weave):
    """Text: one row of positions expanded to all axes turns as one axis does, alone and into a cache."""
    Hkv, D, page = 2, 64, 16
    kw = dict(base=1e4)
    spin, one = att.Rope(D, sections=(12, 10, 10), weave=weave, **kw), att.Rope(D, **kw)
    pos = i32(positions(1, T, T)[0])
    x = rows(T, 5, D, "bf16", 1)
    a, b = torch.zeros_like(x), torch.ones_like(x)
    att.rope(x, pos.expand(3, T), spin, a)
    att.rope(x, pos, one, b)
    assert torch.equal(a, b)
    pages = -(-T // page)
    table, at, seq = i32(np.arange(pages))[None], i32(np.arange(T)), i32(np.zeros(T))
    k, v = rows(T, Hkv, D, "bf16", 2), rows(T, Hkv, D, "bf16", 3)
    caches = [att.KvCache(att.FT_KV_NVFP4, Hkv, D, page, pages) for _ in range(2)]
    att.kv_append(caches[0], k, v, table, at, seq=seq, rope=spin, rope_pos=pos.expand(3, T), q=x, q_out=a)
    att.kv_append(caches[1], k, v, table, at, seq=seq, rope=one, rope_pos=pos, q=x, q_out=b)
    assert torch.equal(a, b)
    for n in ("k", "v", "k_scale", "v_scale", "k_block", "v_block"):
        assert torch.equal(getattr(caches[0], n), getattr(caches[1], n))
