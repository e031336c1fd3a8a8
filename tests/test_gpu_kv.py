"""Rotary positions and the paged key-value cache's rows, written and read
back, against their definitions in 64 bits.  Quantised rows have to be the
definition's exactly."""

import math

import numpy as np
import pytest
import torch

from attn_helpers import DT, FMT, Cache, f64, quantised, random_table, rotated

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def att(cuda_lib):
    from quantized_expert_ffn_router_gb300 import attention

    return attention


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def rows(T, h, D, dtype, seed, offset=8):
    """[T, h, D] inside wider rows, channels and tokens of uneven size."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, h, D, generator=g) * torch.exp(torch.randn(1, h, D, generator=g)) * torch.exp(
        2 * torch.randn(T, h, 1, generator=g))
    wide = torch.zeros(T, offset + h * D, dtype=DT[dtype], device=DEV)
    t = wide[:, offset:].view(T, h, D) if T > 1 else wide[:, offset:].reshape(T, h, D)
    t.copy_(x.clamp(-2e4, 2e4).to(DT[dtype]))  # inside f16's range, rotated too
    return t


def radians(spin):
    return spin.freqs.cpu().numpy().astype(np.float64) * (2 * math.pi / 2.0 ** 64)


def rope_bound(x, spin, dtype, want):
    """The output's rounding, and 2^-21 of the pair's size for angle, cosine, products and sum in fp32."""
    half = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}[dtype]
    pair = np.abs(f64(x)).max(-1, keepdims=True) * 2 * abs(spin.mscale)
    return half * np.abs(want) + pair * 2.0 ** -21 + (2.0 ** -25 if dtype == "f16" else 0)


@pytest.mark.parametrize("D,rot", [(128, 128), (128, 64), (64, 64), (256, 64), (80, 80), (96, 32), (72, 24), (8, 8),
                                   (128, 20), (128, 2), (256, 254), (24, 16)])
@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_rope(att, D, rot, layout, dtype):
    T, h = 5, 3
    x = rows(T, h, D, dtype, D + rot)
    spin = att.Rope(rot, base=5e5, interleaved=layout == "pairs", mscale=1.25)
    pos = [0, 1, 77, 123456, 2 ** 31 - 1]
    out = torch.full((T, h, D), float("nan"), dtype=DT[dtype], device=DEV)
    att.rope(x, i32(pos), spin, out)
    want = rotated(f64(x), pos, radians(spin), layout, 1.25)
    assert (np.abs(f64(out) - want) <= rope_bound(x, spin, dtype, want)).all()
    assert torch.equal(out[..., rot:], x[..., rot:])
    att.rope(x, i32(pos), spin, x)  # in place
    assert torch.equal(x, out)


@pytest.mark.parametrize("T,h", [(1, 1), (1, 64), (3, 17), (700, 40), (0, 4)])
def test_rope_sizes_and_back(att, T, h):
    x = rows(T, h, 128, "f16", 3)
    spin = att.Rope(128, base=1e4, scaling=att.FT_ROPE_PARTS_BY_TURNS, factor=8.0)
    pos = torch.arange(T, dtype=torch.int32, device=DEV) * 997
    out, back = torch.zeros_like(x), torch.zeros_like(x)
    att.rope(x, pos, spin, out)
    if T:
        want = rotated(f64(x), pos.cpu().numpy(), radians(spin), "half", 1.0)
        assert (np.abs(f64(out) - want) <= rope_bound(x, spin, "f16", want)).all()
    att.rope(out, -pos, spin, back)  # negative positions turn back
    assert (np.abs(f64(back) - f64(x)) <= 4 * rope_bound(x, spin, "f16", f64(x)) + np.abs(f64(x)).max(
        initial=0.0, axis=-1, keepdims=True) * 2.0 ** -10).all()


SHAPES = [  # T, Hkv, D, page, rot
    (1, 1, 64, 16, 64), (9, 2, 128, 16, 128), (33, 3, 128, 24, 64), (70, 8, 64, 1, 32), (20, 2, 256, 64, 64),
    (17, 5, 96, 48, 96), (300, 4, 128, 32, 128), (8, 2, 192, 8, 48), (6, 2, 32, 16, 16)]


@pytest.mark.parametrize("T,Hkv,D,page,rot", SHAPES)
@pytest.mark.parametrize("fmt,dtype", [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "bf16"), ("e4m3", "f16"),
                                       ("nvfp4", "bf16"), ("nvfp4", "f16")])
@pytest.mark.parametrize("layout", ["none", "half", "pairs"])
def test_append_and_gather(att, T, Hkv, D, page, rot, fmt, dtype, layout):
    n = [T - T // 3, T // 3] if T > 2 else [T]
    first = [5, 0][:len(n)]
    lens = [a + b for a, b in zip(first, n)]
    pages = sum(-(-x // page) for x in lens) + 1
    table = i32(random_table(lens, page, pages, T))
    seq = np.repeat(np.arange(len(n)), n)
    pos = np.concatenate([np.arange(a, a + b) for a, b in zip(first, n)])
    order = np.random.default_rng(T).permutation(T)
    seq, pos = seq[order], pos[order]
    cache = att.KvCache(FMT[fmt], Hkv, D, page, pages)
    k, v, q = (rows(T, h, D, dtype, s) for h, s in ((Hkv, 1), (Hkv, 2), (2 * Hkv, 3)))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    spin = None if layout == "none" else att.Rope(rot, base=1e4, interleaved=layout == "pairs", mscale=1.125)
    kw, far = {}, pos + 54321
    if spin:
        q_out = torch.zeros(T, 2 * Hkv, D, dtype=DT[dtype], device=DEV)
        kw = dict(rope=spin, rope_pos=i32(far), q=q, q_out=q_out)
    att.kv_append(cache, k, v, table, i32(pos), seq=i32(seq), dev_status=status, **kw)
    ko, vo = (torch.full((T, Hkv, D), float("nan"), device=DEV) for _ in "kv")
    att.kv_gather(cache, table, i32(pos), ko, vo, seq=i32(seq), dev_status=status)
    assert int(status.item()) == 0
    assert (f64(vo) == quantised(fmt, f64(v))).all()
    want = f64(k) if not spin else rotated(f64(k), far, radians(spin), layout, 1.125)
    if fmt in ("bf16", "f16") and spin:
        assert (np.abs(f64(ko) - want) <= rope_bound(k, spin, dtype, want)).all()
    else:
        assert (f64(ko) == quantised(fmt, want)).all()
    if spin:
        wq = rotated(f64(q), far, radians(spin), layout, 1.125)
        assert (np.abs(f64(q_out) - wq) <= rope_bound(q, spin, dtype, wq)).all()
    # nothing else was written
    untouched = att.KvCache(FMT[fmt], Hkv, D, page, pages)
    p, s = table[i32(seq).long(), i32(pos // page).long()].long(), i32(pos % page).long()
    for name in ("k", "v", "k_scale", "v_scale", "k_block", "v_block"):
        a, b = getattr(cache, name), getattr(untouched, name)
        if a is not None:
            a = a.view(torch.uint8) if a.dtype.itemsize == 1 else a
            b = b.view(torch.uint8) if b.dtype.itemsize == 1 else b
            a[p, :, s] = b[p, :, s]
            assert torch.equal(a, b), name


@pytest.mark.parametrize("fmt", ["bf16", "f16", "e4m3", "nvfp4"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("order", ["phsd", "pshd", "hpsd"])
def test_gather_types_and_orders(att, fmt, dtype, order):
    cache = Cache(fmt, 3, 64, 8, 6, 1, order)
    table = random_table([20, 9], 8, 6, 1)
    seq, pos = np.array([0, 1, 0, 0, 1, 0]), np.array([19, 0, 7, 8, 8, -1])
    ko, vo = (torch.full((6, 3, 64), float("nan"), dtype=DT[dtype], device=DEV) for _ in "kv")
    att.kv_gather(cache.desc, i32(table), i32(pos), ko, vo, seq=i32(seq))
    for name, got in (("k", ko), ("v", vo)):
        want = cache.values[name][table[seq, pos // 8], :, pos % 8]
        want[pos < 0] = 0
        assert torch.equal(got.cpu(), torch.from_numpy(want).to(DT[dtype]))
    only = torch.zeros_like(vo)
    att.kv_gather(cache.desc, i32(table), i32(pos), None, only, seq=i32(seq))
    assert torch.equal(only, vo)


def test_special_values(att):
    """Zeros, subnormals, infinities, NaN, the ends of bf16's range and ties of every kind."""
    D = 64
    g = torch.Generator().manual_seed(0)
    x = torch.zeros(12, 1, D)
    x[1] = 1e-30
    x[2] = torch.randn(D, generator=g) * 1e-39
    x[3, 0, 5], x[3, 0, 6], x[3, 0, 20] = math.inf, 3.0, -math.inf
    x[4] = math.inf
    x[5, 0, 17], x[5, 0, 3] = math.nan, 2.0
    x[6] = torch.randn(D, generator=g) * 1e38
    x[7] = -3.3895e38
    x[8] = torch.arange(D) * 0.25  # ties of both formats
    x[9] = 448.0 * torch.linspace(-1, 1, D)
    x[10] = torch.tensor([1.0, 1.0625, 1.1875, 17.0] * 16)
    x[11, 0, 0] = 450.0
    x = x.to(torch.bfloat16).to(DEV)
    for fmt in ("e4m3", "nvfp4"):
        cache = att.KvCache(FMT[fmt], 1, D, 16, 1)
        pages, pos = torch.zeros(12, 1, dtype=torch.int32, device=DEV), torch.arange(12, dtype=torch.int32, device=DEV)
        att.kv_append(cache, x, -x, pages, pos)
        ko, vo = torch.zeros(12, 1, D, device=DEV), torch.zeros(12, 1, D, device=DEV)
        att.kv_gather(cache, pages, pos, ko, vo)
        with np.errstate(over="ignore"):
            want = quantised(fmt, f64(x)).astype(np.float32)  # the outputs' type: 256 * 2^120 is beyond it
        np.testing.assert_array_equal(f64(ko), want)
        np.testing.assert_array_equal(f64(vo), -want)


def test_padding_and_bad_places(att):
    """Padding tokens are not written; bad pages and sequences are recorded and skipped; q is rotated for all."""
    D, page = 64, 8
    cache = att.KvCache(att.FT_KV_BF16, 2, D, page, 4)
    k, v, q = rows(6, 2, D, "bf16", 1), rows(6, 2, D, "bf16", 2), rows(6, 4, D, "bf16", 3)
    table = i32([[0, 1], [2, 9], [-1, 3]])
    spin = att.Rope(64)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.zeros(6, 4, D, dtype=torch.bfloat16, device=DEV)
    seq, pos = [0, 0, 1, 2, 3, 2], [3, -1, 8, 7, 0, 16]
    att.kv_append(cache, k, v, table, i32(pos), seq=i32(seq), rope=spin, rope_pos=i32([1] * 6), q=q, q_out=out,
                  dev_status=status)
    assert int(status.item()) == 5
    assert torch.equal(cache.v[0, :, 3], v[0])
    cache.v[0, :, 3] = 0
    assert not cache.v.any()
    want = rotated(f64(q), [1] * 6, radians(spin), "half", 1.0)
    assert (np.abs(f64(out) - want) <= rope_bound(q, spin, "bf16", want)).all()
    status.zero_()
    got = torch.ones(6, 2, D, dtype=torch.bfloat16, device=DEV)
    att.kv_gather(cache, table, i32(pos), got, None, seq=i32(seq), dev_status=status)
    assert int(status.item()) == 5 and not got[1:].any()
    status.zero_()
    att.kv_append(cache, k[:1], v[:1], table, i32([-1]), dev_status=status)
    assert int(status.item()) == 0


def test_append_on_another_stream_in_a_graph(att):
    D, page, T = 128, 16, 3
    cache = att.KvCache(att.FT_KV_E4M3, 2, D, page, 6)
    k, v = rows(T, 2, D, "bf16", 1), rows(T, 2, D, "bf16", 2)
    table = i32([[0, 1], [2, 3], [4, 5]])
    pos = torch.zeros(T, dtype=torch.int32, device=DEV)
    ko, vo = torch.zeros(T, 2, D, device=DEV), torch.zeros(T, 2, D, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        att.kv_append(cache, k, v, table, pos)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            att.kv_append(cache, k, v, table, pos)
            att.kv_gather(cache, table, pos, ko, vo)
        for p in ([0, 1, 2], [31, 30, 15]):
            pos.copy_(torch.tensor(p, dtype=torch.int32))
            g.replay()
            side.synchronize()
            assert (f64(ko) == quantised("e4m3", f64(k))).all()
            assert (f64(vo) == quantised("e4m3", f64(v))).all()


@pytest.mark.parametrize("T,Hkv,D,page,rot", [(2501, 4, 128, 32, 128), (1300, 12, 256, 48, 64), (1000, 20, 64, 16, 64),
                                              (6000, 1, 128, 64, 96)])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "nvfp4"])
@pytest.mark.parametrize("layout", ["half", "pairs"])
def test_append_many_tokens(att, T, Hkv, D, page, rot, fmt, layout):
    """Several tokens, and several turns of a token's rows, for each block of threads."""
    test_append_and_gather(att, T, Hkv, D, page, rot, fmt, "bf16", layout)


@pytest.mark.parametrize("T,h,D,rot,layout", [(4099, 40, 128, 64, "pairs"), (5001, 40, 128, 128, "half"),
                                              (3001, 7, 256, 100, "half"), (40000, 2, 64, 64, "half")])
def test_rope_many_tokens_in_place(att, T, h, D, rot, layout):
    x = rows(T, h, D, "bf16", 5)
    spin = att.Rope(rot, base=1e4, interleaved=layout == "pairs")
    pos = torch.randint(0, 1 << 20, (T,), dtype=torch.int32, generator=torch.Generator().manual_seed(1)).to(DEV)
    out = torch.full((T, h, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    att.rope(x, pos, spin, out)
    want = rotated(f64(x), pos.cpu().numpy(), radians(spin), layout, 1.0)
    assert (np.abs(f64(out) - want) <= rope_bound(x, spin, "bf16", want)).all()
    same = x.clone()
    att.rope(same, pos, spin, same)
    assert torch.equal(same, out)


@pytest.mark.parametrize("layout,rot", [("half", 64), ("half", 32), ("half", 24), ("pairs", 64)])
@pytest.mark.parametrize("fmt", ["e4m3", "nvfp4"])
def test_special_values_of_rotated_keys(att, fmt, layout, rot):
    """Zeros, subnormals, infinities, NaN and ties in keys that are rotated to position 0 and to others."""
    D, g = 64, torch.Generator().manual_seed(0)
    x = torch.randn(12, 2, D, generator=g)
    x[1] = 0.0
    x[2] = -0.0
    x[3] *= 1e-39
    x[4, 0, 5], x[4, 1, 40] = math.inf, -math.inf
    x[5, 0, 17], x[5, 1, 63] = math.nan, math.nan
    x[6, :, :16] *= 1e-5  # a block scale of zero
    x[7] = torch.arange(D) * 0.25
    x[8] = 448.0 * torch.linspace(-1, 1, D)
    x[9, :, 0] = 450.0
    x[10] *= 1e30
    x = x.to(torch.bfloat16).to(DEV)
    spin = att.Rope(rot, base=1e4, interleaved=layout == "pairs")
    cache = att.KvCache(FMT[fmt], 2, D, 16, 1)
    pages, pos = torch.zeros(12, 1, dtype=torch.int32, device=DEV), torch.arange(12, dtype=torch.int32, device=DEV)
    for at in (0, 3, 70001):
        far = torch.full_like(pos, at)
        att.kv_append(cache, x, -x, pages, pos, rope=spin, rope_pos=far)
        ko, vo = torch.zeros(12, 2, D, device=DEV), torch.zeros(12, 2, D, device=DEV)
        att.kv_gather(cache, pages, pos, ko, vo)
        with np.errstate(invalid="ignore"):
            want = quantised(fmt, rotated(f64(x), far.cpu().numpy(), radians(spin), layout, 1.0))
        np.testing.assert_array_equal(f64(ko), want.astype(np.float32))
        np.testing.assert_array_equal(f64(vo), quantised(fmt, -f64(x)).astype(np.float32))
