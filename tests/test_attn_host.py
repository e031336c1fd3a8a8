"""The attention operators without a GPU: exported symbols, refusals decided on
the host, rotary frequencies, and the kernels' index arithmetic compiled for
the host."""

import ctypes
import math
import os
import re
import subprocess

import numpy as np
import pytest
import torch

from conftest import ROOT

HEADER = os.path.join(ROOT, "include", "ft_attn.h")
CSRC = os.path.join(ROOT, "quantized_expert_ffn_router_gb300", "csrc")


@pytest.fixture(scope="module")
def att():
    from quantized_expert_ffn_router_gb300 import build as b

    b.build()
    from quantized_expert_ffn_router_gb300 import attention

    attention._bind()
    return attention


def test_every_declared_symbol_is_bound(att):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(ft_\w+)\s*\(", text))
    assert names == set(att._SIGS)


def test_row_bytes(att):
    assert att.kv_row_bytes(att.FT_KV_BF16, 128) == 256
    assert att.kv_row_bytes(att.FT_KV_F16, 80) == 160
    assert att.kv_row_bytes(att.FT_KV_E4M3, 128) == 128
    assert att.kv_row_bytes(att.FT_KV_NVFP4, 96) == 48
    for fmt, D in ((0, 8), (0, 100), (2, 272), (3, 80), (4, 128), (-1, 128)):
        assert att.kv_row_bytes(fmt, D) == 0


@pytest.mark.parametrize("scaling,args", [(0, {}), (1, dict(factor=4.0)), (2, dict(factor=4.0)),
                                          (3, dict(factor=8.0, low=1.0, high=4.0, orig_len=8192)),
                                          (4, dict(factor=16.0, low=1.0, high=32.0, orig_len=4096))])
@pytest.mark.parametrize("rot,base", [(128, 1e4), (64, 5e5), (20, 1e6), (4, 2.0)])
def test_rope_frequencies(att, scaling, args, rot, base):
    got = att.Rope(rot, base=base, scaling=scaling, device="cpu", **args).freqs.numpy()
    fac, low, high, n = (args.get(k, 0) for k in ("factor", "low", "high", "orig_len"))
    for i in range(rot // 2):
        b = base * fac ** (rot / (rot - 2)) if scaling == 2 else base
        f = b ** (-2 * i / rot)
        if scaling == 1:
            f /= fac
        if scaling == 3:
            g = min(max((n * f / (2 * math.pi) - low) / (high - low), 0), 1)
            f = g * f + (1 - g) * f / fac
        if scaling == 4:
            ix = lambda t: rot * math.log(n / (t * 2 * math.pi)) / (2 * math.log(base))
            a, z = max(math.floor(ix(high)), 0), min(math.ceil(ix(low)), rot - 1)
            g = 1 - min(max((i - a) / max(z - a, 1e-3), 0), 1)
            f = g * f + (1 - g) * f / fac
        # half a unit of the fixed point; pow and log of two runtimes agree to a few units of 2^-53
        assert abs(int(got[i]) * 2.0 ** -64 - f / (2 * math.pi)) <= 2.0 ** -65 + 2.0 ** -49 * f


def test_rope_refusals(att):
    for bad in (dict(rot_dim=3), dict(rot_dim=0), dict(rot_dim=64, base=0.5), dict(rot_dim=64, scaling=7),
                dict(rot_dim=64, scaling=1, factor=0.5), dict(rot_dim=64, scaling=3, low=4.0, high=1.0, factor=2.0),
                dict(rot_dim=64, scaling=4, orig_len=0, factor=2.0), dict(rot_dim=2, scaling=2, factor=2.0)):
        with pytest.raises(Exception) as e:
            att.Rope(device="cpu", **bad)
        assert getattr(e.value, "status", None) == 1


def _cache(att, fmt=0, Hkv=2, D=64, page=16, pages=4):
    return att.KvCache(fmt, Hkv, D, page, pages, device="cpu")


def _args(att, T=2, heads=4, D=64, dtype=torch.bfloat16):
    z = dict(dtype=dtype)
    return dict(q=torch.zeros(T, heads, D, **z), k=torch.zeros(T, 2, D, **z), v=torch.zeros(T, 2, D, **z),
                pages=torch.zeros(T, 3, dtype=torch.int32), pos=torch.zeros(T, dtype=torch.int32),
                out=torch.zeros(T, heads, D, **z), ws=torch.zeros(1 << 24, dtype=torch.uint8))


def refused(att, status, call, *a, **kw):
    with pytest.raises(Exception) as e:
        call(*a, stream=0, **kw)
    assert getattr(e.value, "status", None) == status, e.value


def test_attention_refusals(att):
    c, x = _cache(att), _args(att)
    f = lambda status=1, cache=c, **kw: refused(att, status, att.attn_decode, cache, *(
        kw.pop(n, x[n]) for n in ("q", "pages", "pos", "out", "ws")), **kw)
    f(q=torch.zeros(2, 3, 64, dtype=torch.bfloat16), out=torch.zeros(2, 3, 64, dtype=torch.bfloat16))  # 3 over 2 heads
    f(q=x["q"].half(), out=x["out"].half())          # a bf16 cache takes bf16 queries
    f(q=x["q"].float(), out=x["out"].float())        # no fp32 queries
    f(out=x["out"].half())                           # an output of another 16-bit type
    f(ws=x["ws"][:100])                              # workspace too small
    f(window=-1)
    f(scale=math.inf)
    f(pos=x["pos"].long())
    f(pages=x["pages"].long())
    f(pages=x["pages"][:1])                          # fewer sequences than rows
    f(q=torch.zeros(2, 4, 65, dtype=torch.bfloat16)[:, :, 1:])  # base and strides off 16 bytes
    f(q=torch.zeros(64, 4, 2, dtype=torch.bfloat16).permute(2, 1, 0))  # channels not contiguous
    f(lse=torch.zeros(2, 4, dtype=torch.float64))
    assert att.attn_decode_workspace(1, 3, 2, 64) == 0 and att.attn_decode_workspace(70000, 4, 2, 64) == 0


def test_cache_refusals(att):
    x = _args(att)
    go = lambda status, cache, **kw: refused(att, status, att.kv_append, cache, kw.get("k", x["k"]), kw.get("v", x["v"]),
                                             x["pages"], x["pos"], **{a: b for a, b in kw.items() if a not in "kv"})
    c = _cache(att)
    go(1, c, k=x["k"].half(), v=x["v"].half())
    go(1, c, k=x["k"].float(), v=x["v"].float())
    go(1, c, v=x["v"].half())
    go(1, c, q=x["q"])                    # q without a rotation
    go(1, c, q=x["q"], q_out=x["q"])
    go(1, c, rope=att.Rope(96, device="cpu"))  # more channels than the head has
    go(1, c, k=x["k"][:, :1], v=x["v"][:, :1])
    c = _cache(att)
    c.desc.page_stride = 1 << 31
    go(2, c)                              # rows beyond 2^32
    c = _cache(att)
    c.desc.D = 72
    go(2, c, k=torch.zeros(2, 2, 64, dtype=torch.bfloat16))
    c = _cache(att, att.FT_KV_NVFP4)
    c.desc.k_block = None
    go(1, c)
    c = _cache(att, att.FT_KV_E4M3)
    c.desc.v_scale = None
    go(1, c)
    c = _cache(att)
    c.desc.k = 8
    go(1, c)
    bad = torch.zeros(4, 2, 16, 128)
    for kw in (dict(k=bad, v=bad), dict(k=bad.bfloat16(), v=bad.bfloat16()[..., ::2])):
        with pytest.raises(Exception):
            att.KvCache.over(att.FT_KV_BF16, 128, **kw)
    # a call of no tokens does nothing
    att.kv_append(_cache(att), x["k"][:0], x["v"][:0], x["pages"], x["pos"][:0], stream=0)
    refused(att, 1, att.kv_gather, _cache(att), x["pages"], x["pos"], None, None)
    refused(att, 1, att.kv_gather, _cache(att), x["pages"], x["pos"], x["k"], x["v"].double())
    refused(att, 1, att.rope, x["q"], x["pos"], att.Rope(96, device="cpu"), x["out"])
    refused(att, 1, att.rope, x["q"], x["pos"], att.Rope(64, device="cpu"), x["out"].half())


# ------------------------------------------------- the kernels' index arithmetic
@pytest.fixture(scope="module")
def index(tmp_path_factory):
    d = tmp_path_factory.mktemp("index")
    src = d / "index.cpp"
    src.write_text("""
#include "ft_kv_index.h"
using namespace ft;
extern "C" {
unsigned div_(unsigned n, unsigned d) { return fast_div(n, make_fast_div(d)); }
long wrong(unsigned d) {  // quotients off by one show next to multiples of d
  const FastDiv f = make_fast_div(d);
  long bad = 0;
  for (unsigned long k = 0; k * d < (1ul << 31); k += 1 + (k >> 9))
    for (long o = -1; o <= 1; ++o) {
      const long n = (long)(k * d) + o;
      if (n >= 0 && n < (1l << 31)) bad += fast_div((unsigned)n, f) != (unsigned)n / d;
    }
  return bad + (fast_div(0x7fffffffu, f) != 0x7fffffffu / d);
}
unsigned row(int page, unsigned slot, unsigned pages, unsigned ps, unsigned ss) {
  KvIndex x{16, make_fast_div(16), pages, ps, 0, ss};
  return kv_row(x, page, slot);
}
void span(int len, int window, long most, int tile, int* out) {
  const RowSpan r = row_span(len, window, most, tile);
  out[0] = r.begin, out[1] = r.first, out[2] = r.len, out[3] = r.tiles;
}
long share(long total, long workers) { return split_share(total, workers); }
int numbers(int tiles, int lead, int units) { return row_numbers(tiles, lead, units); }
void part(int at, int left, int tiles, int lead, int* out) {
  const UnitPart p = unit_part(at, left, tiles, lead);
  out[0] = p.unit, out[1] = p.used, out[2] = p.tile0, out[3] = p.tiles, out[4] = p.rest;
}
}
""")
    so = d / "index.so"
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    lib.wrong.restype = lib.share.restype = ctypes.c_long
    lib.row.restype = lib.div_.restype = ctypes.c_uint32
    lib.share.argtypes = [ctypes.c_long] * 2
    lib.span.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_long, ctypes.c_int, ctypes.c_void_p]
    return lib


@pytest.mark.parametrize("d", [1, 2, 3, 5, 7, 16, 24, 48, 64, 100, 127, 641, 4096, 65537, (1 << 30) + 1, (1 << 31) - 1])
def test_fast_division_is_exact(index, d):
    assert index.wrong(d) == 0


def test_rows_of_bad_pages(index):
    no = 0xFFFFFFFF
    assert index.row(3, 2, 10, 100, 5) == 310
    assert index.row(-1, 0, 10, 100, 5) == no
    assert index.row(10, 0, 10, 100, 5) == no
    assert index.row(2 ** 31 - 1, 0, 10, 100, 5) == no


@pytest.mark.parametrize("tile", [64, 128, 256])
def test_spans_and_shares_cover_every_token_once(index, tile):
    r = np.random.default_rng(tile)
    out = (ctypes.c_int * 4)()
    for _ in range(300):
        T, units = int(r.integers(1, 40)), int(r.integers(1, 9))
        lens = [int(x) for x in r.integers(-3, 2000, T)]
        window, most = int(r.choice([0, 0, 1, 17, 500])), int(r.choice([1500, 10 ** 9]))
        spans = []
        for n in lens:
            index.span(n, window, most, tile, out)
            begin, first, stop, tiles = out
            n = max(0, min(n, most))
            assert stop == n and first == (max(0, n - window) if window else 0)
            assert begin % 16 == 0 and begin <= first < begin + 16
            assert (tiles - 1) * tile < stop - begin <= tiles * tile or (stop == 0 and tiles == 0)
            spans.append(tiles)
        total = sum(spans) * units
        workers = int(r.choice([1, 7, 304, 1024]))
        share = index.share(total, workers)
        assert share >= 1 and share * workers >= total
    index.span(2 ** 31 - 1, 0, 2 ** 31 - 4096, tile, out)
    assert out[2] == 2 ** 31 - 4096 and out[3] > 0


@pytest.mark.parametrize("lead", [0, 1, 2, 5])
def test_unit_parts_cover_every_tile_once(index, lead):
    """Every worker's walk, as the kernel takes it: each tile of each unit once, in order; the worker that holds a
    unit's first tile knows the last one that holds any, and those in between hold some."""
    r = np.random.default_rng(lead)
    out = (ctypes.c_int * 5)()
    for _ in range(200):
        T, units = int(r.integers(1, 12)), int(r.integers(1, 6))
        tiles = [int(x) for x in r.choice([0, 1, 2, 3, 40], T)]
        numbers = [index.numbers(n, lead, units) for n in tiles]
        assert numbers == [(n + lead) * units if n else 0 for n in tiles]
        total, workers = sum(numbers), int(r.choice([1, 3, 16, 64]))
        share = index.share(total, workers)
        held = {}
        for c in range(workers):
            at, left = c * share, min(share, total - c * share)
            t = 0
            while left > 0:
                while at >= numbers[t]:
                    at -= numbers[t]
                    t += 1
                index.part(at, left, tiles[t], lead, out)
                unit, used, tile0, n, rest = out
                assert 0 < used <= left and 0 <= unit < units
                at += used
                left -= used
                if n:
                    held.setdefault((t, unit), []).append((c, tile0, n, rest))
        for t in range(T):
            for u in range(units):
                parts = held.get((t, u), [])
                assert bool(parts) == bool(tiles[t])
                done = 0
                for i, (c, tile0, n, rest) in enumerate(parts):
                    assert tile0 == done and rest == tiles[t] - tile0 - n
                    done += n
                    assert c == parts[0][0] + i
                assert done == tiles[t]
                if parts:
                    c, _, n, rest = parts[0]
                    assert parts[-1][0] == c + -(-rest // share)
