"""ft_attn_decode against attention in 64 bits: formats, head layouts, lengths
around every tile border, pages that end inside a tile, windows, bad pages,
empty rows, values in masked places, streams and graphs."""

import numpy as np
import pytest
import torch

from attn_helpers import DT, Cache, attention, attention_tolerance, f64, random_table

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def att(cuda_lib):
    from quantized_expert_ffn_router_gb300 import attention

    return attention


def queries(T, Hq, D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    wide = torch.randn(T, Hq * D + 16, generator=g).to(DT[dtype]).to(DEV)
    return wide[:, 16:].view(T, Hq, D) if T > 1 else wide[:, 16:].reshape(T, Hq, D)


def check(att, fmt, dtype, out_dtype, D, Hkv, G, page, lens, window=0, seed=0, order="phsd", table=None, cache=None,
          seq=None, width=None, scale=None, status_want=0, weight_step=None):
    T, Hq = len(lens), Hkv * G
    n_pages = sum(-(-int(n) // page) for n in lens) + 2 if table is None else None
    if cache is None:
        cache = Cache(fmt, Hkv, D, page, n_pages, seed, order)
    if table is None:
        table = random_table(lens, page, n_pages, seed, width)
    q = queries(T, Hq, D, dtype, seed + 1)
    out = torch.full((T, Hq, D), float("nan"), dtype=DT[out_dtype], device=DEV)
    lse = torch.full((T, Hq), float("nan"), device=DEV)
    ws = torch.full((att.attn_decode_workspace(T, Hq, Hkv, D),), 0xFF, dtype=torch.uint8, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    i32 = lambda a: None if a is None else torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)
    scale = D ** -0.5 if scale is None else scale
    att.attn_decode(cache.desc, q, i32(table), i32(lens), out, ws, seq=i32(seq), scale=scale, window=window, lse=lse,
                    dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == status_want
    scale32 = float(np.float32(scale))
    want, want_lse, parts = attention(cache, f64(q), table, lens, page, scale32, window, seq)
    tol, tol_lse = attention_tolerance(fmt, out_dtype, D, want, want_lse, parts, weight_step)
    got, got_lse = f64(out), f64(lse)
    assert np.isfinite(got).all()
    bad = np.abs(got - want) > tol
    assert not bad.any(), (np.argwhere(bad)[:5], np.abs(got - want).max(), tol[bad][:3])
    empty = ~np.isfinite(want_lse)
    assert (got_lse[empty] == -np.inf).all() and (got[empty] == 0).all()
    assert (np.abs(got_lse - want_lse)[~empty] <= tol_lse[~empty]).all()


BORDERS = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 255, 257, 300]


@pytest.mark.parametrize("fmt,dtype", [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "bf16"), ("e4m3", "f16"),
                                       ("nvfp4", "bf16")])
@pytest.mark.parametrize("D", [64, 128, 192, 256])
def test_lengths_at_tile_borders(att, fmt, dtype, D):
    check(att, fmt, dtype, dtype, D, 2, 8, 16, BORDERS, seed=D)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "nvfp4"])
@pytest.mark.parametrize("Hkv,G", [(3, 1), (5, 2), (1, 3), (2, 7), (2, 9), (1, 12), (4, 16), (1, 20), (1, 40), (1, 71)])
def test_groups_of_heads(att, fmt, Hkv, G):
    check(att, fmt, "bf16", "bf16", 128, Hkv, G, 32, [70, 1, 333], seed=G)


@pytest.mark.parametrize("fmt,G", [("bf16", 16), ("e4m3", 12), ("nvfp4", 33), ("f16", 9)])
@pytest.mark.parametrize("D", [64, 256])
def test_groups_at_other_head_sizes(att, fmt, G, D):
    check(att, fmt, "f16" if fmt == "f16" else "bf16", "f32", D, 2, G, 16, [257, 90], seed=G + D)


@pytest.mark.parametrize("fmt,D", [("bf16", 16), ("bf16", 80), ("f16", 112), ("bf16", 144), ("bf16", 208), ("e4m3", 16),
                                   ("e4m3", 80), ("e4m3", 176), ("e4m3", 240), ("nvfp4", 32), ("nvfp4", 96),
                                   ("nvfp4", 160), ("nvfp4", 224)])
def test_padded_head_sizes(att, fmt, D):
    check(att, fmt, "f16" if fmt == "f16" else "bf16", "f32", D, 2, 4, 8, [200, 37], seed=D)


@pytest.mark.parametrize("page", [1, 3, 8, 24, 48, 100, 256])
@pytest.mark.parametrize("fmt", ["bf16", "nvfp4"])
def test_page_sizes(att, fmt, page):
    check(att, fmt, "bf16", "bf16", 128, 2, 4, page, [1, 99, 300, 301], seed=page)


@pytest.mark.parametrize("window", [1, 5, 16, 17, 100, 1000])
def test_windows(att, window):
    check(att, "e4m3", "bf16", "bf16", 128, 2, 8, 24, [0, 1, 4, 16, 99, 117, 500, 777], window=window, seed=window)


@pytest.mark.parametrize("fmt", ["bf16", "f16", "e4m3", "nvfp4"])
@pytest.mark.parametrize("out", ["same", "f32"])
def test_long_rows_are_split_and_joined(att, fmt, out):
    dtype = "f16" if fmt == "f16" else "bf16"
    check(att, fmt, dtype, dtype if out == "same" else "f32", 128, 1, 8, 64, [30011, 3], seed=7)


def test_many_uneven_rows(att):
    r = np.random.default_rng(3)
    lens = [int(n) for n in np.exp(r.uniform(0, np.log(400), 150))]
    lens[40:75] = [0] * 35
    check(att, "bf16", "bf16", "bf16", 64, 2, 4, 16, lens, seed=11)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_more_units_than_workers(att, fmt):
    """More (row, key head) units than the grid has CTAs: shares hold many units, and end inside one."""
    r = np.random.default_rng(5)
    lens = [int(n) for n in np.exp(r.uniform(0, np.log(90), 700))]
    lens[10:20], lens[300], lens[699] = [0] * 10, 2500, 0
    check(att, fmt, "bf16", "bf16", 64, 3, 2, 16, lens, seed=12)


@pytest.mark.parametrize("order", ["pshd", "hpsd", "sphd"])
@pytest.mark.parametrize("fmt", ["f16", "e4m3", "nvfp4"])
def test_cache_orders(att, fmt, order):
    check(att, fmt, "f16", "f16", 128, 3, 2, 16, [100, 45], seed=5, order=order)


def test_rows_share_sequences(att):
    """Several rows of one sequence (its last tokens, as a draft is verified), and a wider table than needed."""
    page, n = 16, 7
    cache = Cache("bf16", 2, 64, page, 40, 9)
    table = random_table([100, 200], page, 40, 9, width=20)
    lens, seq = [200, 199, 198, 100, 50], [1, 1, 1, 0, 0]
    check(att, "bf16", "bf16", "bf16", 64, 2, 4, page, lens, table=table, cache=cache, seq=seq)


def test_bad_pages_and_sequences_are_skipped(att):
    page = 16
    cache = Cache("e4m3", 2, 128, page, 40, 9)
    table = random_table([100, 200, 60], page, 40, 9)
    table[0, 2], table[1, 0], table[1, 11] = 40, -7, 2 ** 30
    check(att, "e4m3", "bf16", "bf16", 128, 2, 4, page, [100, 200, 60, 60], table=table, cache=cache,
          seq=[0, 1, 2, 3], status_want=5)
    check(att, "e4m3", "bf16", "bf16", 128, 2, 4, page, [60, 60], table=table, cache=cache, seq=[2, -1], status_want=5)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "nvfp4"])
def test_values_in_masked_places(att, fmt):
    """NaN and infinities in slots past a row's length or before its window do not reach it."""
    page, D, lens = 16, 128, [33, 100]
    cache = Cache(fmt, 2, D, page, 12, 2)
    table = random_table(lens, page, 12, 2)
    used = np.zeros((12, page), bool)
    for t, n in enumerate(lens):
        for j in range(max(0, n - 60), n):
            used[table[t, j // page], j % page] = True
    free = torch.from_numpy(~used).to(DEV)
    for n, a in cache.arrays.items():
        m = free[:, None, :].expand(12, 2, page)
        if n in ("k", "v") and fmt == "bf16":
            a[m] = float("nan") if n == "k" else float("inf")
        else:
            a.view(torch.uint8)[m] = 0x7F if n in ("k", "v") or n.endswith("block") else 0xFF
    check(att, fmt, "bf16", "bf16", D, 2, 4, page, lens, window=60, table=table, cache=cache)


def test_nan_and_infinity_that_count_show(att):
    page, D = 16, 64
    cache = Cache("bf16", 1, D, page, 4, 2)
    table = random_table([40], page, 4, 2)
    cache.arrays["v"][int(table[0, 1]), 0, 3, 5] = float("nan")
    q = queries(1, 2, D, "bf16", 1)
    out = torch.zeros(1, 2, D, dtype=torch.bfloat16, device=DEV)
    ws = torch.zeros(att.attn_decode_workspace(1, 2, 1, D), dtype=torch.uint8, device=DEV)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)
    att.attn_decode(cache.desc, q, i32(table), i32([40]), out, ws)
    nan = torch.isnan(out)
    assert nan[:, :, 5].all() and int(nan.sum()) == 2
    cache.arrays["k"][int(table[0, 0]), 0, 0, :] = float("inf")
    att.attn_decode(cache.desc, q, i32(table), i32([40]), out, ws)
    assert torch.isnan(out).all()


@pytest.mark.parametrize("fmt", ["e4m3", "nvfp4"])
def test_scales_far_apart(att, fmt):
    """Row exponents from 2^-60 to 2^40 in one row: the heavy rows decide, the light ones lose nothing of their own."""
    page, D = 16, 64
    cache = Cache(fmt, 1, D, page, 8, 4)
    r = np.random.default_rng(0)
    for lo, hi in ((67, 90), (100, 167)):
        e = torch.from_numpy(r.integers(lo, hi, (8, 1, page)).astype(np.uint8)).to(DEV)
        old = f64(cache.arrays["v_scale"])
        cache.arrays["v_scale"].copy_(e)
        cache.values["v"] = cache.values["v"] * 2.0 ** (f64(e) - old)[..., None]
        check(att, fmt, "bf16", "f32", D, 1, 4, page, [100], table=random_table([100], page, 8, 4), cache=cache)


@pytest.mark.parametrize("size", [1e-4, 1.0, 3e3])
def test_peaked_and_flat_scores(att, size):
    check(att, "bf16", "bf16", "bf16", 128, 1, 8, 16, [500, 2], seed=1, scale=0.088 * size if size < 100 else 4.0)
    check(att, "e4m3", "bf16", "bf16", 128, 1, 8, 16, [500, 2], seed=1, scale=0.088 * size if size < 100 else 2.0)


def test_rows_beyond_four_gigabytes(att):
    """Pages whose byte offsets pass 2^32."""
    page, D, pages = 16, 128, 3
    small = Cache("bf16", 1, D, page, pages, 8)
    far = (5 << 30) // 2 // (pages - 1)  # elements between pages
    far -= far % D
    for n in ("k", "v"):
        big = torch.empty(far * (pages - 1) + page * D, dtype=torch.bfloat16, device=DEV)
        t = big.as_strided((pages, 1, page, D), (far, page * D, D, 1))
        t.copy_(small.arrays[n])
        small.arrays[n] = t
    small.desc = att.KvCache.over(att.FT_KV_BF16, D, **small.arrays)
    check(att, "bf16", "bf16", "bf16", D, 1, 8, page, [45], table=random_table([45], page, pages, 8), cache=small)


def test_repeats_are_identical(att):
    page, lens = 64, [9000, 20, 4000]
    cache = Cache("bf16", 2, 128, page, 220, 1)
    table = torch.tensor(random_table(lens, page, 220, 1), device=DEV)
    q = queries(3, 16, 128, "bf16", 2)
    ws = torch.empty(att.attn_decode_workspace(3, 16, 2, 128), dtype=torch.uint8, device=DEV)
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    outs = []
    for _ in range(8):
        out = torch.empty(3, 16, 128, dtype=torch.bfloat16, device=DEV)
        att.attn_decode(cache.desc, q, table, n, out, ws)
        outs.append(out)
    assert all(torch.equal(outs[0], o) for o in outs[1:])


def test_a_captured_step_serves_other_lengths(att):
    """The lengths are read on the device: one graph, replayed after the cache has grown, on a stream of its own."""
    page, D, Hkv, G = 16, 128, 2, 4
    cache = Cache("f16", Hkv, D, page, 80, 1)
    table = random_table([600, 600], page, 80, 1)
    td = torch.tensor(table, device=DEV)
    lens = torch.tensor([5, 600], dtype=torch.int32, device=DEV)
    q = queries(2, Hkv * G, D, "f16", 4)
    out = torch.zeros(2, Hkv * G, D, dtype=torch.float16, device=DEV)
    ws = torch.zeros(att.attn_decode_workspace(2, Hkv * G, Hkv, D), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        att.attn_decode(cache.desc, q, td, lens, out, ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            att.attn_decode(cache.desc, q, td, lens, out, ws)
        for n in ([5, 600], [599, 1], [0, 17]):
            lens.copy_(torch.tensor(n, dtype=torch.int32))
            g.replay()
            side.synchronize()
            want, lse, parts = attention(cache, f64(q), table, n, page, float(np.float32(D ** -0.5)))
            tol, _ = attention_tolerance("f16", "f16", D, want, lse, parts)
            assert (np.abs(f64(out) - want) <= tol).all()


def test_differences_of_the_log_sum_are_the_output(att):
    """d lse / d q = scale * sum p k: with v = k, the output is the gradient of lse (central differences)."""
    page, D = 16, 64
    cache = Cache("bf16", 1, D, page, 8, 6)
    cache.arrays["v"].copy_(cache.arrays["k"])
    cache.values["v"] = cache.values["k"]
    table = torch.tensor(random_table([120], page, 8, 6), device=DEV)
    lens = torch.tensor([120], dtype=torch.int32, device=DEV)
    q = (queries(1, 1, D, "bf16", 3).float() * 0.5).to(torch.bfloat16)
    ws = torch.zeros(att.attn_decode_workspace(1, 1, 1, D), dtype=torch.uint8, device=DEV)

    def run(x):
        out, lse = torch.zeros(1, 1, D, device=DEV), torch.zeros(1, 1, device=DEV)
        att.attn_decode(cache.desc, x, table, lens, out, ws, scale=0.125, lse=lse)
        return out, float(lse)

    out, _ = run(q)
    for d in (0, 13, 63):
        h = 2.0 ** -4
        up, dn = q.clone(), q.clone()
        base = round(float(q[0, 0, d]) * 16) / 16  # so that base +- h are exact in bf16
        q2 = q.clone()
        q2[0, 0, d] = base
        up[0, 0, d], dn[0, 0, d] = base + h, base - h
        o2, _ = run(q2)
        slope = (run(up)[1] - run(dn)[1]) / (2 * h)
        # third-derivative term h^2/6 * (0.125 * |k|)^3 < 2^-8/6 * 0.13, fp32 lse 2^-20 / h
        assert abs(slope - 0.125 * float(o2[0, 0, d])) <= 2.0 ** -8 / 6 * 0.2 + 2.0 ** -15


def weight_step(fmt, out):
    """The largest relative error of a weight: half a step of its type (bf16 2^-8, f16 2^-11), squared where it is two
    terms (16-bit caches, and fp32 outputs)."""
    return 2.0 ** -16 if fmt == "bf16" else 2.0 ** -22 if fmt == "f16" or out == "f32" else 2.0 ** -11


@pytest.mark.parametrize("fmt,out", [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "bf16"), ("nvfp4", "f32")])
@pytest.mark.parametrize("D,Hkv,G", [(64, 3, 17), (64, 1, 64), (80, 1, 36), (96, 2, 20), (128, 1, 33), (128, 2, 48),
                                     (160, 1, 11), (192, 2, 16), (192, 1, 32), (256, 1, 24), (224, 2, 9)])
def test_heads_over_several_warps(att, fmt, out, D, Hkv, G):
    if fmt == "nvfp4" and D % 32:
        D += 16
    dtype = "f16" if fmt == "f16" else "bf16"
    kw = dict(seed=D + G, weight_step=weight_step(fmt, out))
    check(att, fmt, dtype, out, D, Hkv, G, 24, [0, 1, 15, 16, 17, 65, 0, 401, 1290], **kw)
    check(att, fmt, dtype, out, D, Hkv, G, 7, [5, 0, 700, 3, 99], window=61, **kw)


@pytest.mark.parametrize("fmt", ["bf16", "nvfp4"])
@pytest.mark.parametrize("G", [24, 64])
def test_many_rows_of_heads_over_several_warps(att, fmt, G):
    r = np.random.default_rng(4)
    lens = [int(n) for n in np.exp(r.uniform(0, np.log(400), 90))] + [9001]
    lens[40:60] = [0] * 20
    check(att, fmt, "bf16", "bf16", 128, 2, G, 16, lens, seed=12, weight_step=weight_step(fmt, "bf16"))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_bad_pages_and_sequences_with_heads_over_several_warps(att, fmt):
    page = 16
    cache = Cache(fmt, 1, 128, page, 40, 9)
    table = random_table([100, 200, 60], page, 40, 9)
    table[0, 2], table[1, 0], table[1, 11] = 40, -7, 2 ** 30
    for G in (20, 50):
        check(att, fmt, "bf16", "bf16", 128, 1, G, page, [100, 200, 60, 60], table=table, cache=cache, seq=[0, 1, 2, 3],
              status_want=5, weight_step=weight_step(fmt, "bf16"))
        check(att, fmt, "bf16", "bf16", 128, 1, G, page, [60, 60, 100], table=table, cache=cache, seq=[2, -1, 1],
              status_want=5, weight_step=weight_step(fmt, "bf16"))
