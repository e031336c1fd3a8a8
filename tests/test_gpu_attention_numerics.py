"""ft_attn_decode where rounding to fewer bits, or a number's range, could show:
light weights beside heavy ones, 16-bit outputs of 8- and 4-bit caches, small
query elements, keys and scores at the ends of fp32, infinities that count.
Rows are written by kv_append and compared as kv_gather reads them back."""

import math

import numpy as np
import pytest
import torch

from attn_helpers import DT, FMT, f64

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def att(cuda_lib):
    from quantized_expert_ffn_router_gb300 import attention

    return attention


class Rows:
    """One sequence's k and v [n, Hkv, D] in a cache of its own, and what they stand for."""

    def __init__(self, att, fmt, dtype, k, v, page=16):
        n, self.Hkv, self.D = k.shape
        pages = -(-n // page) + 2
        self.att, self.n = att, n
        self.cache = att.KvCache(FMT[fmt], self.Hkv, self.D, page, pages)
        order = np.random.default_rng(n).permutation(pages)[:-(-n // page)].astype(np.int32)
        self.table = torch.from_numpy(order[None]).to(DEV)
        pos, seq = torch.arange(n, dtype=torch.int32, device=DEV), torch.zeros(n, dtype=torch.int32, device=DEV)
        att.kv_append(self.cache, k.to(DT[dtype]).to(DEV), v.to(DT[dtype]).to(DEV), self.table, pos, seq=seq)
        ko, vo = (torch.empty(n, self.Hkv, self.D, device=DEV) for _ in "kv")
        att.kv_gather(self.cache, self.table, pos, ko, vo, seq=seq)
        self.k, self.v = f64(ko), f64(vo)
        self.ev = np.zeros((n, self.Hkv))  # exponents of the value rows
        if self.cache.v_scale is not None:
            at = np.arange(n)
            self.ev = f64(self.cache.v_scale)[order[at // page], :, at % page] - 127

    def attend(self, q, out_dtype, scale):
        att, (_, Hq, D) = self.att, q.shape
        out = torch.full((1, Hq, D), float("nan"), dtype=DT[out_dtype], device=DEV)
        lse = torch.full((1, Hq), float("nan"), device=DEV)
        ws = torch.full((att.attn_decode_workspace(1, Hq, self.Hkv, D),), 0xFF, dtype=torch.uint8, device=DEV)
        lens = torch.tensor([self.n], dtype=torch.int32, device=DEV)
        att.attn_decode(self.cache, q, self.table, lens, out, ws, scale=scale, lse=lse)
        return out, lse

    def exact(self, q, scale):
        """(output, log-sum, weights [Hq, n], scores' reach) in 64 bits."""
        q, scale = f64(q)[0], float(np.float32(scale))
        G = q.shape[0] // self.Hkv
        out, lse, w, reach = np.zeros_like(q), np.zeros(len(q)), np.zeros((len(q), self.n)), np.zeros(len(q))
        for h in range(len(q)):
            x = scale * (self.k[:, h // G] @ q[h])
            e = np.exp(x - x.max())
            w[h] = e / e.sum()
            out[h], lse[h] = w[h] @ self.v[:, h // G], x.max() + np.log(e.sum())
            reach[h] = (abs(scale) * np.abs(self.k[:, h // G]) @ np.abs(q[h])).max()
        return out, lse, w, reach


def bound(rows, fmt, out_dtype, out, w, reach):
    """What the output may be off by.  The weights: scores are fp32 sums of D / 16 steps (2^-23 of their reach each) and
    their scaling, the exponential 2^-22, a step of 16 tokens 2^-23, two terms of f16 2^-22 or of bf16 2^-16, and with
    f16 2^-36 of the heaviest weight (times its value's exponent) for each token.  Then the output's own half step."""
    G = len(w) // rows.Hkv
    v = np.repeat(rows.v.transpose(1, 0, 2), G, 0)                 # [Hq, n, D]
    ev = np.repeat(rows.ev.T, G, 0)                                # [Hq, n]
    mass = np.einsum("hn,hnd->hd", w, np.abs(v))
    heavy = (w * 2.0 ** ev).max(-1)
    floor = 0.0 if fmt == "bf16" else 2.0 ** -36 * heavy[:, None] * (np.abs(v) * 2.0 ** -ev[..., None]).sum(1)
    each = 2 * (rows.D / 16 + 6) * 2.0 ** -23 * reach + (rows.n / 16 + 16) * 2.0 ** -23 + 2.0 ** -21
    each = each + (2.0 ** -16 if fmt == "bf16" else 2.0 ** -22)
    half = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}[out_dtype]
    return half * np.abs(out) + mass * each[:, None] + floor + 2.0 ** -25 * (out_dtype == "f16")


def lse_bound(D, lse, reach):
    return (D / 16 + 6) * 2.0 ** -23 * reach + 2.0 ** -20 * (1 + np.abs(lse))


@pytest.mark.parametrize("fmt,dtype,out_dtype", [("bf16", "bf16", "bf16"), ("bf16", "bf16", "f32"), ("f16", "f16", "f16"),
                                                 ("f16", "f16", "f32"), ("e4m3", "bf16", "bf16"), ("e4m3", "f16", "f32"),
                                                 ("nvfp4", "bf16", "f32"), ("nvfp4", "bf16", "bf16")])
@pytest.mark.parametrize("gap", [8, 20, 26, 30])
@pytest.mark.parametrize("G", [4, 20])
def test_light_weights_beside_heavy_ones(att, fmt, dtype, out_dtype, gap, G):
    """Every 16th token weighs 2^gap times what the others do, and only the others have values outside channel 0."""
    n, D, g = 1003, 128, torch.Generator().manual_seed(gap)
    dirn = torch.randn(D, generator=g)
    q = dirn.repeat(1, G, 1).to(DT[dtype])
    k = torch.randn(n, 1, D, generator=g) * 0.05
    v = (torch.randn(n, 1, D, generator=g) + 1.0).clamp(-4, 6) * 256
    heavy = torch.arange(n) % 16 == 3
    scale = D ** -0.5
    k[heavy, 0] = dirn * (gap * math.log(2.0) / (scale * float(dirn.square().sum())))
    v[heavy] = 0.0
    v[heavy, 0, 0] = 256.0
    rows = Rows(att, fmt, dtype, k, v)
    out, lse = rows.attend(q.to(DEV), out_dtype, scale)
    want, want_lse, w, reach = rows.exact(q, scale)
    err = np.abs(f64(out)[0] - want)
    assert (err <= bound(rows, fmt, out_dtype, want, w, reach)).all(), (err / np.abs(want))[:, 1:].max()
    assert (np.abs(f64(lse)[0] - want_lse) <= lse_bound(D, want_lse, reach)).all()


@pytest.mark.parametrize("fmt", ["e4m3", "nvfp4", "bf16", "f16"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,Hkv,G,n", [(128, 2, 4, 3000), (64, 1, 40, 700), (256, 3, 1, 90), (192, 2, 16, 1)])
def test_sixteen_bit_outputs_are_the_fp32_ones_rounded(att, fmt, dtype, D, Hkv, G, n):
    """The output's type decides the last rounding and nothing before it."""
    if fmt in ("bf16", "f16") and fmt != dtype:
        pytest.skip("a 16-bit cache takes queries of its own type")
    g = torch.Generator().manual_seed(D + n)
    k, v = torch.randn(n, Hkv, D, generator=g), torch.randn(n, Hkv, D, generator=g)
    q = torch.randn(1, Hkv * G, D, generator=g).to(DT[dtype]).to(DEV)
    rows = Rows(att, fmt, dtype, k, v)
    short, lse = rows.attend(q, dtype, D ** -0.5)
    full, full_lse = rows.attend(q, "f32", D ** -0.5)
    assert torch.equal(short, full.to(DT[dtype])) and torch.equal(lse, full_lse)
    want, _, w, reach = rows.exact(q, D ** -0.5)
    assert (np.abs(f64(full)[0] - want) <= bound(rows, fmt, "f32", want, w, reach)).all()


@pytest.mark.parametrize("fmt", ["e4m3", "nvfp4"])
@pytest.mark.parametrize("small", [-12, -20, -28])
def test_query_elements_far_below_the_largest(att, fmt, small):
    """bf16 queries keep their eight bits 2^28 below the head's largest element: keys are zero where that one is."""
    n, D, g = 200, 64, torch.Generator().manual_seed(1)
    q = torch.zeros(1, 4, D)
    q[..., 0] = 1.9921875
    q[0, :, 1] = torch.tensor([1.9921875, 1.7578125, -1.1796875, 1.0078125]) * 2.0 ** small
    k = torch.zeros(n, 1, D)
    k[:, 0, 1] = (torch.randint(-16, 17, (n,), generator=g) / 4.0) * 2.0 ** -small
    rows = Rows(att, fmt, "bf16", k, torch.randn(n, 1, D, generator=g))
    q = q.bfloat16().to(DEV)
    out, lse = rows.attend(q, "f32", 1.0)
    want, want_lse, w, reach = rows.exact(q, 1.0)
    assert (np.abs(f64(out)[0] - want) <= bound(rows, fmt, "f32", want, w, reach)).all()
    assert (np.abs(f64(lse)[0] - want_lse) <= lse_bound(D, want_lse, reach)).all()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "nvfp4"])
def test_keys_near_the_end_of_the_range(att, fmt):
    """Scores of 2^121: far apart, but finite, so the largest takes all."""
    n, D, g = 9, 64, torch.Generator().manual_seed(2)
    u = torch.randn(D, generator=g).bfloat16().float()
    k = (torch.arange(n) - 4).view(n, 1, 1) * 2.0 ** 116 * u
    rows = Rows(att, fmt, "bf16", k, torch.randn(n, 1, D, generator=g))
    q = torch.stack([u, -u])[None].bfloat16().to(DEV)
    out, lse = rows.attend(q, "f32", 0.125)
    assert (np.abs(f64(out)[0] - rows.v[[n - 1, 0], 0]) <= 2.0 ** -20 * np.abs(rows.v[[n - 1, 0], 0])).all()
    top = 0.125 * (rows.k[:, 0] @ f64(q)[0].T).max(0)
    assert (np.abs(f64(lse)[0] - top) <= 2.0 ** -20 * top).all()


def test_a_score_near_the_lowest_number(att):
    """A lone token takes all the weight, whatever its score."""
    D = 64
    k, v = torch.zeros(1, 1, D), torch.randn(1, 1, D, generator=torch.Generator().manual_seed(3))
    k[0, 0, 0] = 2.0 ** 64
    q = torch.zeros(1, 2, D)
    q[..., 0] = -1.3046875 * 2.0 ** 63  # -2.2e38, -3.2e38 in powers of two
    rows = Rows(att, "bf16", "bf16", k, v)
    out, lse = rows.attend(q.bfloat16().to(DEV), "f32", 1.0)
    assert (np.abs(f64(out)[0] - rows.v[0]) <= 2.0 ** -20 * np.abs(rows.v[0])).all()
    assert (np.abs(f64(lse)[0] + 1.3046875 * 2.0 ** 127) <= 2.0 ** 127 * 2.0 ** -20).all()


@pytest.mark.parametrize("fmt", ["bf16", "f16", "e4m3", "nvfp4"])
@pytest.mark.parametrize("G", [2, 20])
def test_sums_of_the_largest_values(att, fmt, G):
    """A mean of values at the end of the type's range is inside it, of whichever number of tokens."""
    n, D, g = 1501, 64, torch.Generator().manual_seed(6)
    dtype = "f16" if fmt == "f16" else "bf16"
    most = {"bf16": 3.3895313892515355e38, "f16": 65504.0}.get(fmt, 2.0 ** 126)  # 8- and 4-bit: read back below 2^128
    v = torch.full((n, 1, D), most)
    v[..., 1] *= torch.randn(n, 1, generator=g).sign()
    v[..., 2:] *= torch.rand(n, 1, D - 2, generator=g) * 2 - 1
    rows = Rows(att, fmt, dtype, torch.randn(n, 1, D, generator=g) * 0.3, v)
    q = torch.randn(1, G, D, generator=g).to(DT[dtype]).to(DEV)
    for out_dtype in (dtype, "f32"):
        out, _ = rows.attend(q, out_dtype, D ** -0.5)
        want, _, w, reach = rows.exact(q, D ** -0.5)
        assert torch.isfinite(out).all()
        assert (np.abs(f64(out)[0] - want) <= bound(rows, fmt, out_dtype, want, w, reach)).all()


@pytest.mark.parametrize("fmt", ["bf16", "f16"])
@pytest.mark.parametrize("G", [4, 40])
@pytest.mark.parametrize("n", [20, 300])
def test_an_infinite_value_that_counts_is_nan_in_its_channel_only(att, fmt, G, n):
    D, g = 64, torch.Generator().manual_seed(4)
    k, v = torch.randn(n, 2, D, generator=g), torch.randn(n, 2, D, generator=g)
    q = torch.randn(1, 2 * G, D, generator=g).to(DT[fmt]).to(DEV)
    plain, lse = Rows(att, fmt, fmt, k, v).attend(q, fmt, 0.125)
    v[n // 4, 1, 5] = math.inf
    out, inf_lse = Rows(att, fmt, fmt, k, v).attend(q, fmt, 0.125)
    assert torch.isnan(out[0, G:, 5]).all() and torch.equal(lse, inf_lse)
    out[0, G:, 5] = plain[0, G:, 5]
    assert torch.equal(out, plain)


@pytest.mark.parametrize("fmt", ["e4m3", "nvfp4"])
def test_exponent_bytes_outside_the_format(att, fmt):
    """Bytes that no row is written with: reading back and attending take them for the nearest that one is (2^-64, and
    2^120 or, with block scales, 2^117)."""
    D, g = 64, torch.Generator().manual_seed(5)
    byte = torch.tensor([0, 1, 40, 62, 63, 64, 127, 243, 244, 245, 247, 248, 250, 254, 255], dtype=torch.uint8)
    n = len(byte)
    x = torch.randint(-6, 7, (n, 1, D), generator=g).float()
    x[..., ::16] = 6.0  # every block's largest
    rows = Rows(att, fmt, "bf16", x * 448 / 6 if fmt == "e4m3" else x, x * 0.5, page=16)
    cache, at = rows.cache, int(rows.table[0, 0])
    was = {w: f64(getattr(cache, w + "_scale"))[at, 0, :n] for w in "kv"}
    held = np.clip(byte.numpy().astype(np.float64), 63, 247 if fmt == "e4m3" else 244)
    for w in "kv":
        getattr(cache, w + "_scale")[at, 0, :n] = byte.to(DEV)
        setattr(rows, w, getattr(rows, w) * 2.0 ** (held - was[w])[:, None, None])
    ko, vo = torch.empty(n, 1, D, device=DEV), torch.empty(n, 1, D, device=DEV)
    pos, seq = torch.arange(n, dtype=torch.int32, device=DEV), torch.zeros(n, dtype=torch.int32, device=DEV)
    att.kv_gather(cache, rows.table, pos, ko, vo, seq=seq)
    with np.errstate(over="ignore"):
        assert (f64(ko) == rows.k.astype(np.float32)).all() and (f64(vo) == rows.v.astype(np.float32)).all()
    # one token at a time: its value is the output, its key the score
    q = torch.zeros(1, 1, D, dtype=torch.bfloat16, device=DEV)
    q[..., 0] = 2.0 ** -30
    for j in range(n):
        one = torch.tensor([j + 1], dtype=torch.int32, device=DEV)
        out, lse = torch.zeros(1, 1, D, device=DEV), torch.zeros(1, 1, device=DEV)
        ws = torch.zeros(att.attn_decode_workspace(1, 1, 1, D), dtype=torch.uint8, device=DEV)
        att.attn_decode(cache, q, rows.table, one, out, ws, scale=2.0 ** -30, window=1, lse=lse)
        with np.errstate(over="ignore"):
            want = rows.v[j, 0].astype(np.float32)
        got, score = f64(out)[0, 0], rows.k[j, 0, 0] * 2.0 ** -60
        fin = np.isfinite(want)
        assert (np.abs(got - want)[fin] <= 2.0 ** -20 * np.abs(want)[fin]).all() and (got[~fin] == want[~fin]).all()
        assert abs(float(lse) - score) <= 2.0 ** -20 * (1 + abs(score))
