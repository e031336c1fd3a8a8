"""64-bit definitions that the attention operators' tests compare with: number
formats, rotation, cached rows, attention.  Plain numpy, no code of the library."""

import numpy as np
import torch

from quantized_expert_ffn_router_gb300 import attention as att

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
FMT = {"bf16": att.FT_KV_BF16, "f16": att.FT_KV_F16, "e4m3": att.FT_KV_E4M3, "nvfp4": att.FT_KV_NVFP4}
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([m / 8 * 2.0 ** -6 if x == 0 else (1 + m / 8) * 2.0 ** (x - 7) for x in range(16) for m in range(8)][:127])
E4M3_BYTE = np.concatenate([E4M3, [np.nan], -E4M3, [np.nan]])
E_MIN = -64


def f64(t):
    return t.detach().cpu().double().numpy()


def nearest(levels, y):
    """|y| to the nearest level, ties to the even index, at most the last."""
    y = np.abs(y)
    i = np.clip(np.searchsorted(levels, y), 1, len(levels) - 1)
    lo, hi = levels[i - 1], levels[i]
    up = (y - lo > hi - y) | ((y - lo == hi - y) & (i % 2 == 0))
    return np.where(up, hi, lo)


def quantised(fmt, y):
    """What rows y [..., D] read back as."""
    y = np.asarray(y, np.float64)
    if fmt == "bf16":
        return f64(torch.from_numpy(y).to(torch.bfloat16))
    if fmt == "f16":
        return f64(torch.from_numpy(y).to(torch.float16))
    top = 448.0 if fmt == "e4m3" else 2688.0
    fin = np.where(np.isfinite(y), np.abs(y), 0.0)
    most = fin.max(-1)
    e = np.full(most.shape, E_MIN)
    while np.any(most > top * 2.0 ** e):
        e = np.where(most > top * 2.0 ** e, e + 1, e)
    s = 2.0 ** e[..., None]
    z = y / s
    if fmt == "e4m3":
        return np.where(np.isnan(z), np.nan, np.sign(z) * nearest(E4M3, np.where(np.isnan(z), 0, z)) * s)
    z = z.reshape(*z.shape[:-1], -1, 16)
    b = nearest(E4M3, np.where(np.isfinite(z), np.abs(z), 0.0).max(-1) / 6)[..., None]
    w = np.divide(z, b, out=np.zeros_like(z), where=b > 0)
    code = np.sign(w) * nearest(E2M1, np.where(np.isnan(w), 0, w))
    out = np.where(np.isnan(z).any(-1, keepdims=True), np.nan, code * b)
    return out.reshape(y.shape) * s


def rotated(y, pos, freqs, layout, mscale):
    """Rows [T, h, D] turned to pos by freqs (radians a position), in 64 bits."""
    y = np.array(y, np.float64)
    n = len(freqs)
    a = np.asarray(pos, np.float64)[:, None] * np.asarray(freqs)[None, :]
    c, s = (np.cos(a) * mscale)[:, None, :], (np.sin(a) * mscale)[:, None, :]
    at = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if layout == "pairs" else (slice(0, n), slice(n, 2 * n))
    u, v = y[..., at[0]].copy(), y[..., at[1]].copy()
    y[..., at[0]], y[..., at[1]] = u * c - v * s, v * c + u * s
    return y


class Cache:
    """A random cache on the device, with what its rows stand for in 64 bits."""

    def __init__(self, fmt, Hkv, D, page, pages, seed, order="phsd", fill=None, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.fmt, self.D = fmt, D
        dims = dict(p=pages, h=Hkv, s=page)
        shape = tuple(dims[c] for c in order[:3])
        perm = tuple(order.index(c) for c in "phs")

        def arr(w, dtype, values):
            t = torch.empty(*shape, w, dtype=dtype).permute(*perm, 3)
            t.copy_(values)
            return t

        self.arrays, self.values = {}, {}
        std = (pages, Hkv, page)
        for n in ("k", "v"):
            if fmt in ("bf16", "f16"):
                self.arrays[n] = arr(D, DT[fmt], torch.randn(*std, D, generator=g))
                self.values[n] = f64(self.arrays[n])
                continue
            ex = torch.randint(118, 126, std, generator=g, dtype=torch.uint8)
            sc = torch.empty(shape, dtype=torch.uint8).permute(*perm)
            sc.copy_(ex)
            self.arrays[n + "_scale"] = sc
            s = 2.0 ** (f64(ex) - 127)[..., None]
            if fmt == "e4m3":
                code = (torch.randn(*std, D, generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                self.arrays[n] = arr(D, torch.uint8, code)
                self.values[n] = E4M3_BYTE[code.numpy()] * s
            else:
                code = torch.randint(0, 256, (*std, D // 2), generator=g, dtype=torch.uint8)
                blk = torch.randint(0x40, 0x70, (*std, D // 16), generator=g, dtype=torch.uint8)
                self.arrays[n] = arr(D // 2, torch.uint8, code)
                self.arrays[n + "_block"] = arr(D // 16, torch.uint8, blk)
                x = np.concatenate([E2M1, -E2M1])
                y = np.stack([x[code.numpy() & 15], x[code.numpy() >> 4]], -1).reshape(*std, D)
                self.values[n] = y * np.repeat(E4M3_BYTE[blk.numpy()], 16, -1) * s / 64
                self.arrays[n + "_scale"] -= 6
        dev = {n: torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device=device) for n, t in self.arrays.items()}
        for n, t in self.arrays.items():
            dev[n].copy_(t)
        self.arrays = dev
        self.desc = att.KvCache.over(FMT[fmt], D, **dev)

    def row(self, name, page, head):
        return self.values[name][page, head]


def random_table(lens, page, pages, seed, width=None, device="cuda"):
    """[n, width] page table over shuffled pages, -1 past a sequence's length."""
    r = np.random.default_rng(seed)
    need = [-(-int(n) // page) for n in lens]
    assert sum(need) <= pages
    order = r.permutation(pages)
    width = width or max(1, max(need))
    table = np.full((len(lens), width), -1, np.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return table


def attention(cache, q, table, lens, page, scale, window=0, seq=None):
    """(out, lse, what bounds the error) in 64 bits, for q [T, Hq, D]; tokens on bad pages do not count."""
    T, Hq, D = q.shape
    Hkv = cache.desc.Hkv
    G = Hq // Hkv
    pages = cache.desc.n_pages
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    mass, reach, floor = np.zeros((T, Hq, D)), np.zeros((T, Hq)), np.zeros((T, Hq))
    for t in range(T):
        n = int(lens[t])
        s = t if seq is None else int(seq[t])
        j = np.arange(max(0, n - window) if window else 0, n)
        if not (0 <= s < len(table)):
            continue
        p, sl = table[s][j // page], j % page
        ok = (p >= 0) & (p < pages)
        p, sl = p[ok], sl[ok]
        if not len(p):
            continue
        for h in range(Hq):
            k, v = cache.values["k"][p, h // G, sl], cache.values["v"][p, h // G, sl]
            x = scale * (k @ q[t, h])
            m = x.max()
            w = np.exp(x - m)
            z = w.sum()
            out[t, h] = w @ v / z
            lse[t, h] = m + np.log(z)
            mass[t, h] = w @ np.abs(v) / z
            reach[t, h] = (abs(scale) * (np.abs(k) @ np.abs(q[t, h]))).max()
            # what weights too small for f16 can add up to: 2^-25 of the heaviest row each
            row = np.abs(v).max(-1)
            floor[t, h] = len(p) * (w / z * np.maximum(row, 1e-30)).max() * 64
    return out, lse, (mass, reach, floor)


def attention_tolerance(fmt, out_dtype, D, out, lse, parts, weight_step=None):
    """Bounds on |kernel - exact|, from the roundings that the kernel makes:
    scores: fp32 sums of D / 16 truncated steps, and their scaling (2^-23 each);
    weights: f16 (2^-12), two f16 terms (2^-23) or two bf16 terms (2^-17);
    2^-22 for the exponential, 2^-23 for each fp32 sum; the output's own.
    Those of the weights are typical: the largest, for rows of few tokens, are
    twice as large, and a test that meets them gives its `weight_step`."""
    mass, reach, floor = parts
    ds = (D / 16 + 6) * 2.0 ** -23 * reach + 2.0 ** -20
    dp = 2.0 ** -17 if fmt == "bf16" else 2.0 ** -22 if out_dtype == "f32" else 2.0 ** -12
    dp = dp if weight_step is None else weight_step
    small = 0.0 if fmt == "bf16" else 2.0 ** -36 if out_dtype == "f32" else 2.0 ** -25
    half = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -23}[out_dtype]
    tol = half * np.abs(out) + mass * (dp + 2 * ds[..., None]) + small * floor[..., None] + 2.0 ** -25 * (out_dtype == "f16")
    return tol, ds + 2.0 ** -21 + np.where(np.isfinite(lse), np.abs(lse), 0) * 2.0 ** -22
