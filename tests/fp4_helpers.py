"""64-bit definitions that the 4-bit matrices' tests compare with.  Plain numpy,
no code of the library but its constants."""

import numpy as np
import torch

from attn_helpers import DT, E2M1, E4M3, E4M3_BYTE, E_MIN, f64, nearest
from quantized_expert_ffn_router_gb300 import fp4

__all__ = ["DT", "FMT", "ORDER", "BLOCK", "f64", "quantised", "place", "codes_at", "scales_at", "multiplied", "random_matrix", "dense"]

FMT = {"nvfp4": fp4.FT_FP4_NVFP4, "mxfp4": fp4.FT_FP4_MXFP4}
ORDER = {"tiles": fp4.FT_FP4_TILES, "rows": fp4.FT_FP4_ROWS}
BLOCK = {"nvfp4": 16, "mxfp4": 32}


def quantised(fmt, x, given=None):
    """(signed values of the codes, block scales, row scales or None) of rows x [R, K] in 64 bits; `given`: the scale
    of each row."""
    x = np.asarray(x, np.float64)
    fin = np.where(np.isfinite(x), np.abs(x), 0.0)
    if fmt == "mxfp4":
        m = fin.reshape(len(x), -1, 32).max(-1)
        _, e = np.frexp(m)
        e = np.where(m > 0, np.clip(e - 3, -127, 127), -127)
        b = 2.0 ** e.astype(np.float64)
        z, s = x.reshape(len(x), -1, 32) / b[..., None], None
    else:
        if given is None:
            m = fin.max(-1)
            e = np.full(m.shape, E_MIN)
            while np.any(m > 2688.0 * 2.0 ** e):
                e = np.where(m > 2688.0 * 2.0 ** e, e + 1, e)
            s = 2.0 ** e.astype(np.float64)
            y = x / s[:, None]
        else:
            s = np.asarray(given, np.float64)
            with np.errstate(all="ignore"):
                inv = (np.float32(1.0) / np.asarray(given, np.float32))[:, None]
                y = (np.asarray(x, np.float32) * inv).astype(np.float64)
        y = y.reshape(len(x), -1, 16)
        b = nearest(E4M3, np.where(np.isfinite(y), np.abs(y), 0.0).max(-1) / 6)
        z = np.divide(y, b[..., None], out=np.zeros_like(y), where=b[..., None] > 0)
    c = np.sign(np.nan_to_num(z, posinf=1, neginf=-1)) * nearest(E2M1, np.where(np.isnan(z), 0, z))
    nan = np.isnan(x).reshape(z.shape).any(-1)
    return c, np.where(nan, np.nan, b), s


def dense(c, b, s=None):
    y = (c * b[..., None]).reshape(len(c), -1)
    return y if s is None else y * s[:, None]


def place(rows, blocks):
    """Where block scale (r, b) lies in the order of tiles."""
    r, b = np.arange(rows)[:, None], np.arange(blocks)[None, :]
    return ((r // 128) * -(-blocks // 4) + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4


def scales_at(m, fmt):
    """A matrix's block scales [rows, blocks] in 64 bits."""
    blocks = m.K // BLOCK[fmt]
    s = m.scales.view(torch.uint8).cpu().numpy().reshape(-1)
    s = s[place(m.rows, blocks)] if m.order == fp4.FT_FP4_TILES else s[:m.rows * blocks].reshape(m.rows, blocks)
    return E4M3_BYTE[s] if fmt == "nvfp4" else np.where(s == 255, np.nan, 2.0 ** (s.astype(np.float64) - 127))


def codes_at(m):
    c = m.codes.cpu().numpy()[:, :m.K // 2]
    n = np.stack([c & 15, c >> 4], -1).reshape(m.rows, m.K)
    return np.where(n >= 8, -1.0, 1.0) * E2M1[n & 7]


def row_scales(m):
    return np.ones(m.rows) if m.scale is None else np.broadcast_to(f64(m.scale).reshape(-1), m.rows)


def multiplied(x, w, fmt):
    """x w^T in 64 bits: the sums first, which 64 bits hold exactly, then the row scales."""
    x_b, w_b = (codes_at(m) * np.repeat(scales_at(m, fmt), BLOCK[fmt], -1) for m in (x, w))
    return (x_b @ w_b.T) * row_scales(x)[:, None] * row_scales(w)[None, :]


def random_matrix(fmt, rows, K, seed, device="cuda", plain=True, scale="rows"):
    """A matrix of random codes and block scales of 1 to 1.875 (powers of two from 1/4 to 2), laid out in tiles, with
    NaN where no row's scales are.  `plain`: rows scaled by powers of two, so that sums of 64-bit size come out
    exactly in 32 bits."""
    g = np.random.default_rng(seed)
    codes = g.integers(0, 256, (rows, -(-K // 32) * 16)).astype(np.uint8)
    blocks = K // BLOCK[fmt]
    tiles = np.full(-(-rows // 128) * -(-blocks // 4) * 512, 0x7F if fmt == "nvfp4" else 0xFF, np.uint8)
    up = -(-blocks // 4) * 4
    tiles[place(rows, up)] = 0
    tiles[place(rows, blocks)] = g.integers(0x38, 0x40, (rows, blocks)) if fmt == "nvfp4" else g.integers(125, 129, (rows, blocks))
    s = None
    if fmt == "nvfp4" and scale != "none":
        n = rows if scale == "rows" else 1
        s = 2.0 ** g.integers(-6, 7, n) if plain else np.exp(g.normal(0, 2, n))
        s = torch.from_numpy(s.astype(np.float32)).to(device)
    return fp4.Fp4Matrix.over(FMT[fmt], K, torch.from_numpy(codes).to(device), torch.from_numpy(tiles).to(device), scale=s)
