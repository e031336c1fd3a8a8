"""Products of 4-bit matrices at a shape for every kind of tile that the library
chooses: single CTAs and pairs, each width, each number of slices of K, one wave
of tiles, two, and more; out by boxes and row by row, residuals beside and in
place.  test_fp4_tiles_host.py holds the list against the rule that chooses."""

import numpy as np
import pytest
import torch

from attn_helpers import E2M1, E4M3_BYTE
from fp4_helpers import BLOCK, FMT
from test_gpu_fp4 import DT, HALF, LEAST, fp4  # noqa: F401

DEV = "cuda"

SHAPES = [  # T, N, K
    (1, 150, 32), (1, 19457, 32), (1, 38915, 32), (1, 4894, 2848), (1, 2436, 1824), (1, 150, 1824), (17, 150, 32),
    (17, 19457, 32), (17, 38915, 32), (17, 4950, 3392), (17, 2480, 2336), (17, 150, 1824), (33, 150, 32),
    (33, 19461, 32), (33, 38948, 32), (34, 4896, 3872), (33, 2484, 2592), (33, 150, 2336), (49, 150, 32),
    (65, 9822, 32), (65, 19467, 32), (66, 2435, 4544), (65, 1158, 2912), (49, 150, 2592), (66, 9749, 832),
    (65, 29291, 544), (65, 49074, 544), (66, 4955, 9248), (65, 2434, 8800), (67, 1208, 17440), (9733, 150, 800),
    (129, 32477, 544), (130, 53272, 544), (4902, 150, 10720), (2442, 150, 8832), (1217, 150, 15616),
    (193, 9842, 1568), (390, 14655, 1312), (195, 49117, 1312), (203, 4933, 17312), (195, 2564, 17952),
    (68, 39046, 18720), (129, 9999, 9632), (132, 19744, 4640), (130, 39674, 3200), (195, 9860, 4448),
    (385, 15289, 2080), (394, 19560, 1824)]


def random_on_gpu(fp4, fmt, rows, K, seed):  # noqa: F811
    """As fp4_helpers.random_matrix: sums are exact in 32 bits; NaN where no row's scales are."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    draw = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device=DEV, dtype=torch.int32)
    codes = draw(0, 256, rows, -(-K // 32) * 16).to(torch.uint8)
    blocks = K // BLOCK[fmt]
    tall, wide = -(-rows // 128), -(-blocks // 4)
    s = draw(0x38, 0x40, tall * 128, wide * 4) if fmt == "nvfp4" else draw(125, 129, tall * 128, wide * 4)
    s[:, blocks:] = 0
    s[rows:] = 0x7F if fmt == "nvfp4" else 0xFF
    # [tile][row / 32][row % 32][tile of scales][scale] to tiles of [row % 32][row / 32][scale]
    tiles = s.view(tall, 4, 32, wide, 4).permute(0, 3, 2, 1, 4).to(torch.uint8).contiguous().view(-1)
    scale = torch.exp2(draw(-6, 7, rows).float()) if fmt == "nvfp4" else None
    lut = torch.from_numpy(np.concatenate([E2M1, -E2M1])).to(DEV)
    byte = torch.from_numpy(E4M3_BYTE if fmt == "nvfp4" else 2.0 ** (np.arange(256.0) - 127)).to(DEV)
    values = torch.stack((lut[(codes & 15).int()], lut[(codes >> 4).int()]), -1).view(rows, -1)[:, :K]
    values = (values.reshape(rows, blocks, -1) * byte[s[:rows, :blocks]][..., None]).view(rows, K)
    return fp4.Fp4Matrix.over(FMT[fmt], K, codes, tiles, scale=scale), values


@pytest.mark.gpu
@pytest.mark.parametrize("T,N,K", SHAPES)
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_products_of_every_kind_of_tile(fp4, fmt, T, N, K):  # noqa: F811
    (x, xv), (w, wv) = random_on_gpu(fp4, fmt, T, K, 1), random_on_gpu(fp4, fmt, N, K, 2)
    sums = xv @ wv.T  # exact in 64 bits
    del xv, wv
    bare = [fp4.Fp4Matrix.over(m.fmt, K, m.codes, m.scales) for m in (x, w)]  # f16 holds the sums without row scales
    want = sums if x.scale is None else sums * x.scale.double()[:, None] * w.scale.double()[None]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def check(dtype, offset, pad, added):
        a, b, y = (*bare, sums) if dtype == "f16" else (x, w, want)
        wide = torch.full((T + 1, offset + N + pad), float("nan"), dtype=DT[dtype], device=DEV)
        out, add, z = wide[:T, offset:offset + N], None, y
        if added:
            g = torch.Generator(device=DEV).manual_seed(3)
            more = (torch.randn(T, N, generator=g, device=DEV) * 100).to(DT[dtype])
            z = y + more.double()
            if added == "in place":
                out.copy_(more)
                add = out
            else:
                add = torch.empty_like(wide)[:T, offset:offset + N].copy_(more)
        fp4.fp4_matmul(a, b, out, add=add, dev_status=status)
        name = (dtype, offset, pad, added)
        assert int(status.item()) == 0, name
        assert wide[T:].isnan().all() and wide[:, :offset].isnan().all() and wide[:, offset + N:].isnan().all(), name
        # exact up to the addition, which fp32 rounds, and the output's rounding
        bound = 2.0 ** -24 * z.abs() if added else torch.zeros_like(z)
        if dtype != "f32":
            bound += HALF[dtype] * z.abs() * (1 + 2.0 ** -10) + LEAST[dtype]
        assert ((out.double() - z).abs() <= bound).all(), name

    whole = -N % 8 + 8
    check("f32", 0, 0, False)
    check("f32", 3, 2, "in place")
    check("bf16", 8, whole, False)  # by boxes
    check("bf16", 8, whole, "beside")
    check("bf16", 8, whole, "in place")
    check("f16", 8, whole, "in place")
    odd = 1 if (N + 4) % 2 else 2  # rows of an odd number of elements
    check("bf16", 1, 2 + odd, False)
    check("bf16", 1, 2 + odd, "beside")
    check("f16", 1, 2 + odd, "in place")
    if N % 2 == 0:  # two at a time
        check("bf16", 2, 6 - N % 4, "in place")
        check("f16", 2, 6 - N % 4, False)
