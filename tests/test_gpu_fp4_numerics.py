"""Products of 4-bit matrices where numbers are out of the ordinary: row scales
far from one, NaN, weights and rows at the ends of the exponents."""

import numpy as np
import pytest
import torch

from fp4_helpers import DT, FMT, f64, multiplied, random_matrix
from test_gpu_fp4 import HALF, LEAST, fp4, product  # noqa: F401

pytestmark = pytest.mark.gpu
DEV = "cuda"
# T, N, K: slices of K, rows of out by boxes and one by one, tiles of many tokens
PATHS = [(1, 128, 4096), (70, 264, 528), (70, 261, 528), (300, 2008, 272), (1500, 520, 64), (1500, 518, 64)]


def beside(N):
    """Where out lies in wider rows: on 16-byte boundaries, or one or two elements off them."""
    return dict(pad=0, offset=0) if N % 8 == 0 else dict(pad=2, offset=2) if N % 2 == 0 else dict(pad=3, offset=1)


def rounded_once(got, want, dtype, products=2):
    """A rounding of each of the two products with row scales, and the output's; past its largest number, infinities."""
    # the largest number is 2^128 (1 - HALF), and half a step past it, from where on numbers round to infinity, is
    # 2^128 (1 - HALF / 2): both of a number within its three fp32 roundings of that may be
    border = 2.0 ** 128 * (1 - HALF[dtype] / 2)
    past, under = np.abs(want) > border * (1 + 2.0 ** -22), np.abs(want) < border * (1 - 2.0 ** -22)
    if not (got[past] == np.sign(want[past]) * np.inf).all():
        return False
    got, want = got[under], want[under]
    bound = (products + 1) * 2.0 ** -24 * np.abs(want) + LEAST["f32"]
    if dtype != "f32":
        bound = bound + HALF[dtype] * np.abs(want) * (1 + 2.0 ** -10) + LEAST[dtype]
    return (np.abs(got - want) <= bound).all()


@pytest.mark.parametrize("T,N,K", PATHS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("w_exp,x_exp", [(125, -110), (117, -64), (75, -60), (-110, 100), (-140, 125), (-64, 64)])
def test_row_scales_far_from_one(fp4, T, N, K, dtype, w_exp, x_exp):  # noqa: F811
    """The sum times one scale is infinite, or below the normal numbers, where the whole is neither."""
    x, w = random_matrix("nvfp4", T, K, 3), random_matrix("nvfp4", N, K, 4)
    x.scale.fill_(1.0).mul_(2.0 ** x_exp)
    w.scale.fill_(1.0)
    w.scale[::3] = 2.0 ** w_exp * (1.0 if w_exp == -140 else 1.37)
    got = product(fp4, x, w, "nvfp4", dtype, **beside(N))
    want = multiplied(x, w, "nvfp4")
    assert np.isfinite(want).all()
    assert rounded_once(got, want, dtype)


def test_weights_at_the_top_of_the_exponents(fp4):  # noqa: F811
    """Scales that were found: weights near bf16's largest, rows of small numbers."""
    T, N, K = 20, 136, 512
    g = torch.Generator(device=DEV).manual_seed(1)
    weight = (torch.randn(N, K, generator=g, device=DEV) * 5e37).to(torch.bfloat16)
    rows = (torch.randn(T, K, generator=g, device=DEV) * 1e-18).to(torch.bfloat16)
    x, w = fp4.Fp4Matrix(FMT["nvfp4"], T, K), fp4.Fp4Matrix(FMT["nvfp4"], N, K)
    fp4.fp4_quantize(rows, x), fp4.fp4_quantize(weight, w)
    got = product(fp4, x, w, "nvfp4", "f32")
    want = multiplied(x, w, "nvfp4")
    size = multiplied_sizes(x, w)
    assert (np.abs(got - want) <= K * 2.0 ** -23 * size).all()  # the sum's own roundings: see test_projection


def multiplied_sizes(x, w):
    from fp4_helpers import codes_at, row_scales, scales_at

    a, b = (np.abs(codes_at(m)) * np.repeat(scales_at(m, "nvfp4"), 16, -1) for m in (x, w))
    return (a @ b.T) * row_scales(x)[:, None] * row_scales(w)[None, :]


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,N,K", PATHS)
def test_nan_stays_in_its_row_and_column(fp4, fmt, dtype, T, N, K):  # noqa: F811
    """A block scale that is NaN makes its token's row of out NaN, or its weight row's column, and no other value."""
    K += -K % 32
    clean = [random_matrix(fmt, n, K, s) for n, s in ((T, 5), (N, 6))]
    want = multiplied(*clean, fmt)
    rows, cols = sorted({0, T // 2, T - 1}), sorted({1, N // 3, N - 1})
    blocks = K // (16 if fmt == "nvfp4" else 32)
    from fp4_helpers import place

    for m, at, b in ((clean[0], rows, blocks - 1), (clean[1], cols, 0)):
        where = place(m.rows, blocks)[at, b]
        m.scales[torch.from_numpy(where).to(DEV)] = 0x7F if fmt == "nvfp4" else 0xFF
    got = product(fp4, *clean, fmt, dtype, **beside(N))
    nan = np.zeros((T, N), bool)
    nan[rows], nan[:, cols] = True, True
    assert (np.isnan(got) == nan).all()
    assert rounded_once(got[~nan], want[~nan], dtype)


@pytest.mark.parametrize("T,N,K", PATHS + [(600, 2048, 8192), (2500, 4000, 528)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("added", [False, True])
def test_nothing_is_written_where_a_wait_gave_up_before(cuda_lib, fp4, dtype, added, T, N, K):  # noqa: F811
    """The status word that a call finds: of a wait that gave up, or another error, or none."""
    x, w = random_matrix("nvfp4", T, K, 1), random_matrix("nvfp4", N, K, 2)
    place = beside(N)
    wide = torch.full((T, place["offset"] + N + place["pad"]), 7.0, dtype=DT[dtype], device=DEV)
    out = wide[:, place["offset"]:place["offset"] + N]
    add = torch.full_like(wide, 8.0)[:, place["offset"]:place["offset"] + N] if added else None
    status = torch.full((1,), cuda_lib.FT_ERR_TIMEOUT, dtype=torch.int32, device=DEV)
    fp4.fp4_matmul(x, w, out, add=add, dev_status=status)
    assert (wide == 7.0).all() and int(status.item()) == cuda_lib.FT_ERR_TIMEOUT
    want = multiplied(x, w, "nvfp4") + (8.0 if added else 0.0)
    for found in (cuda_lib.FT_ERR_BAD_ID, 0):
        out.fill_(7.0), status.fill_(found)
        fp4.fp4_matmul(x, w, out, add=add, dev_status=status)
        assert rounded_once(f64(out), want, dtype) and int(status.item()) == found


@pytest.mark.parametrize("T,N,K", [(394, 19560, 1824), (385, 15289, 2080), (130, 39674, 3200), (132, 19744, 4640), (193, 9842, 1568),
                                   (390, 14655, 1312), (129, 32477, 544), (66, 9749, 832), (65, 19467, 32), (65, 1158, 2912),
                                   (1217, 150, 15616), (17, 38915, 32), (2, 4894, 2848)])
def test_far_scales_in_tiles_of_every_width(fp4, T, N, K):  # noqa: F811
    """Rows with far scales, in both directions, among others: pairs of CTAs and single ones, several tiles each, slices;
    out by boxes and row by row, residuals in place."""
    from test_gpu_fp4_tiles import random_on_gpu

    (x, xv), (w, wv) = random_on_gpu(fp4, "nvfp4", T, K, 1), random_on_gpu(fp4, "nvfp4", N, K, 2)
    sums = xv @ wv.T
    del xv, wv
    for w_exp, x_exp in ((120, -100), (-130, 110)):
        x.scale.fill_(2.0 ** x_exp * 1.25)
        w.scale.fill_(1.0)
        w.scale[5::37] = 2.0 ** w_exp
        w.scale[-1] = 2.0 ** w_exp
        y = sums * x.scale.double()[:, None] * w.scale.double()[None]
        for dtype, offset, pad, added in (("f32", 1, 0, False), ("bf16", 8, -N % 8 + 8, False), ("bf16", 8, -N % 8 + 8, True),
                                          ("bf16", 1, 2 + N % 2, True), ("bf16", 1, 3 + N % 2, False)):
            wide = torch.full((T + 1, offset + N + pad), float("nan"), dtype=DT[dtype], device=DEV)
            out, z = wide[:T, offset:offset + N], y
            if added:
                out.copy_(torch.randn(T, N, generator=torch.Generator(device=DEV).manual_seed(3), device=DEV))
                z = y + out.double()
            fp4.fp4_matmul(x, w, out, add=out if added else None)
            assert wide[T:].isnan().all() and wide[:, :offset].isnan().all() and wide[:, offset + N:].isnan().all()
            # roundings of the two products, of the sum, and of the output
            bound = 3 * 2.0 ** -24 * (y.abs() + z.abs()) + LEAST["f32"]
            if dtype != "f32":
                bound = bound + HALF[dtype] * z.abs() * (1 + 2.0 ** -10) + LEAST[dtype]
            border = 2.0 ** 128 * (1 - HALF[dtype] / 2)
            past, under = z.abs() > border * (1 + 2.0 ** -20), z.abs() < border * (1 - 2.0 ** -20)
            assert (out.double()[past] == torch.sign(z[past]) * float("inf")).all()
            assert ((out.double() - z).abs() <= bound)[under].all(), (w_exp, dtype, offset, added)
