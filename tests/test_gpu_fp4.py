"""Microscaled 4-bit matrices against their definitions in 64 bits: rows
quantised (every code and scale), read back, and multiplied."""

import numpy as np
import pytest
import torch

from fp4_helpers import BLOCK, DT, FMT, ORDER, codes_at, dense, f64, multiplied, place, quantised, random_matrix, scales_at

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
LEAST = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -150}  # half of the smallest step


@pytest.fixture(scope="module")
def fp4(cuda_lib):
    from quantized_expert_ffn_router_gb300 import fp4

    return fp4


def rows_of(R, K, dtype, seed, offset=8):
    """[R, K] inside wider rows: channels and rows of uneven size, some values exactly at borders between codes."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(R, K, generator=g) * torch.exp(torch.randn(1, K, generator=g)) * torch.exp(2 * torch.randn(R, 1, generator=g))
    x[::3] = torch.randint(-28, 29, x[::3].shape, generator=g).float() / 4  # 7/4 halves of the block's largest, 7
    x = x.clamp(-6e4, 6e4)
    if R > 1:
        x[1, :min(16, K)] = 0
    if R > 4:
        x[4] = 0
    wide = torch.zeros(R, offset + K + offset, dtype=DT[dtype], device=DEV)
    t = wide[:, offset:offset + K]
    t.copy_(x.to(DT[dtype]))
    return t


def check_quantised(m, fmt, want, found):
    c, b, s = want
    assert np.array_equal(scales_at(m, fmt), b, equal_nan=True)
    got = codes_at(m).reshape(c.shape)
    keep = ~np.isnan(b)[..., None]  # codes under a NaN say nothing
    assert (np.where(keep, got, 0) == np.where(keep, c, 0)).all()
    if found:
        assert (f64(m.scale) == s).all()


QUANT = [(1, 16), (1, 32), (2, 48), (5, 96), (129, 160), (3, 2048), (37, 4112), (260, 544), (9, 16384), (2, 17408), (2, 65536)]


@pytest.mark.parametrize("R,K", QUANT)
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("order", ["tiles", "rows"])
def test_quantize_and_values(fp4, R, K, fmt, dtype, order):
    if K % BLOCK[fmt]:
        K += 16
    x = rows_of(R, K, dtype, R + K)
    m = fp4.Fp4Matrix(FMT[fmt], R, K, ORDER[order])
    m.codes.fill_(0x5A), m.scales.fill_(0x5A)
    fp4.fp4_quantize(x, m)
    want = quantised(fmt, f64(x))
    check_quantised(m, fmt, want, fmt == "nvfp4")
    # the bytes behind a row's codes are left, scales behind a row's last are 0, those of rows behind the last are left
    assert (m.codes[:, K // 2:] == 0x5A).all()
    if order == "tiles":
        n = K // BLOCK[fmt]
        up = -(-n // 4) * 4
        s = m.scales.cpu().numpy()
        assert (s[place(R, up)][:, n:] == 0).all()
        rest = np.ones(s.size, bool)
        rest[place(R, up)] = False
        assert (s[rest] == 0x5A).all()
    out = torch.full((R, K), float("nan"), dtype=DT[dtype], device=DEV)
    fp4.fp4_values(m, out)
    y = dense(*want)
    assert (np.abs(f64(out) - y) <= HALF[dtype] * np.abs(y) + LEAST[dtype]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("per", ["rows", "one", "none"])
def test_quantize_by_a_given_scale(fp4, dtype, per):
    R, K = 70, 1040
    x = rows_of(R, K, dtype, 5)
    m = fp4.Fp4Matrix(FMT["nvfp4"], R, K, ORDER["rows"])
    s = torch.exp(torch.randn(R if per == "rows" else 1, generator=torch.Generator().manual_seed(1))).to(DEV)
    m = fp4.Fp4Matrix.over(m.fmt, K, m.codes, m.scales, scale=None if per == "none" else s, order=m.order)
    fp4.fp4_quantize(x, m, given=True)
    given = np.ones(R) if per == "none" else np.broadcast_to(f64(s), R)
    want = quantised("nvfp4", f64(x), given)
    check_quantised(m, "nvfp4", want, False)
    out = torch.empty(R, K, dtype=torch.float32, device=DEV)
    fp4.fp4_values(m, out)
    y = dense(want[0], want[1], given)
    assert (np.abs(f64(out) - y) <= 2.0 ** -24 * np.abs(y)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_border_between_codes(fp4, dtype):
    """x = border * block scale, and its neighbours, for every block scale that a row of this size can have."""
    from attn_helpers import E2M1, E4M3

    b = E4M3[1:]
    mid = (E2M1[1:] + E2M1[:-1]) / 2
    x = np.zeros((len(b), 32))
    x[:, 0], x[:, 16] = 6 * b, -6 * b
    x[:, 1:8] = mid * b[:, None]
    x[:, 17:24] = -x[:, 1:8]
    near = torch.from_numpy(x).to(DT[dtype])
    up = f64(torch.nextafter(near, torch.full_like(near, 1e30)))
    down = f64(torch.nextafter(near, torch.full_like(near, -1e30)))
    for y in (f64(near), np.concatenate([up[:, :1] * 0 + x[:, :1], up[:, 1:]], 1),
              np.concatenate([down[:, :1] * 0 + x[:, :1], down[:, 1:]], 1)):
        for far in (2.0 ** -60, 1.0, 2.0 ** 60):
            t = torch.from_numpy(y * far).to(DT[dtype]).to(DEV)
            m = fp4.Fp4Matrix(FMT["nvfp4"], len(b), 32)
            fp4.fp4_quantize(t, m)
            check_quantised(m, "nvfp4", quantised("nvfp4", f64(t)), True)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("given", [False, True])
def test_infinities_and_nan(fp4, fmt, given):
    K = 96
    for dtype in ("bf16", "f16", "f32"):
        top = torch.finfo(DT[dtype]).max
        least = torch.finfo(DT[dtype]).smallest_normal / 64
        x = rows_of(12, K, dtype, 7)
        inf = float("inf")
        x[0, 3], x[1, 20], x[2, 40] = inf, -inf, float("nan")
        x[3] = 0
        x[3, 5] = -inf
        x[5] = inf
        x[6] = float("nan")
        x[7] = top
        x[8] = least
        x[9] = least
        x[9, 50] = top
        x[10, ::2], x[10, 1::2] = 0, -inf
        m = fp4.Fp4Matrix(FMT[fmt], 12, K)
        if given and fmt == "nvfp4":
            m.scale.fill_(0.37)
        fp4.fp4_quantize(x, m, given=given)
        s = np.full(12, np.float32(0.37)) if given and fmt == "nvfp4" else None
        check_quantised(m, fmt, quantised(fmt, f64(x), s), fmt == "nvfp4" and not given)


def product(fp4, x, w, fmt, dtype, add=None, pad=0, offset=0):
    T, N = x.rows, w.rows
    wide = torch.full((T + 1, offset + N + pad), float("nan"), dtype=DT[dtype], device=DEV)
    out = wide[:T, offset:offset + N]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    fp4.fp4_matmul(x, w, out, add=add, dev_status=status)
    assert int(status.item()) == 0
    assert wide[T:].isnan().all() and wide[:, :offset].isnan().all() and wide[:, offset + N:].isnan().all()
    return f64(out)


SIZES = [  # T, N, K
    (1, 1, 32), (1, 5, 16), (3, 131, 48), (70, 260, 16), (300, 300, 272), (1, 128, 256), (1, 200, 4096), (3, 130, 96), (16, 128, 2048), (17, 384, 544), (33, 5, 1024), (64, 2560, 2048),
    (65, 129, 608), (100, 333, 288), (128, 128, 512), (129, 257, 320), (191, 640, 32), (256, 256, 256), (300, 1000, 1120),
    (777, 512, 96), (1237, 200, 2592), (2048, 1024, 512), (2, 70000, 64), (5000, 17, 160)]


@pytest.mark.parametrize("T,N,K", SIZES)
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_products_are_exact_where_32_bits_hold_them(fp4, T, N, K, fmt):
    """Products are whole multiples of 2^-8 (2^-6), sums below 2^24 of those: nothing is rounded."""
    K += -K % BLOCK[fmt]
    x, w = random_matrix(fmt, T, K, 1), random_matrix(fmt, N, K, 2)
    got = product(fp4, x, w, fmt, "f32")
    assert (got == multiplied(x, w, fmt)).all()


@pytest.mark.parametrize("T,N,K", [(1, 100, 1040), (7, 4096, 4096), (64, 300, 528), (200, 130, 784), (600, 1111, 1040),
                                   (1000, 2048, 272)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("scale", ["rows", "one", "none"])
@pytest.mark.parametrize("aligned", [False, True])
def test_scales_and_a_sum(fp4, T, N, K, dtype, scale, aligned):
    """Sums are exact before the row scales: two products, the sum and the output's rounding are left."""
    x, w = random_matrix("nvfp4", T, K, 3, plain=False, scale=scale), random_matrix("nvfp4", N, K, 4, plain=False, scale=scale)
    lift = 2.0 ** -6  # inside f16's range
    if w.scale is not None:
        w.scale.mul_(lift).clamp_(max=4 * lift)
        x.scale.clamp_(max=2.0)
    y = multiplied(x, w, "nvfp4")
    # rows on 16-byte boundaries, which are written by whole boxes, or one element off them
    pad, offset = (-N % 8 + 8, 8) if aligned else (3, 1)
    add = torch.randn(T, offset + N + pad, generator=torch.Generator().manual_seed(0)).mul_(30).to(DT[dtype]).to(DEV)
    add = add[:, offset:offset + N]
    for more in (None, add):
        z = y if more is None else y + f64(more)
        got = product(fp4, x, w, "nvfp4", dtype, add=more, pad=pad, offset=offset)
        bound = 3 * 2.0 ** -24 * (np.abs(y) + np.abs(z))
        if dtype != "f32":
            bound = bound + HALF[dtype] * np.abs(z) * (1 + 2.0 ** -10) + LEAST[dtype]
        if dtype == "f16":
            z = np.where(np.abs(z) >= 65520, np.copysign(np.inf, z), z)
            bound = np.where(np.isinf(z), np.inf, bound)
        ok = np.isinf(z) | (np.abs(got - z) <= bound)
        assert ok.all()


@pytest.mark.parametrize("N", [296, 300])
@pytest.mark.parametrize("T", [5, 400])
def test_onto_itself_and_repeated(fp4, T, N):
    """add may be out; two runs give the same bits (slices of K are added in one order)."""
    x, w = random_matrix("nvfp4", T, 8192, 1, plain=False), random_matrix("nvfp4", N, 8192, 2, plain=False)
    res = torch.randn(T, N, device=DEV).to(torch.bfloat16)
    outs = []
    for _ in range(3):
        out = res.clone()
        fp4.fp4_matmul(x, w, out, add=out)
        outs.append(out)
    other = torch.empty_like(res)
    fp4.fp4_matmul(x, w, other, add=res)
    assert all(torch.equal(o, other) for o in outs)


@pytest.mark.parametrize("T,N,K", [(3, 256, 4096), (200, 256, 128), (200, 251, 128), (900, 1024, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_row_added_to_all(fp4, T, N, K, dtype):
    x, w = random_matrix("mxfp4", T, K, 1), random_matrix("mxfp4", N, K, 2)
    row = (torch.arange(N, device=DEV) - 100).to(DT[dtype])
    got = product(fp4, x, w, "mxfp4", dtype, add=row.expand(T, N), pad=-N % 8 + 8)
    want = multiplied(x, w, "mxfp4") + f64(row)
    assert (np.abs(got - want) <= HALF[dtype] * np.abs(want)).all()


def test_views(fp4):
    """Codes in wider rows, row scales a step apart, x whose rows are one row, in- and outputs of one row of any stride."""
    T, N, K = 37, 150, 96
    x, w = random_matrix("nvfp4", T, K, 1), random_matrix("nvfp4", N, K, 2)
    wide = lambda m: torch.cat((m.codes, torch.full((m.rows, 80), 0x77, dtype=torch.uint8, device=DEV)), 1)[:, :m.codes.shape[1]]
    apart = lambda m: torch.stack((m.scale, torch.full_like(m.scale, float("nan"))), 1)[:, 0]
    views = [fp4.Fp4Matrix.over(m.fmt, K, wide(m), m.scales, scale=apart(m)) for m in (x, w)]
    assert views[0].desc.pitch == 128 and views[0].desc.scale_stride == 2
    assert (product(fp4, *views, "nvfp4", "f32") == multiplied(x, w, "nvfp4")).all()
    row = rows_of(1, K, "bf16", 3)
    fp4.fp4_quantize(row.expand(T, K), views[0])
    want = quantised("nvfp4", np.broadcast_to(f64(row), (T, K)))
    check_quantised(views[0], "nvfp4", want, True)
    assert torch.isnan(views[0].scale.as_strided((2 * T - 1,), (1,))[1::2]).all()
    out = torch.empty(1, 3 * N, device=DEV)[:, ::3].as_strided((1, N), (7, 1))
    one = fp4.Fp4Matrix(FMT["nvfp4"], 1, K)
    fp4.fp4_quantize(row.as_strided((1, K), (5, 1)), one)
    fp4.fp4_matmul(one, w, out)
    want = multiplied(one, w, "nvfp4")
    assert (np.abs(f64(out) - want) <= 2.0 ** -23 * np.abs(want)).all()


def test_a_matrix_by_itself(fp4):
    x = random_matrix("mxfp4", 200, 320, 1)
    assert (product(fp4, x, x, "mxfp4", "f32") == multiplied(x, x, "mxfp4")).all()


def test_nothing_to_do(fp4):
    for T, N in ((0, 5), (5, 0)):
        x, w = fp4.Fp4Matrix(FMT["nvfp4"], T, 64), fp4.Fp4Matrix(FMT["nvfp4"], N, 64)
        fp4.fp4_quantize(torch.zeros(T, 64, device=DEV), x)
        fp4.fp4_values(x, torch.zeros(T, 64, device=DEV))
        fp4.fp4_matmul(x, w, torch.zeros(T, N, device=DEV))
