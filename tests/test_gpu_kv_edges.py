"""The paged cache's rows where numbers or sizes are out of the ordinary:
infinities, keys next to a border between codes, and more threads than 32 bits
number."""

import math

import numpy as np
import pytest
import torch

from attn_helpers import f64, quantised, rotated

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def att(cuda_lib):
    from quantized_expert_ffn_router_gb300 import attention

    return attention


def rows_next_to_borders(T, D, rot, layout, far, turn, fmt, seed):
    """T rows of bf16 numbers whose rotation to position `far` has an element right next to a border between two codes of
    the unrotated kind of scale: the closest among millions, by a 64-bit search."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    a = torch.from_numpy(far * turn).to(DEV)
    c, s = torch.cos(a), torch.sin(a)
    n = rot // 2
    at = (slice(0, rot, 2), slice(1, rot, 2)) if layout == "pairs" else (slice(0, n), slice(n, rot))
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV, dtype=torch.float64)
    best_x, best_d = None, None
    for _ in range(24):
        x = torch.randn(1 << 17, D, generator=g, device=DEV).to(torch.bfloat16)
        x[:, -1] = 0.0  # the infinity's place
        y = x[:, :rot].double()
        u, v = y[:, at[0]].clone(), y[:, at[1]].clone()
        y[:, at[0]], y[:, at[1]] = u * c - v * s, v * c + u * s
        if fmt == "nvfp4":
            whole = torch.cat([y, x[:, rot:].double()], 1)
            _, e = torch.frexp(whole.abs().amax(-1, keepdim=True) / 2688.0)
            z = (whole * torch.exp2(-e.double())).view(len(x), -1, 16)
            b = (z.abs().amax(-1, keepdim=True) / 6).float().to(torch.float8_e4m3fn).double()
            w = (z / b).view(len(x), D)[:, :rot].abs()
            near = torch.full_like(w, 9.0)
            for t in ties:
                near = torch.minimum(near, (w / t - 1).abs())
        else:  # ties of four-bit significands
            m, _ = torch.frexp(y.abs())
            near = ((m * 16 - 0.5) - torch.round(m * 16 - 0.5)).abs() / (m * 16)
        d = near.amin(-1)
        best_x = x if best_x is None else torch.cat([best_x, x])
        best_d = d if best_d is None else torch.cat([best_d, d])
        best_d, i = torch.topk(best_d, T, largest=False)
        best_x = best_x[i]
    return best_x


@pytest.mark.parametrize("fmt", ["e4m3", "nvfp4"])
@pytest.mark.parametrize("layout,D,rot", [("half", 64, 32), ("half", 64, 40), ("pairs", 64, 48), ("half", 160, 128)])
@pytest.mark.parametrize("infinite", [True, False])
def test_rotated_rows_next_to_borders(att, fmt, layout, D, rot, infinite):
    """The closest cases of three million rows, with an infinity in each or without."""
    T, page, far = 512, 64, 30011
    spin = att.Rope(rot, base=1e4, interleaved=layout == "pairs")
    turn = spin.freqs.cpu().numpy().astype(np.float64) * (2 * math.pi / 2.0 ** 64)
    k = rows_next_to_borders(T, D, rot, layout, far, turn, fmt, rot).view(T, 1, D)
    if infinite:
        k[..., -1] = math.inf
    cache = att.KvCache(att.FT_KV_E4M3 if fmt == "e4m3" else att.FT_KV_NVFP4, 1, D, page, T // page)
    table = torch.arange(T // page, dtype=torch.int32, device=DEV)[None]
    pos, seq = torch.arange(T, dtype=torch.int32, device=DEV), torch.zeros(T, dtype=torch.int32, device=DEV)
    att.kv_append(cache, k, -k, table, pos, seq=seq, rope=spin, rope_pos=torch.full_like(pos, far))
    ko, vo = torch.zeros(T, 1, D, device=DEV), torch.zeros(T, 1, D, device=DEV)
    att.kv_gather(cache, table, pos, ko, vo, seq=seq)
    want = quantised(fmt, rotated(f64(k), [far] * T, turn, layout, 1.0))
    assert (f64(ko) == want).all(), int((f64(ko) != want).sum())
    assert (f64(vo) == quantised(fmt, -f64(k))).all()


def test_gather_of_more_threads_than_32_bits_number(att):
    """2^28 + 64 rows of 256 channels, 16 threads a row: the last row is read (its page is a bad one, which is
    recorded).  The others are padding, and the output's rows are one place."""
    T, D = (1 << 28) + 64, 256
    cache = att.KvCache(att.FT_KV_E4M3, 1, D, 16, 1)
    pos = torch.full((T,), -1, dtype=torch.int32, device=DEV)
    pos[-1] = 3
    seq = torch.zeros(1, dtype=torch.int32, device=DEV).expand(T).contiguous()
    table = torch.full((1, 1), 7, dtype=torch.int32, device=DEV)
    out = torch.full((1, 1, D), 5.0, dtype=torch.bfloat16, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    att.kv_gather(cache, table, pos, out.expand(T, 1, D), None, seq=seq, dev_status=status)
    assert int(status.item()) == 5 and not out.any()


def test_infinities_in_nvfp4_blocks(att):
    """An infinity takes the block's largest code, 6 times its scale: the scale is that of the finite values, so 0 where
    there are none but zeros."""
    D = 64
    x = torch.zeros(3, 1, D)
    x[0, 0, :4] = torch.tensor([math.inf, 3.0, -math.inf, -1.5])
    x[0, 0, 20] = math.inf                      # alone in its block
    x[0, 0, 32] = 768.0                         # decides the row's exponent, not the first block's scale
    x[1, 0, 5] = -math.inf                      # alone in its row
    x[2, 0, :16], x[2, 0, 16:32] = 6.0, math.inf
    cache = att.KvCache(att.FT_KV_NVFP4, 1, D, 16, 1)
    pages, pos = torch.zeros(3, 1, dtype=torch.int32, device=DEV), torch.arange(3, dtype=torch.int32, device=DEV)
    att.kv_append(cache, x.bfloat16().to(DEV), -x.bfloat16().to(DEV), pages, pos)
    ko, vo = torch.ones(3, 1, D, device=DEV), torch.ones(3, 1, D, device=DEV)
    att.kv_gather(cache, pages, pos, ko, vo)
    want = torch.zeros(3, 1, D)
    want[0, 0, :4] = torch.tensor([3.0, 3.0, -3.0, -1.5])
    want[0, 0, 32] = 768.0
    want[2, 0, :16] = 6.0
    assert torch.equal(ko.cpu(), want) and torch.equal(vo.cpu(), -want)
