"""The decoder block example: its attention against attention computed in 64
bits from the same projections, its expert layer against the layer's own entry
point's oracle-checked call, step by step as the sequences grow, and the same
steps from one captured graph."""

import os
import sys

import numpy as np
import pytest
import torch

from attn_helpers import f64, quantised, rotated
from conftest import ROOT

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def example(cuda_lib):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import decoder_block

    return decoder_block


def attention_reference(block, qkvs):
    """The last step's attention from every step's projections [T, heads, D]."""
    T, Hq, Hkv, D = block.T, block.Hq, block.Hkv, block.D
    fmt = {0: "bf16", 2: "e4m3", 3: "nvfp4"}[block.cache.fmt]
    turn = block.rope.freqs.cpu().numpy().astype(np.float64) * (2 * np.pi / 2.0 ** 64)
    spin = lambda x, t: rotated(x, [t] * T, turn, "half", 1.0)
    n = len(qkvs)
    last = f64(torch.from_numpy(spin(qkvs[-1][:, :Hq], n - 1)).to(torch.bfloat16))
    k = np.stack([quantised(fmt, spin(x[:, Hq:Hq + Hkv], t)) for t, x in enumerate(qkvs)])
    v = np.stack([quantised(fmt, x[:, Hq + Hkv:]) for x in qkvs])
    out = np.zeros((T, Hq, D))
    for t in range(T):
        for h in range(Hq):
            s = k[:, t, h * Hkv // Hq] @ last[t, h] * D ** -0.5
            p = np.exp(s - s.max())
            out[t, h] = p @ v[:, t, h * Hkv // Hq] / p.sum()
    return out


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "nvfp4"])
def test_block_steps(example, fmt):
    block = example.DecoderBlock(fmt, longest=80, page_size=16)
    g = torch.Generator(device=DEV).manual_seed(1)
    qkvs = []
    for n in range(70):
        x = torch.randn(block.T, block.cfg.H, generator=g, device=DEV).to(torch.bfloat16)
        qkv = example.rms_norm(x) @ block.w_qkv.t()
        qkvs.append(f64(qkv).reshape(block.T, -1, block.D))
        y = block.step(x)
        if n in (0, 1, 15, 16, 69):
            want = attention_reference(block, qkvs)
            got = f64(block.attention.out)
            # the output's rounding, and that of q (and of keys held in bf16) to bf16 before the scores: 2^-8 each
            # of scores below 16, so 2^-3 at most of the weights' deviations; weights themselves 2^-12
            size = np.abs(want).max() + 1e-3
            assert np.abs(got - want).max() <= 2.0 ** -8 * size + 0.02 * size
            assert np.linalg.norm(got - want) <= 0.01 * np.linalg.norm(want)
    assert int(block.attention.status.item()) == 0 and int(block.moe.status.item()) == 0
    assert block.pos.tolist() == [70] * block.T and torch.isfinite(y.float()).all()


def test_block_in_a_graph(example):
    """A captured step replayed gives what separate steps give."""
    one, two = (example.DecoderBlock("e4m3", longest=40, page_size=16) for _ in range(2))
    x = torch.randn(one.T, one.cfg.H, device=DEV).to(torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        two.step(x)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            y = two.step(x)
        two.pos.zero_()
        for _ in range(20):
            graph.replay()
            z = one.step(x)
        side.synchronize()
        # the experts' cache states differ by the warm-up step, which may move a pair between slot and pool only
        assert torch.equal(one.attention.out, two.attention.out)
        assert torch.allclose(y.float(), z.float(), rtol=2.0 ** -7, atol=2.0 ** -7)
