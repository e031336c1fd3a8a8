"""4-bit matrices and rotations by several axes as they are used: a block's
projections around its attention, expert blocks made from weights, captured
steps, calls on several streams, sizes past 32 bits."""

import os
import sys

import numpy as np
import pytest
import torch

from attn_helpers import rotated
from conftest import ROOT
from fp4_helpers import FMT, codes_at, dense, f64, multiplied, quantised, random_matrix, scales_at
from test_gpu_rope_axes import axis_of

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def fp4(cuda_lib):
    from quantized_expert_ffn_router_gb300 import fp4

    return fp4


@pytest.fixture(scope="module")
def pipeline(cuda_lib):
    from quantized_expert_ffn_router_gb300 import pipeline

    return pipeline


@pytest.fixture(scope="module")
def example(cuda_lib):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import decoder_block

    return decoder_block


def bf16(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV).to(torch.bfloat16)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T,N,K", [(1, 384, 256), (3, 100, 1056), (130, 264, 512), (500, 1000, 320)])
def test_projection(pipeline, fmt, T, N, K):
    """Of both quantised matrices, exactly as their definitions give them: fp32's sums of K products and the output's
    rounding are left (a sum of K terms in any order, with terms cut off at fp32's step: K 2^-23 of their sizes)."""
    g = gen(T + N)
    weight, x, add = bf16(g, N, K), bf16(g, T, K), bf16(g, T, N)
    p = pipeline.Projection(weight, T, FMT[fmt])
    wq, xq = (dense(*quantised(fmt, f64(t))) for t in (weight, x))
    size = np.abs(xq) @ np.abs(wq).T
    for more in (None, add):
        want = xq @ wq.T + (0 if more is None else f64(more))
        got = f64(p(x, add=more))
        assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -7) + K * 2.0 ** -23 * size).all()
    assert int(p.status.item()) == 0


@pytest.mark.parametrize("weights", ["nvfp4", "mxfp4"])
def test_decoder_block_with_4_bit_projections(example, weights):
    """The block's first half step: attention of the projections as they come out of the 4-bit products, then the 4-bit
    output projection onto the residual."""
    block = example.DecoderBlock("bf16", longest=40, page_size=16, weights=weights)
    T, Hq, Hkv, D = block.T, block.Hq, block.Hkv, block.D
    turn = block.rope.freqs.cpu().numpy().astype(np.float64) * (2 * np.pi / 2.0 ** 64)
    held = lambda y: f64(torch.from_numpy(y).to(torch.bfloat16))
    spin = lambda y, t: rotated(y, [t] * T, turn, "half", 1.0)
    g, qkvs = gen(1), []
    for step in range(20):
        x = bf16(g, T, block.cfg.H)
        y = block.step(x)
        qkvs.append(f64(block.qkv.out).reshape(T, Hq + 2 * Hkv, D))
        xq, wq = (dense(*quantised(weights, f64(t))) for t in (example.rms_norm(x), block.w_qkv))
        want = xq @ wq.T
        K = xq.shape[1]
        assert (np.abs(f64(block.qkv.out) - want) <= 2.0 ** -8 * np.abs(want) * 1.01 + K * 2.0 ** -23 * (np.abs(xq) @ np.abs(wq).T)).all()
    q = held(spin(qkvs[-1][:, :Hq], 19))
    k, v = np.stack([held(spin(z[:, Hq:Hq + Hkv], t)) for t, z in enumerate(qkvs)]), np.stack([z[:, Hq + Hkv:] for z in qkvs])
    att = np.zeros((T, Hq, D))
    for t in range(T):
        for h in range(Hq):
            s = k[:, t, h * Hkv // Hq] @ q[t, h] * D ** -0.5
            p = np.exp(s - s.max())
            att[t, h] = p @ v[:, t, h * Hkv // Hq] / p.sum()
    got = f64(block.attention.out)
    assert np.linalg.norm(got - att) <= 0.01 * np.linalg.norm(att)  # as the block's bf16 test
    oq, wq = dense(*quantised(weights, got.reshape(T, -1))), dense(*quantised(weights, f64(block.w_out)))
    want = oq @ wq.T + f64(x)
    assert (np.abs(f64(block.project.out) - want) <= 2.0 ** -8 * np.abs(want) * 1.01
            + oq.shape[1] * 2.0 ** -23 * (np.abs(oq) @ np.abs(wq).T)).all()
    assert not any(int(s.status.item()) for s in (block.attention, block.moe, block.qkv, block.project))
    assert torch.isfinite(y.float()).all()


def test_decoder_block_in_a_graph(example):
    """A captured step replayed gives what separate steps give, up to the experts' order between slot and pool."""
    one, two = (example.DecoderBlock("e4m3", longest=40, page_size=16, weights="nvfp4") for _ in range(2))
    x = bf16(gen(2), one.T, one.cfg.H)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        two.step(x)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            two.step(x)
        two.pos.zero_()
        for _ in range(15):
            graph.replay()
            one.step(x)
        side.synchronize()
    assert torch.equal(one.attention.out, two.attention.out) and torch.equal(one.project.out, two.project.out)


def test_attention_by_several_axes(pipeline):
    """DecodeAttention with positions of time, height and width that are not the cache's."""
    from quantized_expert_ffn_router_gb300 import attention as att

    T, Hq, Hkv, D, steps, sections = 3, 4, 2, 64, 9, (12, 10, 10)
    cache = att.KvCache(att.FT_KV_BF16, Hkv, D, 4, 3 * T)
    pages = torch.arange(3 * T, dtype=torch.int32, device=DEV).view(T, 3)
    spin = att.Rope(D, base=1e4, sections=sections, weave=True)
    layer = pipeline.DecodeAttention(cache, Hq, T, spin)
    freqs = spin.freqs.cpu().numpy().astype(np.float64) * (2 * np.pi / 2.0 ** 64)
    axis, r, g = axis_of(sections, True), np.random.default_rng(0), gen(3)
    ks, vs = [], []
    held = lambda y: f64(torch.from_numpy(y).to(torch.bfloat16))

    def turned(x, pos):
        y = np.array(x)
        for i, a in enumerate(axis):
            y[..., (i, i + D // 2)] = rotated(x, pos[a], np.where(np.arange(D // 2) == i, freqs, 0), "half", 1.0)[..., (i, i + D // 2)]
        return held(y)

    for step in range(steps):
        qkv, turns = bf16(g, T, (Hq + 2 * Hkv) * D), r.integers(0, 5000, (3, T))
        out = layer(qkv, pages, torch.full((T,), step, dtype=torch.int32, device=DEV),
                    rope_pos=torch.tensor(turns, dtype=torch.int32, device=DEV))
        x = f64(qkv).reshape(T, -1, D)
        q = turned(x[:, :Hq], turns)
        ks.append(turned(x[:, Hq:Hq + Hkv], turns))
        vs.append(x[:, Hq + Hkv:])
    k, v, got = np.stack(ks), np.stack(vs), f64(out).reshape(T, Hq, D)
    assert int(layer.status.item()) == 0
    for t in range(T):
        for h in range(Hq):
            s = k[:, t, h // 2] @ q[t, h] * D ** -0.5
            p = np.exp(s - s.max())
            p /= p.sum()
            want = p @ v[:, t, h // 2]
            # the output's rounding; scores off by the rounding of q and k at a border (2^-8 of 64 products' size at most)
            off = 2.0 ** -8 * np.abs(want) + 2 * 2.0 ** -8 * (np.abs(k[:, t, h // 2]) @ np.abs(q[t, h]) * D ** -0.5).max() * (
                p @ np.abs(v[:, t, h // 2]))
            assert (np.abs(got[t, h] - want) <= off).all()


def test_expert_blocks_from_weights(cuda_lib, fp4):
    """Blocks quantised from weights in place, read by the expert layer: its output is that of the values they stand for."""
    ft = cuda_lib
    H, I, E, T, k = 256, 128, 4, 3, 2
    total, _ = ft.block_bytes(ft.FT_NVFP4, H, I, 16)
    g = gen(5)
    blocks = torch.zeros(E, total + 16, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(E, 3, dtype=torch.float32, device=DEV)
    mats = []
    for e in range(E):
        ws = [torch.randn(n, m, generator=g, device=DEV) * m ** -0.5 for n, m in ((I, H), (I, H), (H, I))]
        scales[e] = torch.stack([w.abs().max() / 2688 for w in ws])
        views = fp4.expert_matrices(blocks[e], H, I, scales[e])
        for w, m in zip(ws, views):
            fp4.fp4_quantize(w, m, given=True)
            s = np.full(m.rows, f64(m.scale)[0])
            c, b, _ = quantised("nvfp4", f64(w), s)
            assert (codes_at(m).reshape(c.shape) == c).all() and (scales_at(m, "nvfp4") == b).all()
        mats.append([dense(*quantised("nvfp4", f64(w), np.full(len(w), f64(m.scale)[0]))[:2]) * f64(m.scale)[0]
                     for w, m in zip(ws, views)])
    assert (blocks[:, total:] == 0).all()
    bank = ft.make_bank(ft.FT_NVFP4, H, I, 16, blocks, scales)
    x = bf16(g, T, H)
    ids = torch.tensor([[0, 3], [2, 1], [3, 3]], dtype=torch.int32, device=DEV)[:, :k].contiguous()
    ids[2, 1] = 0
    w = torch.tensor([[0.7, 0.3], [0.5, 0.5], [0.9, 0.1]], dtype=torch.float32, device=DEV)
    out = torch.empty(T, H, dtype=torch.float32, device=DEV)
    ws = torch.zeros(ft.experts_workspace(ft.FT_DECODE, T, k, H, I, E), dtype=torch.uint8, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    ft.experts_fwd(bank, bank, 0, E, x.view(torch.int16), T, k, ids, ids, w, out, ws, dev_status=status)
    want = np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            gate, up, down = mats[int(ids[t, j])]
            a, b = gate @ f64(x)[t], up @ f64(x)[t]
            want[t] += float(w[t, j]) * (down @ (a / (1 + np.exp(-a)) * b))
    assert int(status.item()) == 0
    assert np.linalg.norm(f64(out) - want) <= 5e-3 * np.linalg.norm(want)  # the layer's own bound


def test_two_streams_and_captured_calls(fp4):
    """Products that run at once share nothing; graphs captured over the same matrices replay to the same bits."""
    sizes = [(5, 700, 2048), (300, 520, 1024), (64, 128, 4096), (1, 4096, 4096)]
    sets = [(random_matrix("nvfp4", T, K, i, plain=False), random_matrix("nvfp4", N, K, i + 9, plain=False),
             torch.zeros(T, N, device=DEV, dtype=torch.bfloat16)) for i, (T, N, K) in enumerate(sizes)]
    want = []
    for x, w, out in sets:
        fp4.fp4_matmul(x, w, out)
        want.append(out.clone())
        out.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(20):
        for (x, w, out), s in zip(sets, streams):
            fp4.fp4_matmul(x, w, out, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(out, y) for (_, _, out), y in zip(sets, want))
    graphs = []
    for (x, w, out), s in zip(sets, streams):
        out.zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            fp4.fp4_matmul(x, w, out)
        graphs.append(graph)
    for _ in range(10):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out, y) for (_, _, out), y in zip(sets, want))


def test_quantise_then_multiply_without_waiting(fp4):
    """Rows quantised over and over between products that read them."""
    g = gen(7)
    w = random_matrix("nvfp4", 640, 1024, 1)
    xs = [bf16(g, 70, 1024) for _ in range(6)]
    alone = []
    for x in xs:
        m = fp4.Fp4Matrix(FMT["nvfp4"], 70, 1024)
        fp4.fp4_quantize(x, m)
        out = torch.empty(70, 640, device=DEV)
        fp4.fp4_matmul(m, w, out)
        torch.cuda.synchronize()
        alone.append(out)
    m = fp4.Fp4Matrix(FMT["nvfp4"], 70, 1024)
    outs = [torch.empty(70, 640, device=DEV) for _ in xs]
    for x, out in zip(xs, outs):
        fp4.fp4_quantize(x, m)
        fp4.fp4_matmul(m, w, out)
    assert all(torch.equal(a, b) for a, b in zip(alone, outs))


def test_rows_past_32_bits(fp4):
    """Elements of x and of out past 2^32, bytes of codes past 2^31."""
    R, K = 70000, 65536
    x = torch.zeros(R, K, dtype=torch.bfloat16, device=DEV)
    rows = [0, 1, 65537, R - 129, R - 1]
    x[rows] = bf16(gen(9), len(rows), K)
    m = fp4.Fp4Matrix(FMT["nvfp4"], R, K)
    fp4.fp4_quantize(x, m)
    y = torch.empty_like(x)
    fp4.fp4_values(m, y)
    c, b, s = quantised("nvfp4", f64(x[rows]))
    want = dense(c, b, s)
    assert (np.abs(f64(y[rows]) - want) <= 2.0 ** -8 * np.abs(want)).all()
    assert float(y.float().abs().sum(-1).ne(0).sum()) == len(rows)
    del x, y, m
    T, N = 36000, 65600
    a, w = random_matrix("nvfp4", T, 32, 1), random_matrix("nvfp4", N, 32, 2)
    out = torch.zeros(T, N, dtype=torch.bfloat16, device=DEV)
    fp4.fp4_matmul(a, w, out)
    at = np.array([0, 32767, 32768, T - 1])
    want = multiplied(a, w, "nvfp4")[at]
    got = f64(out[torch.from_numpy(at).to(DEV)])
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want)).all()
