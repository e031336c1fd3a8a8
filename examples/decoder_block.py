"""A decoder block's decode step: attention over a paged, quantised key-value
cache, then the routed, quantised expert layer, captured into one CUDA graph
that serves the sequences as they grow.

    python examples/decoder_block.py [--cache bf16|e4m3|nvfp4] [--weights bf16|nvfp4|mxfp4] [--steps N]

Sizes are those of the tiny expert layer (synth.TINY) with 8 query heads over
2 key heads of 64 channels; weights and inputs are random.
"""

from __future__ import annotations

import argparse
import os
import sys
import time

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import quantized_expert_ffn_router_gb300 as ft  # noqa: E402
import synth  # noqa: E402
from quantized_expert_ffn_router_gb300 import attention as att, fp4  # noqa: E402
from quantized_expert_ffn_router_gb300.pipeline import DecodeAttention, DecodeLayer, Projection  # noqa: E402

FORMATS = {"bf16": att.FT_KV_BF16, "e4m3": att.FT_KV_E4M3, "nvfp4": att.FT_KV_NVFP4}
WEIGHTS = {"bf16": None, "nvfp4": fp4.FT_FP4_NVFP4, "mxfp4": fp4.FT_FP4_MXFP4}


def rms_norm(x):
    y = x.float()
    return (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


class DecoderBlock:
    """One block for T sequences of up to `longest` tokens, its weights random from `seed`; the projections around the
    attention in bf16, or in 4 bits (with the rows in front of them quantised each step)."""

    def __init__(self, cache_format="e4m3", longest=4096, page_size=64, Hq=8, Hkv=2, D=64, seed=0, device="cuda",
                 weights="bf16"):
        cfg = synth.get_config("tiny")
        self.cfg, T, H = cfg, cfg.tokens[0], cfg.H
        self.T, self.Hq, self.Hkv, self.D = T, Hq, Hkv, D
        g = torch.Generator(device=device).manual_seed(seed)
        weight = lambda n, m: (torch.randn(n, m, generator=g, device=device) / m ** 0.5).to(torch.bfloat16)
        self.w_qkv, self.w_out = weight((Hq + 2 * Hkv) * D, H), weight(H, Hq * D)
        self.qkv = self.project = None
        if WEIGHTS[weights] is not None:
            self.qkv, self.project = (Projection(w, T, WEIGHTS[weights]) for w in (self.w_qkv, self.w_out))
        # attention: a cache whose pages are handed out to the sequences in turn
        per = -(-longest // page_size)
        self.cache = att.KvCache(FORMATS[cache_format], Hkv, D, page_size, T * per, device=device)
        self.pages = torch.arange(T * per, dtype=torch.int32, device=device).view(per, T).t().contiguous()
        self.rope = att.Rope(D, base=5e5, scaling=att.FT_ROPE_PARTS_BY_TURNS, factor=8.0, device=device)
        self.attention = DecodeAttention(self.cache, Hq, T, self.rope, device=device)
        # experts: every block in the pool, and in as many cache slots as the configuration has
        pool = torch.stack([torch.from_numpy(synth.bank_block_np(cfg.seed, e, cfg.fmt, H, cfg.I, cfg.g))
                            for e in range(cfg.E)]).to(device)
        self.pool_blocks = pool
        self.slot_blocks = torch.zeros((cfg.slots, pool.shape[1]), dtype=torch.uint8, device=device)
        self.router = torch.from_numpy(synth.router_weights(cfg.seed, 0, cfg.E, H, cfg.router_std)).to(device)
        self.state = ft.DeviceCacheState(1, cfg.E, cfg.slots, device=device)
        self.moe = DecodeLayer(self.state, ft.make_bank(cfg.fmt, H, cfg.I, cfg.g, self.slot_blocks),
                               ft.make_bank(cfg.fmt, H, cfg.I, cfg.g, pool), cfg.E, cfg.k, T, device=device)
        self.moe_out = torch.empty((T, H), dtype=torch.bfloat16, device=device)
        self.pos = torch.zeros(T, dtype=torch.int32, device=device)

    def step(self, x):
        """x [T, H] bf16 -> [T, H]: attention, then experts, each around a residual; the sequences grow by a token."""
        if self.qkv is None:
            qkv = rms_norm(x) @ self.w_qkv.t()
            x = x + self.attention(qkv, self.pages, self.pos) @ self.w_out.t()
        else:
            x = self.project(self.attention(self.qkv(rms_norm(x)), self.pages, self.pos), add=x)
        # the library reads bf16 as bit patterns
        self.moe(0, rms_norm(x).view(torch.int16), self.router, self.cfg.phis[0], self.moe_out.view(torch.int16),
                 overlapped=False)
        self.pos.add_(1)
        return x + self.moe_out


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--cache", choices=sorted(FORMATS), default="e4m3")
    ap.add_argument("--weights", choices=sorted(WEIGHTS), default="bf16")
    ap.add_argument("--steps", type=int, default=1000)
    a = ap.parse_args()
    block = DecoderBlock(a.cache, longest=a.steps + 8, weights=a.weights)
    x = torch.randn(block.T, block.cfg.H, device="cuda").to(torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block.step(x)  # loads the kernels
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            y = block.step(x)
        block.pos.zero_()
        side.synchronize()
        t0 = time.perf_counter()
        for _ in range(a.steps):
            graph.replay()
        side.synchronize()
        seconds = time.perf_counter() - t0
    bad = int(block.attention.status.item()) or int(block.moe.status.item())
    if block.qkv is not None:
        bad = bad or int(block.qkv.status.item()) or int(block.project.status.item())
    print(f"{block.T} sequences to {int(block.pos[0].item())} tokens, {a.cache} cache, {a.weights} projections: "
          f"{a.steps / seconds:.0f} steps/s, "
          f"status {bad}, |y| {float(y.float().norm()):.3f}")
    return 1 if bad else 0


if __name__ == "__main__":
    sys.exit(main())
