"""The attention operators' arguments and build, as far as they need no GPU:
what is refused before a kernel could see it, and what is not."""

import os
import re

import pytest
import torch

from conftest import ROOT

CSRC = os.path.join(ROOT, "quantized_expert_ffn_router_gb300", "csrc")


def test_every_header_is_a_dependency_of_the_build():
    """What a source includes from the tree makes its object stale."""
    from quantized_expert_ffn_router_gb300 import build as b

    known = {os.path.basename(h) for h in b.headers()}
    for name in os.listdir(CSRC):
        if name.endswith((".cu", ".cuh", ".h")):
            text = open(os.path.join(CSRC, name)).read()
            for inc in re.findall(r'^\s*#\s*include\s+"([^"]+)"', text, flags=re.M):
                assert os.path.basename(inc) in known, (name, inc)


@pytest.fixture(scope="module")
def att():
    from quantized_expert_ffn_router_gb300 import build as b

    b.build()
    from quantized_expert_ffn_router_gb300 import attention

    attention._bind()
    return attention


def refused(call, *a, status=1, **kw):
    with pytest.raises(Exception) as e:
        call(*a, **kw)
    assert getattr(e.value, "status", None) == status, e.value
    return str(e.value)


def cpu_call(att, T=2, D=64):
    """The arguments of calls that would be right but for where they are."""
    rows = lambda h: torch.zeros(T, h, D, dtype=torch.bfloat16)
    ints = lambda *s: torch.zeros(*s, dtype=torch.int32)
    return dict(cache=att.KvCache(att.FT_KV_BF16, 2, D, 16, 4, device="cpu"), q=rows(4), k=rows(2), v=rows(2),
                out=rows(4), pages=ints(T, 3), pos=ints(T), spin=att.Rope(D, device="cpu"),
                ws=torch.zeros(1 << 24, dtype=torch.uint8))


@pytest.mark.parametrize("stream", [None, 0])
def test_tensors_that_are_not_on_a_gpu_are_refused(att, stream):
    x, kw = cpu_call(att), dict(stream=stream)
    for message in (refused(att.rope, x["q"], x["pos"], x["spin"], x["out"], **kw),
                    refused(att.kv_append, x["cache"], x["k"], x["v"], x["pages"], x["pos"], **kw),
                    refused(att.kv_append, x["cache"], x["k"], x["v"], x["pages"], x["pos"], rope=x["spin"], q=x["q"],
                            q_out=x["out"], **kw),
                    refused(att.kv_gather, x["cache"], x["pages"], x["pos"], x["k"], None, **kw),
                    refused(att.attn_decode, x["cache"], x["q"], x["pages"], x["pos"], x["out"], x["ws"], **kw)):
        assert "GPU" in message
    # a call of no tokens reads nothing
    x = cpu_call(att, T=0)
    pages = torch.zeros(1, 3, dtype=torch.int32)
    att.rope(x["q"], x["pos"], x["spin"], x["out"], **kw)
    att.kv_append(x["cache"], x["k"], x["v"], pages, x["pos"], **kw)
    att.kv_gather(x["cache"], pages, x["pos"], x["k"], None, **kw)
    att.attn_decode(x["cache"], x["q"], pages, x["pos"], x["out"], x["ws"], **kw)


def test_buffers_that_are_smaller_than_they_seem_are_refused(att):
    x = cpu_call(att)
    args = [x[n] for n in ("cache", "q", "pages", "pos", "out")]
    assert "ws" in refused(att.attn_decode, *args, torch.zeros(1, dtype=torch.uint8).expand(1 << 24))
    for status in (torch.zeros(1, dtype=torch.int8), torch.zeros(1, dtype=torch.int64), torch.zeros(0, dtype=torch.int32)):
        assert "dev_status" in refused(att.attn_decode, *args, x["ws"], dev_status=status)
        assert "dev_status" in refused(att.kv_append, x["cache"], x["k"], x["v"], x["pages"], x["pos"], dev_status=status)
        assert "dev_status" in refused(att.kv_gather, x["cache"], x["pages"], x["pos"], x["k"], None, dev_status=status)


@pytest.mark.gpu
def test_one_tensor_elsewhere_is_refused(cuda_lib, att):
    """Each argument in turn on the host, the others on the GPU: the library is not given its address."""
    cpu = cpu_call(att)
    gpu = {n: t.cuda() for n, t in cpu.items() if isinstance(t, torch.Tensor)}
    gpu |= dict(cache=att.KvCache(att.FT_KV_BF16, 2, 64, 16, 4), spin=att.Rope(64))
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)
    cpu |= dict(seq=i32(2), rope_pos=i32(2), status=i32(1), lse=torch.zeros(2, 4))
    gpu |= {n: cpu[n].cuda() for n in ("seq", "rope_pos", "status", "lse")}
    calls = {
        "rope": (("q", "pos", "spin", "out"), lambda x: att.rope(x["q"], x["pos"], x["spin"], x["out"])),
        "append": (("cache", "k", "v", "pages", "pos", "seq", "spin", "rope_pos", "q", "out", "status"),
                   lambda x: att.kv_append(x["cache"], x["k"], x["v"], x["pages"], x["pos"], seq=x["seq"], rope=x["spin"],
                                           rope_pos=x["rope_pos"], q=x["q"], q_out=x["out"], dev_status=x["status"])),
        "gather": (("cache", "pages", "pos", "k", "v", "seq", "status"),
                   lambda x: att.kv_gather(x["cache"], x["pages"], x["pos"], x["k"], x["v"], seq=x["seq"],
                                           dev_status=x["status"])),
        "decode": (("cache", "q", "pages", "pos", "out", "ws", "seq", "lse", "status"),
                   lambda x: att.attn_decode(x["cache"], x["q"], x["pages"], x["pos"], x["out"], x["ws"], seq=x["seq"],
                                             lse=x["lse"], dev_status=x["status"]))}
    gpu["pos"][1] = 1  # two places
    for names, call in calls.values():
        call(gpu)
        for n in names:
            assert "GPU" in refused(call, gpu | {n: cpu[n]}), n
    k = gpu["cache"].k
    assert "the keys are on" in refused(att.KvCache.over, att.FT_KV_BF16, 64, k, k.cpu())
    torch.cuda.synchronize()


def test_page_tables_of_one_page(att):
    """A transposed [1, n] table is contiguous as [n, 1] and keeps its strides (1, n)."""
    x = cpu_call(att, T=4)
    x["pages"] = torch.arange(4, dtype=torch.int32).view(1, 4).t().contiguous()
    assert x["pages"].stride() == (1, 4)
    message = refused(att.kv_gather, x["cache"], x["pages"], x["pos"], x["k"], None)
    assert "GPU" in message and "pages" not in message
    for bad in (torch.zeros(2, 8, dtype=torch.int32)[:, ::2], torch.zeros(8, dtype=torch.int32)):
        assert "pages" in refused(att.kv_gather, x["cache"], bad, x["pos"], x["k"], None)


@pytest.mark.gpu
def test_a_decoder_block_of_one_page_a_sequence(cuda_lib):
    """The example with sequences that end inside their first page."""
    import sys

    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import decoder_block

    block = decoder_block.DecoderBlock("bf16", longest=10, page_size=16)
    x = torch.randn(block.T, block.cfg.H, device="cuda").to(torch.bfloat16)
    for _ in range(10):
        y = block.step(x)
    assert int(block.attention.status.item()) == 0 and torch.isfinite(y.float()).all()
    assert block.cache.k[:block.T, :, :10].float().abs().sum((1, 3)).min() > 0  # every sequence's ten places are written
    assert not block.cache.k[:, :, 10:].any()


@pytest.mark.parametrize("shape", [(0, 3), (0, 0), (2, 0)])
def test_no_tokens_need_no_page_table(att, shape):
    x, pages = cpu_call(att, T=0), torch.zeros(shape, dtype=torch.int32)
    att.kv_append(x["cache"], x["k"], x["v"], pages, x["pos"], stream=0)
    att.kv_gather(x["cache"], pages, x["pos"], x["k"], x["v"], stream=0)
    att.attn_decode(x["cache"], x["q"], pages, x["pos"], x["out"], x["ws"], stream=0)
    x = cpu_call(att)
    assert "bad page table" in refused(att.kv_append, x["cache"], x["k"], x["v"], pages, x["pos"], stream=0)


def test_cache_arrays_of_another_floating_type_are_refused(att):
    z = lambda dtype, *s: torch.zeros(*s, dtype=torch.uint8).to(dtype) if dtype.itemsize > 1 else torch.zeros(
        *s, dtype=torch.uint8).view(dtype)
    rows = lambda dtype: dict(k=z(dtype, 2, 1, 4, 32), v=z(dtype, 2, 1, 4, 32))
    scales = lambda dtype: dict(k_scale=z(dtype, 2, 1, 4), v_scale=z(dtype, 2, 1, 4))
    blocks = lambda dtype: dict(k_block=z(dtype, 2, 1, 4, 4), v_block=z(dtype, 2, 1, 4, 4))
    e4, e5, e8, u8 = torch.float8_e4m3fn, torch.float8_e5m2, torch.float8_e8m0fnu, torch.uint8
    for fmt, dtype, other in ((att.FT_KV_BF16, torch.bfloat16, torch.float16), (att.FT_KV_F16, torch.float16, torch.bfloat16)):
        for fine in (dtype, torch.int16, torch.uint16):
            att.KvCache.over(fmt, 32, **rows(fine))
        assert "cache k" in refused(att.KvCache.over, fmt, 32, **rows(other))
    for codes, scale in ((e4, u8), (u8, e8), (torch.int8, u8)):
        att.KvCache.over(att.FT_KV_E4M3, 32, **rows(codes), **scales(scale))
    assert "cache k" in refused(att.KvCache.over, att.FT_KV_E4M3, 32, **rows(e5), **scales(u8))
    assert "cache k_scale" in refused(att.KvCache.over, att.FT_KV_E4M3, 32, **rows(e4), **scales(e4))
    for codes, block in ((u8, u8), (torch.float4_e2m1fn_x2, e4)):
        att.KvCache.over(att.FT_KV_NVFP4, 64, **rows(codes), **scales(u8), **blocks(block))
    assert "cache k_block" in refused(att.KvCache.over, att.FT_KV_NVFP4, 64, **rows(u8), **scales(u8), **blocks(e5))
