"""What is measured of the operators around a decoder block's dense projections:
microscaled 4-bit matrices (rows quantised and read back, and the product of two
such matrices, for prompts and for single tokens), and rotary positions with
several axes, by themselves and on the way into the key-value cache.

Each case is a dict of plain values.  `run` computes it in its plain form
(elementary torch operations; `own` false) or through the framework's
operators (`own` true).
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BLOCK = {"nvfp4": 16, "mxfp4": 32}  # values that share a block scale
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
E_MIN = -64  # the smallest exponent of a row's power-of-two scale


# ---------------------------------------------------------------------- cases
def listed():
    return [
        # a decode step's activations of one token: pure latency
        dict(name="quantise 1 x 2048", op="quantise", rows=1, K=2048, dtype="bf16", fmt="nvfp4", order="tiles", scale="rows"),
        # a long prompt's activations before a projection
        dict(name="quantise 8192 x 4096", op="quantise", rows=8192, K=4096, dtype="bf16", fmt="nvfp4", order="tiles",
             scale="rows"),
        # a ragged prompt, with power-of-two block scales
        dict(name="quantise 1237 x 2560 mxfp4", op="quantise", rows=1237, K=2560, dtype="f16", fmt="mxfp4", order="tiles",
             scale="none"),
        # the gate matrices of 32 experts, in the order of the expert blocks, with the tensors' scale given
        dict(name="quantise experts 20480 x 2560", op="quantise", rows=20480, K=2560, dtype="bf16", fmt="nvfp4",
             order="rows", scale="one"),
        # one token's query, key and value projection: latency
        dict(name="project 1, 2048 to 2560", op="product", T=1, N=2560, K=2048, dtype="bf16", fmt="nvfp4", add=False,
             chain=False),
        # a decode batch's output projection, onto the residual
        dict(name="project 8, 4096 to 4096 mxfp4", op="product", T=8, N=4096, K=4096, dtype="f16", fmt="mxfp4", add=True,
             chain=False),
        # a decode batch's logits
        dict(name="project 64, 2048 to 131072", op="product", T=64, N=131072, K=2048, dtype="bf16", fmt="nvfp4", add=False,
             chain=False),
        # a prompt of odd length, odd sizes everywhere
        dict(name="project 1237, 2592 to 5003", op="product", T=1237, N=5003, K=2592, dtype="bf16", fmt="nvfp4", add=False,
             chain=False),
        # a prompt's projection from its activations: quantised, multiplied, onto the residual
        dict(name="linear 2048, 4096 to 4096", op="product", T=2048, N=4096, K=4096, dtype="bf16", fmt="nvfp4", add=True,
             chain=True),
        # a long prompt's query, key and value projection
        dict(name="project 8192, 4096 to 6144", op="product", T=8192, N=6144, K=4096, dtype="bf16", fmt="nvfp4", add=False,
             chain=False),
        # queries of a prompt with an image in it: time, height and width woven over the channels
        dict(name="spin prompt 4099", op="spin", T=4099, heads=32, D=128, rot=128, layout="half", dtype="bf16",
             sections="24 20 20", weave=True, base=5e6, far=200000),
        # the decode step of a batch: rotate q and k by three axes in runs of channels, write k and v in 8 bits
        dict(name="append 16 rows", op="append", T=16, seqs=0, heads=16, kv=2, D=256, rot=64, layout="half", dtype="bf16",
             fmt="e4m3", page=16, sections="8 12 12", weave=False, base=1e7, far=30000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        c = _draw(rng)
        w = work(c)
        if w["flops"] <= 2.5e11 and w["bytes"] <= 2e8:
            return c


def _draw(rng):
    op = rng.choice(["quantise", "quantise", "product", "product", "product", "product", "spin", "append"])
    fmt = rng.choice(["nvfp4", "nvfp4", "mxfp4"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    B = BLOCK[fmt]
    if op == "quantise":
        K = B * _log(rng, 1, 16384 // B)
        order = rng.choice(["tiles", "tiles", "rows"])
        return dict(op=op, rows=_log(rng, 1, 16384), K=K, dtype=rng.choice([dtype, dtype, "f32"]), fmt=fmt, order=order,
                    scale="none" if fmt == "mxfp4" else rng.choice(["rows", "rows", "one"]))
    if op == "product":
        return dict(op=op, T=_log(rng, 1, 8192), N=_log(rng, 1, 32768), K=B * _log(rng, 1, 8192 // B), dtype=dtype,
                    fmt=fmt, add=rng.choice([False, True]), chain=rng.choice([False, True]))
    D = rng.choice([64, 96, 128, 128, 192, 256])
    rot = rng.choice([D, D, D // 2])
    n, half = rng.choice([2, 3, 3, 4]), rot // 2
    weave = rng.choice([False, True])
    if weave:  # the axes take turns; the first has what is left
        rest = [half // n - rng.choice([0, 0, 1, 2]) for _ in range(n - 1)]
        sections = [half - sum(rest)] + rest
    else:
        cut = sorted(rng.sample(range(1, half), n - 1))
        sections = [b - a for a, b in zip([0] + cut, cut + [half])]
    c = dict(op=op, heads=rng.choice([1, 3, 8, 16, 32, 40]), D=D, rot=rot, layout=rng.choice(["half", "half", "pairs"]),
             dtype=dtype, sections=" ".join(map(str, sections)), weave=weave, base=rng.choice([1e4, 1e6, 1e7]), far=_log(rng, 100, 1000000))
    if op == "spin":
        return dict(c, T=_log(rng, 1, 4099))
    T, kv = _log(rng, 1, 4099), rng.choice([1, 2, 4, 8])
    return dict(c, T=T, seqs=0 if T <= 64 else min(T, rng.choice([1, 2, 5])), kv=kv, heads=kv * rng.choice([1, 4, 5, 8]),
                fmt=rng.choice([dtype, "e4m3", "e4m3"]), page=rng.choice([1, 16, 24, 64]))


def _matrix_bytes(rows, K, fmt):
    return rows * (K // 2 + K // BLOCK[fmt]) + (4 * rows if fmt == "nvfp4" else 0)


def work(case):
    c = case
    if c["op"] == "quantise":  # written in 4 bits, and read back
        n = c["rows"] * c["K"]
        size = 4 if c["dtype"] == "f32" else 2
        return {"bytes": 2 * n * size + 2 * _matrix_bytes(c["rows"], c["K"], c["fmt"]), "flops": 4 * n}
    T = c["T"]
    if c["op"] == "product":
        x = T * c["K"] * 2 if c["chain"] else _matrix_bytes(T, c["K"], c["fmt"])
        return {"bytes": x + _matrix_bytes(c["N"], c["K"], c["fmt"]) + T * c["N"] * (4 if c["add"] else 2),
                "flops": 2 * T * c["N"] * c["K"]}
    n, axes = T * c["heads"] * c["D"], len(_sections(c))
    if c["op"] == "spin":
        return {"bytes": 4 * n + 4 * axes * T, "flops": 6 * T * c["heads"] * c["rot"] // 2}
    row = c["D"] + 1 if c["fmt"] == "e4m3" else 2 * c["D"]
    return {"bytes": 4 * n + 2 * T * c["kv"] * (2 * c["D"] + row) + 4 * (axes + 1) * T,
            "flops": 6 * T * (c["heads"] + c["kv"]) * c["rot"] // 2 + 4 * T * c["kv"] * c["D"]}


# -------------------------------------------------------- 4-bit matrices, plain
def _two(e):
    """2^e in 64 bits, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _round_float(y, mantissa, least, top):
    """y (64 bits) to the nearest value of a small float format, ties to even: `mantissa` bits after the point,
    2^least its smallest normal value, |y| held to `top`."""
    _, x = torch.frexp(y)
    q = _two((x - 1).clamp(min=least) - mantissa)
    return (torch.round(y / q) * q).clamp(-top, top)


def _pitch(K):
    return -(-K // 32) * 16  # bytes of a row of codes: whole 16 bytes


def _tile_at(rows, blocks):
    """Where block scale (r, b) lies: tiles of 128 rows x 4 block scales, 512 bytes each, those of the same rows one
    after the other; in a tile, row r's four scales are the word (r mod 32) * 4 + r / 32."""
    r, b = torch.arange(rows, device=DEV)[:, None], torch.arange(blocks, device=DEV)[None, :]
    tile = (r // 128) * -(-blocks // 4) + b // 4
    return tile * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4


def _empty_matrix(rows, K, fmt, order, scale):
    blocks = K // BLOCK[fmt]
    if order == "tiles":
        scales = torch.zeros(-(-rows // 128) * -(-blocks // 4) * 512, dtype=torch.uint8, device=DEV)
    else:
        scales = torch.zeros(rows, blocks, dtype=torch.uint8, device=DEV)
    m = dict(rows=rows, K=K, fmt=fmt, order=order, codes=torch.zeros(rows, _pitch(K), dtype=torch.uint8, device=DEV),
             scales=scales, scale=None)
    if scale != "none":
        m["scale"] = torch.ones(rows if scale == "rows" else 1, dtype=torch.float32, device=DEV)
    return m


def _quantise(x, m, given):
    """Rows x into the matrix m; in 64 bits, because values lie next to borders between codes."""
    rows, K, fmt = m["rows"], m["K"], m["fmt"]
    at = _tile_at(rows, K // BLOCK[fmt]) if m["order"] == "tiles" else None
    for r in range(0, rows, 4096):  # the intermediate values of a few rows at a time
        y = x[r:r + 4096].float()
        if fmt == "nvfp4":
            if given:
                z = (y * (1.0 / m["scale"])).double()
            else:
                # the smallest 2^e with max|x| <= 6 * 448 * 2^e
                f, e = torch.frexp(y.abs().amax(-1))
                e = torch.where(f > 0, e - 12 + (f > 0.65625).to(e.dtype), E_MIN).clamp(min=E_MIN)
                m["scale"][r:r + 4096] = _two(e).float()
                z = y.double() * _two(-e)[:, None]
            z = z.unflatten(-1, (-1, 16))
            b = _round_float(z.abs().amax(-1) / 6, 3, -6, 448.0)
            bits = b.to(torch.float8_e4m3fn).view(torch.uint8)
            z = torch.where(b[..., None] > 0, z / b[..., None], 0.0)
        else:
            z = y.double().unflatten(-1, (-1, 32))
            f, e = torch.frexp(z.abs().amax(-1))
            e = torch.where(f > 0, e - 3, -127).clamp(-127, 127)  # 2^(floor(log2 max) - 2)
            bits = (e + 127).to(torch.uint8)
            z = z * _two(-e)[..., None]
        code = _round_float(z, 1, 0, 6.0).flatten(-2)
        level = torch.bucketize(code.abs(), torch.tensor(E2M1, device=DEV, dtype=torch.float64)).to(torch.uint8)
        level |= torch.signbit(code).to(torch.uint8) << 3
        m["codes"][r:r + 4096, :K // 2] = level[:, 0::2] | (level[:, 1::2] << 4)
        if at is None:
            m["scales"][r:r + 4096] = bits
        else:
            m["scales"][at[r:r + 4096]] = bits


def _values(m):
    """What a matrix stands for, in 32 bits."""
    level = torch.tensor(E2M1 + [-v for v in E2M1], device=DEV)
    c = m["codes"][:, :m["K"] // 2]
    y = level[torch.stack((c & 15, c >> 4), -1).flatten(-2).int()]
    B = BLOCK[m["fmt"]]
    s = m["scales"][_tile_at(m["rows"], m["K"] // B)] if m["order"] == "tiles" else m["scales"]
    if m["fmt"] == "nvfp4":
        s = s.view(torch.float8_e4m3fn).float()
    else:
        s = _two(s.int() - 127).float()
    y = (y.unflatten(-1, (-1, B)) * s[..., None]).flatten(-2)
    return y if m["scale"] is None else y * m["scale"][:, None]


# --------------------------------------------------------------------- inputs
def _rand(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _acts(g, rows, K, dtype):
    """Activations: channels of uneven size, a few of them large, rows of uneven size."""
    chan = torch.exp(0.5 * _rand(g, 1, K)) * torch.where(torch.rand(1, K, generator=g, device=DEV) < 0.01, 8.0, 1.0)
    return (_rand(g, rows, K) * chan * torch.exp(0.3 * _rand(g, rows, 1))).to(DT[dtype])


def _weights(g, rows, K, fmt):
    """A projection's weights, laid out once."""
    m = _empty_matrix(rows, K, fmt, "tiles", "rows" if fmt == "nvfp4" else "none")
    w = torch.empty(rows, K, device=DEV).normal_(generator=g).mul_(K ** -0.5)
    _quantise(w.mul_(torch.exp(0.2 * _rand(g, rows, 1))), m, False)
    return m


def _heads(g, T, h, D, dtype, offset=0):
    """[T, h, D] as a slice of a wider projection row: channels of uneven size, tokens of uneven size."""
    wide = torch.zeros(T, offset + h * D, device=DEV, dtype=DT[dtype])
    x = wide[:, offset:].view(T, h, D)
    x.copy_((_rand(g, T, h, D) * torch.exp(0.5 * _rand(g, 1, h, D)) * torch.exp(0.3 * _rand(g, T, h, 1))).to(DT[dtype]))
    return x


def _sections(c):
    """How many channel pairs turn by each axis."""
    return [int(v) for v in c["sections"].split()]


def _axes_of(c):
    """The axis that each channel pair turns by: a run of pairs for each, or woven, where they take turns for as long
    as they have pairs left, and the first has the rest."""
    sections = _sections(c)
    n, half = len(sections), c["rot"] // 2
    if not c["weave"]:
        return np.repeat(np.arange(n), sections)
    i = np.arange(half)
    return np.where(i // n < np.array(sections)[i % n], i % n, 0)


def _inv_freq(c):
    """Radians a position, in 64 bits."""
    return c["base"] ** (-np.arange(0, c["rot"], 2, dtype=np.float64) / c["rot"])


def _positions(g, c):
    """[axes, T] positions of a sequence of text with images in it: text counts on every axis, an image's tokens stay
    at one time and count rows and columns."""
    T, n = c["T"], len(_sections(c))
    start = int(torch.randint(0, max(1, c["far"] - T), (1,), generator=g, device=DEV))
    at = torch.arange(T, device=DEV)
    wide = max(1, int(math.sqrt(T / 2)))
    inside = (at >= T // 4) & (at < T // 4 + T // 2)
    j = at - T // 4
    pos = torch.empty(n, T, dtype=torch.int32, device=DEV)
    for a in range(n):
        grid = T // 4 + (j // wide if a % 3 == 1 else j % wide if a % 3 == 2 else torch.zeros_like(j))
        pos[a] = start + torch.where(inside, grid, at)
    return pos


def _paged(g, need, total):
    """A page table over `total` shuffled pages for sequences of these many pages: [n, most], -1 past a sequence's."""
    need = torch.tensor(need, device=DEV)
    most = max(1, int(need.max()))
    at = torch.arange(most, device=DEV)[None, :]
    first = torch.cumsum(need, 0) - need
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    return torch.where(at < need[:, None], order[(first[:, None] + at).clamp(max=total - 1)], -1).to(torch.int32).contiguous()


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": c}
    if c["op"] == "quantise":
        s["x"] = _acts(g, c["rows"], c["K"], c["dtype"])
        s["m"] = _empty_matrix(c["rows"], c["K"], c["fmt"], c["order"], c["scale"])
        if c["scale"] == "one":
            s["m"]["scale"].copy_(s["x"].abs().amax().float() / 2688.0)
        s["values"] = torch.zeros(c["rows"], c["K"], device=DEV, dtype=DT[c["dtype"]])
        return s
    T = c["T"]
    if c["op"] == "product":
        s["w"] = _weights(g, c["N"], c["K"], c["fmt"])
        s["x"] = _acts(g, T, c["K"], c["dtype"])
        s["xq"] = _empty_matrix(T, c["K"], c["fmt"], "tiles", "rows" if c["fmt"] == "nvfp4" else "none")
        if not c["chain"]:
            _quantise(s["x"], s["xq"], False)
        s["add"] = _rand(g, T, c["N"]).to(DT[c["dtype"]]) if c["add"] else None
        s["out"] = torch.zeros(T, c["N"], device=DEV, dtype=DT[c["dtype"]])
        return s
    D = c["D"]
    s["inv_freq"] = torch.from_numpy(_inv_freq(c)).to(DEV)
    s["axes"] = torch.from_numpy(_axes_of(c)).to(DEV)
    s["turns"] = _positions(g, c)
    s["q"] = _heads(g, T, c["heads"], D, c["dtype"])
    s["q_out"] = torch.zeros(T, c["heads"], D, device=DEV, dtype=DT[c["dtype"]])
    if c["op"] == "spin":
        return s
    # one new token of each of T sequences, or T tokens of a few
    n = [1] * T if c["seqs"] == 0 else [T // c["seqs"] + (i < T % c["seqs"]) for i in range(c["seqs"])]
    first = torch.randint(0, 3 * c["page"], (len(n),), generator=g, device=DEV).tolist()
    total = T // c["page"] + 5 * len(n) + 3  # the same for every seed
    s["pages"] = _paged(g, [-(-(a + b) // c["page"]) for a, b in zip(first, n)], total)
    s["seq"] = torch.tensor(np.repeat(np.arange(len(n)), n), device=DEV, dtype=torch.int32)
    s["pos"] = torch.tensor(np.concatenate([np.arange(a, a + b) for a, b in zip(first, n)]), device=DEV, dtype=torch.int32)
    s["k"], s["v"] = _heads(g, T, c["kv"], D, c["dtype"], D), _heads(g, T, c["kv"], D, c["dtype"], 2 * D)
    shape = (total, c["kv"], c["page"])
    kind = torch.float8_e4m3fn if c["fmt"] == "e4m3" else DT[c["fmt"]]
    s["cache"] = {n: torch.zeros(*shape, D, dtype=kind, device=DEV) for n in ("k", "v")}
    if c["fmt"] == "e4m3":
        s["cache"] |= {n: torch.full(shape, 127, dtype=torch.uint8, device=DEV) for n in ("k_scale", "v_scale")}
    return s


# ------------------------------------------------------------- the plain form
def _rotate(x, s):
    """x [T, h, D] -> the rotated rows in 64 bits."""
    c, rot = s["case"], s["case"]["rot"]
    ang = (s["turns"].double()[s["axes"]] * s["inv_freq"][:, None]).t()
    cos, sin = torch.cos(ang)[:, None, :], torch.sin(ang)[:, None, :]
    y = x.double()
    out = y.clone()
    if c["layout"] == "pairs":
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        out[..., 0:rot:2], out[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        h = rot // 2
        a, b = y[..., :h], y[..., h:rot]
        out[..., :h], out[..., h:rot] = a * cos - b * sin, b * cos + a * sin
    return out


def _write(s, name, y):
    """Write the rows y [T, kv, D] (64 bits) into the cache's array `name`."""
    c, cache = s["case"], s["cache"]
    page = s["pages"][s["seq"].long(), (s["pos"] // c["page"]).long()].long()
    slot = (s["pos"] % c["page"]).long()
    if c["fmt"] != "e4m3":
        cache[name][page, :, slot] = y.to(DT[c["fmt"]])
        return
    f, e = torch.frexp(y.abs().amax(-1))
    e = torch.where(f > 0, e - 9 + (f > 0.875).to(e.dtype), E_MIN).clamp(min=E_MIN)
    code = _round_float(y * _two(-e)[..., None], 3, -6, 448.0)
    cache[name].view(torch.uint8)[page, :, slot] = code.to(torch.float8_e4m3fn).view(torch.uint8)
    cache[name + "_scale"][page, :, slot] = (e + 127).to(torch.uint8)


def _plain(s):
    c = s["case"]
    if c["op"] == "quantise":
        _quantise(s["x"], s["m"], c["scale"] == "one")
        out = {"values": _values(s["m"]).to(DT[c["dtype"]])}
        return out | {"scale": s["m"]["scale"]} if c["scale"] == "rows" else out
    if c["op"] == "product":
        if c["chain"]:
            _quantise(s["x"], s["xq"], False)
        y = torch.matmul(_values(s["xq"]), _values(s["w"]).t())
        if c["add"]:
            y += s["add"].float()
        return y.to(DT[c["dtype"]])
    q = _rotate(s["q"], s).to(DT[c["dtype"]])
    if c["op"] == "spin":
        return q
    _write(s, "k", _rotate(s["k"], s))
    _write(s, "v", s["v"].double())
    return {"q": q} | s["cache"]


# --------------------------------------------------------- the framework's own
def _handles(s):
    """What a user's program makes once: the matrices' descriptors, the rotary table, the cache's descriptor."""
    from quantized_expert_ffn_router_gb300 import attention as att
    from quantized_expert_ffn_router_gb300 import fp4

    c = s["case"]
    h = {"att": att, "fp4": fp4}
    fmt = {"nvfp4": fp4.FT_FP4_NVFP4, "mxfp4": fp4.FT_FP4_MXFP4}
    order = {"tiles": fp4.FT_FP4_TILES, "rows": fp4.FT_FP4_ROWS}
    for n in ("m", "w", "xq"):
        if n in s:
            m = s[n]
            h[n] = fp4.Fp4Matrix.over(fmt[m["fmt"]], m["K"], m["codes"], m["scales"], scale=m["scale"],
                                      order=order[m["order"]])
    if "turns" in s:
        h["rope"] = att.Rope(c["rot"], base=c["base"], interleaved=c["layout"] == "pairs", sections=_sections(c),
                             weave=c["weave"])
    if "cache" in s:
        kind = {"bf16": att.FT_KV_BF16, "f16": att.FT_KV_F16, "e4m3": att.FT_KV_E4M3}
        h["cache"] = att.KvCache.over(kind[c["fmt"]], c["D"], **s["cache"])
    h["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    return h


def _own(s):
    c = s["case"]
    h = s.get("handles")
    if h is None:
        h = s["handles"] = _handles(s)
    att, fp4 = h["att"], h["fp4"]
    if c["op"] == "quantise":
        fp4.fp4_quantize(s["x"], h["m"], given=c["scale"] == "one")
        fp4.fp4_values(h["m"], s["values"])
        out = {"values": s["values"]}
        return out | {"scale": s["m"]["scale"]} if c["scale"] == "rows" else out
    if c["op"] == "product":
        if c["chain"]:
            fp4.fp4_quantize(s["x"], h["xq"])
        fp4.fp4_matmul(h["xq"], h["w"], s["out"], add=s["add"], dev_status=h["status"])
        return s["out"]
    if c["op"] == "spin":
        att.rope(s["q"], s["turns"], h["rope"], s["q_out"])
        return s["q_out"]
    att.kv_append(h["cache"], s["k"], s["v"], s["pages"], s["pos"], seq=s["seq"], rope=h["rope"], rope_pos=s["turns"],
                  q=s["q"], q_out=s["q_out"], dev_status=h["status"])
    return {"q": s["q_out"]} | s["cache"]


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------- the 64-bit answers
def _levels(name):
    if name == "e2m1":
        lev = E2M1
    else:  # e4m3
        lev = [i / 8 * 2.0 ** -6 for i in range(8)] + [(1 + i / 8) * 2.0 ** x for x in range(-6, 9) for i in range(8)][:119]
    return torch.tensor(lev, dtype=torch.float64, device=DEV)


def _nearest(lev, y):
    """The level nearest to each |y|, ties to the even index, at most the last."""
    mid = (lev[1:] + lev[:-1]) / 2
    a = torch.searchsorted(mid, y.abs().contiguous())
    b = torch.searchsorted(mid, y.abs().contiguous(), right=True)
    return lev[torch.where(a % 2 == 0, a, b)]


def _coded(x, fmt, scale):
    """(values, row scales) of rows x, quantised from the definition; `scale`: the tensor's, or None."""
    four = _levels("e2m1")
    y = x.double()
    if fmt == "mxfp4":
        y = y.unflatten(-1, (-1, 32))
        most = y.abs().amax(-1, keepdim=True)
        e = torch.floor(torch.log2(most))
        e = torch.where(torch.exp2(e) > most, e - 1, torch.where(torch.exp2(e + 1) <= most, e + 1, e))
        s = torch.where(most > 0, torch.exp2((e - 2).clamp(-127, 127)), 2.0 ** -127)
        return (torch.sign(y) * _nearest(four, y / s) * s).flatten(-2), None
    if scale is None:
        most = y.abs().amax(-1, keepdim=True)
        e = torch.ceil(torch.log2(most / 2688.0)).clamp(min=E_MIN)
        e = torch.where(most > 2688.0 * torch.exp2(e), e + 1, e)
        e = torch.where((most <= 2688.0 * torch.exp2(e - 1)) & (e > E_MIN), e - 1, e)
        r = torch.exp2(e)
        z = y / r
    else:
        # the tensor's scale divides as a product with its reciprocal, each rounded to 32 bits
        inv = (1.0 / scale.double()).float().double()
        z, r = (y * inv).float().double(), scale.double()
    z = z.unflatten(-1, (-1, 16))
    b = _nearest(_levels("e4m3"), z.abs().amax(-1, keepdim=True) / 6)
    code = torch.where(b > 0, torch.sign(z) * _nearest(four, z / torch.where(b > 0, b, 1.0)), 0.0)
    return (code * b).flatten(-2) * r, r


def _decoded(m):
    """A matrix's values in 64 bits."""
    c = m["codes"][:, :m["K"] // 2].long()
    nib = torch.empty(m["rows"], m["K"], dtype=torch.long, device=DEV)
    nib[:, 0::2], nib[:, 1::2] = c % 16, c // 16
    k = nib % 8
    mag = torch.where(k < 2, k * 0.5, (1 + (k % 2) * 0.5) * torch.exp2((k // 2 - 1).double()))
    y = torch.where(nib >= 8, -mag, mag)
    B = BLOCK[m["fmt"]]
    nb = m["K"] // B
    # the tiles in memory order: [row tile][scale tile][row mod 32][row / 32][scale]
    t = m["scales"].view(-(-m["rows"] // 128), -(-nb // 4), 32, 4, 4).permute(0, 3, 2, 1, 4)
    s = t.reshape(t.shape[0] * 128, -1)[:m["rows"], :nb].long()
    if m["fmt"] == "nvfp4":
        f, x = s % 8, s // 8 % 16
        s = torch.where(x == 0, f * 2.0 ** -9, (8 + f) * torch.exp2((x - 10).double()))
    else:
        s = torch.exp2((s - 127).double())
    y = y * s.repeat_interleave(B, -1)
    return y if m["scale"] is None else y * m["scale"].double()[:, None]


def _spun(x, s):
    c = s["case"]
    rot, half = c["rot"], c["rot"] // 2
    out = x.detach().cpu().double().numpy()
    pos = s["turns"].cpu().numpy().astype(np.float64)
    w = np.exp(1j * np.stack([pos[a] * f for a, f in zip(_axes_of(c), _inv_freq(c))], -1))[:, None, :]
    if c["layout"] == "pairs":
        z = (out[..., 0:rot:2] + 1j * out[..., 1:rot:2]) * w
        out[..., 0:rot:2], out[..., 1:rot:2] = z.real, z.imag
    else:
        z = (out[..., :half] + 1j * out[..., half:rot]) * w
        out[..., :half], out[..., half:rot] = z.real, z.imag
    return out


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "quantise":
        values, scale = _coded(s["x"], c["fmt"], s["m"]["scale"] if c["scale"] == "one" else None)
        out = {"values": values.cpu().numpy()}
        return out | {"scale": scale.cpu().numpy()[:, 0]} if c["scale"] == "rows" else out
    if c["op"] == "product":
        x = _coded(s["x"], c["fmt"], None)[0] if c["chain"] else _decoded(s["xq"])
        y = x @ _decoded(s["w"]).t()
        if c["add"]:
            y += s["add"].double()
        return y.cpu().numpy()
    q = _spun(s["q"], s)
    if c["op"] == "spin":
        return q
    page = s["pages"][s["seq"].long(), (s["pos"] // c["page"]).long()].cpu().numpy()
    slot = (s["pos"] % c["page"]).cpu().numpy()
    out = {"q": q}
    for n, y in (("k", _spun(s["k"], s)), ("v", s["v"].detach().cpu().double().numpy())):
        full = np.zeros(tuple(s["cache"][n].shape))
        if c["fmt"] == "e4m3":
            most = np.abs(y).max(-1)
            with np.errstate(divide="ignore"):
                e = np.maximum(np.ceil(np.log2(most / 448.0)), E_MIN)
            e = np.where(most > 448.0 * 2.0 ** e, e + 1, np.where((most <= 448.0 * 2.0 ** (e - 1)) & (e > E_MIN), e - 1, e))
            z = torch.from_numpy(y / 2.0 ** e[..., None]).to(DEV)
            y = (torch.sign(z) * _nearest(_levels("e4m3"), z)).cpu().numpy()
            sc = np.full(tuple(s["cache"][n + "_scale"].shape), 127, np.uint8)
            sc[page, :, slot] = (e + 127).astype(np.uint8)
            out[n + "_scale"] = sc
        full[page, :, slot] = y
        out[n] = full
    return out
