"""The library's operators around a 4-bit KV cache, in a plain form and through the library.

The path of a serving step over a cache held in 4 bits, operator by operator:

* ``rotary``  norms of queries and keys per head and their rotation by position, in one call
* ``cache``   new K/V rows quantised into the paged cache, and each sequence's history read back
* ``decode``  one query token per sequence over the 4-bit cache
* ``prompt``  causal attention of packed prompts (or of chunks after a history), grouped heads

``run`` computes them with elementary torch operations while ``own`` is false, and with the
library's calls where it is true.

The 4-bit cache.  A (block, kv head) holds block / 16 tiles of 16 rows.  A tile is 16 x dim/2
bytes of codes (element 2j of a row in the low nibble of byte j, element 2j+1 in the high one)
followed by 16 x dim/16 bytes of e4m3 scales, one per 16 elements of a row.  A code is e2m1
(sign, 2 exponent bits, 1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6); the value of an element is
code * scale of its 16 * scale of its kv head.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------

def listed():
    return [
        # one decode step of a 7B-shaped model with 64 running sequences: pure latency
        dict(name="rotary_step", op="rotary", tokens=64, far=2048, heads=28, kv_heads=4, dim=128, rot=128,
             layout="half", scaling="none", norm=True, dtype="bf16"),
        # a chunked-prefill step: 512 prompt rows and 128 decodes in one batch
        dict(name="rotary_mixed", op="rotary", tokens=640, far=4096, heads=28, kv_heads=4, dim=128, rot=128,
             layout="half", scaling="linear", norm=True, dtype="bf16"),
        # long prompts at far positions, part of the head rotated, frequencies scaled by parts
        dict(name="rotary_prompt", op="rotary", tokens=16381, far=131072, heads=32, kv_heads=8, dim=128, rot=64,
             layout="interleaved", scaling="parts", norm=False, dtype="f16"),
        # a handful of short sequences gets its newest token and is read back
        dict(name="cache_small", op="cache", seqs=4, low=6, high=37, pick=1, new=1, kv_heads=4, dim=64,
             dtype="f16", block=16, scaled=False),
        # a 512-row chunk goes into the cache, and its 4-bit history comes back for the chunk's attention
        dict(name="cache_chunk", op="cache", seqs=1, low=4096, high=4096, pick=1, new=512, kv_heads=4, dim=128,
             dtype="bf16", block=16, scaled=True),
        # the chunks of several long prompts at once
        dict(name="cache_prompts", op="cache", seqs=8, low=9000, high=16384, pick=3, new=4096, kv_heads=8, dim=128,
             dtype="bf16", block=32, scaled=True),
        # the smallest decode: four short sequences, one query head per kv head
        dict(name="decode_small", op="decode", seqs=4, low=6, high=37, pick=1, heads=4, kv_heads=4, dim=64,
             dtype="f16", block=16, scaled=False),
        # the 7B-shaped decode batch
        dict(name="decode_batch", op="decode", seqs=64, low=128, high=2048, pick=2, heads=28, kv_heads=4, dim=128,
             dtype="bf16", block=16, scaled=True),
        # few sequences with long contexts
        dict(name="decode_long", op="decode", seqs=8, low=32768, high=131072, pick=4, heads=32, kv_heads=8, dim=128,
             dtype="bf16", block=16, scaled=True),
        # a 512-row chunk after 3584 tokens of history
        dict(name="prompt_chunk", op="prompt", seqs=1, low=512, high=512, pick=1, before=3584, heads=28, kv_heads=4,
             dim=128, dtype="bf16", packed=False),
        # ragged prompts packed into one batch
        dict(name="prompt_packed", op="prompt", seqs=16, low=64, high=2048, pick=5, before=0, heads=28, kv_heads=4,
             dim=128, dtype="bf16", packed=True),
        # one long prompt
        dict(name="prompt_long", op="prompt", seqs=1, low=8192, high=8192, pick=1, before=0, heads=32, kv_heads=8,
             dim=128, dtype="bf16", packed=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rotary", "cache", "decode", "prompt"))
    dtype = rng.choice(("bf16", "f16"))
    if op == "rotary":
        kv = rng.choice((1, 2, 4, 8))
        dim = rng.choice((64, 80, 96, 128, 256))
        heads = kv * rng.randint(1, 8)
        tokens = _log_int(rng, 1, max(1, 16381 * 40 * 128 // ((heads + kv) * dim)))
        return dict(op=op, tokens=min(tokens, 16381), far=_log_int(rng, 64, 1 << 20), heads=heads, kv_heads=kv, dim=dim,
                    rot=16 * rng.randint(1, dim // 16), layout=rng.choice(("half", "interleaved")),
                    scaling=rng.choice(("none", "linear", "ntk", "parts")), norm=rng.random() < 0.5, dtype=dtype)
    if op == "cache":
        seqs = _log_int(rng, 1, 64)
        high = _log_int(rng, 1, 60000 // seqs)
        return dict(op=op, seqs=seqs, low=max(1, high // rng.randint(1, 8)), high=high, pick=rng.randrange(1 << 20),
                    new=_log_int(rng, 1, 4096), kv_heads=rng.randint(1, 8), dim=rng.choice((64, 128)), dtype=dtype,
                    block=rng.choice((16, 32)), scaled=rng.random() < 0.5)
    if op == "decode":
        seqs = _log_int(rng, 1, 256)
        high = _log_int(rng, 1, min(131072, 560000 // seqs))
        kv = rng.randint(1, 8)
        return dict(op=op, seqs=seqs, low=max(1, high // rng.randint(1, 8)), high=high, pick=rng.randrange(1 << 20),
                    heads=kv * rng.randint(1, 8), kv_heads=kv, dim=rng.choice((64, 128)), dtype=dtype,
                    block=rng.choice((16, 32)), scaled=rng.random() < 0.5)
    seqs = _log_int(rng, 1, 32)
    high = _log_int(rng, 1, int(6000 / math.sqrt(seqs)))
    kv = rng.choice((1, 2, 4))
    return dict(op="prompt", seqs=seqs, low=max(1, high // rng.randint(1, 8)), high=high, pick=rng.randrange(1 << 20),
                before=rng.choice((0, 0, rng.randint(0, high // 2))), heads=kv * rng.randint(1, 7), kv_heads=kv,
                dim=rng.choice((64, 128)), dtype=dtype, packed=False)


def _lens(c):
    """The sequences' lengths: fixed by the case."""
    r = random.Random(c["pick"])
    return [r.randint(c["low"], c["high"]) for _ in range(c["seqs"])]


def work(c):
    d = c["dim"]
    if c["op"] == "rotary":
        n = c["tokens"] * (c["heads"] + c["kv_heads"]) * d
        return {"bytes": 4 * n + 4 * c["tokens"], "flops": n * (3 + (5 if c["norm"] else 0))}
    lens = _lens(c)
    total = sum(lens)
    tables = 4 * sum(-(-n // c.get("block", 16)) for n in lens)
    if c["op"] == "cache":
        new = sum(min(n, c["new"]) for n in lens)
        row, packed = 2 * c["kv_heads"] * d * 2, 2 * c["kv_heads"] * d * 9 // 16
        return {"bytes": new * (row + packed + 8) + total * (row + packed) + tables, "flops": 3 * (new + total) * row / 2}
    if c["op"] == "decode":
        packed = 2 * c["kv_heads"] * d * 9 // 16
        return {"bytes": total * packed + tables + 4 * c["seqs"] * c["heads"] * d,
                "flops": 4 * d * c["heads"] * total}
    b = c["before"]
    pairs = sum(n * b + n * (n + 1) // 2 for n in lens)
    rows = 2 * total * c["heads"] + 2 * sum(n + b for n in lens) * c["kv_heads"]
    return {"bytes": 2 * d * rows, "flops": 4 * d * c["heads"] * pairs}


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------

def _normal(g, shape, dtype, outliers=False):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    if outliers:                        # a few channels of the keys are several times larger than the rest
        x[..., :: 37] *= 6.0
    return x.to(dtype)


def _pool(g, c, num_blocks):
    """A 4-bit pool of quantised rows."""
    hkv, d, tiles = c["kv_heads"], c["dim"], c["block"] // 16
    x = torch.randn((num_blocks, hkv, tiles, 16, d), generator=g, device="cuda", dtype=torch.float32)
    codes, scales = _quantise(x)
    return torch.cat([codes.flatten(-2), scales.flatten(-2)], -1).contiguous()


def _paged(g, c, lens):
    """Tables of shuffled blocks for the sequences, padded with -1."""
    block = c["block"]
    need = [-(-n // block) for n in lens]
    num_blocks = sum(need) + max(1, sum(need) // 10)
    order = torch.randperm(num_blocks, generator=g, device="cuda")[: sum(need)].to(torch.int32)
    tables = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device="cuda")
    used = torch.arange(max(need), device="cuda")[None] < torch.tensor(need, device="cuda")[:, None]
    tables[used] = order
    return tables, num_blocks


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt, d = DTYPES[c["dtype"]], c["dim"]
    i32 = dict(dtype=torch.int32, device="cuda")
    s = {"case": c}
    if c["op"] == "rotary":
        t, hq, hk = c["tokens"], c["heads"], c["kv_heads"]
        qkv = _normal(g, (t, hq + 2 * hk, d), dt)     # as the projection leaves them
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hk]
        s["positions"] = torch.randint(0, c["far"], (t,), generator=g, device="cuda", dtype=torch.int32)
        if c["norm"]:
            s["q_weight"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt)
            s["k_weight"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt)
        s["q_out"] = torch.empty((t, hq, d), dtype=dt, device="cuda")
        s["k_out"] = torch.empty((t, hk, d), dtype=dt, device="cuda")
        return s
    lens = _lens(c)
    hkv = c["kv_heads"]
    if c["op"] == "prompt":
        q_lens, k_lens = lens, [n + c["before"] for n in lens]
        s["q_lens"], s["k_lens"] = q_lens, k_lens
        if c["packed"]:
            qkv = _normal(g, (sum(lens), c["heads"] + 2 * hkv, d), dt)
            s["q"], s["k"], s["v"] = qkv.split([c["heads"], hkv, hkv], 1)
        else:
            s["q"] = _normal(g, (sum(q_lens), c["heads"], d), dt)
            s["k"] = _normal(g, (sum(k_lens), hkv, d), dt)
            s["v"] = _normal(g, (sum(k_lens), hkv, d), dt)
        s["cu_q"] = torch.tensor(np.cumsum([0] + q_lens), **i32)
        s["cu_k"] = torch.tensor(np.cumsum([0] + k_lens), **i32)
        s["out"] = torch.empty((sum(q_lens), c["heads"], d), dtype=dt, device="cuda")
        return s
    s["lens"] = lens
    s["tables"], num_blocks = _paged(g, c, lens)
    s["k_cache"], s["v_cache"] = _pool(g, c, num_blocks), _pool(g, c, num_blocks)
    s["k_scale"] = s["v_scale"] = None
    if c["scaled"]:
        s["k_scale"] = 0.5 + torch.rand(hkv, generator=g, device="cuda")
        s["v_scale"] = 0.5 + torch.rand(hkv, generator=g, device="cuda")
    if c["op"] == "decode":
        s["context_lens"] = torch.tensor(lens, **i32)
        s["q"] = _normal(g, (len(lens), c["heads"], d), dt)
        s["out"] = torch.empty_like(s["q"])
        return s
    new = [min(n, c["new"]) for n in lens]            # the newest tokens of each sequence
    seq = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), torch.tensor(new, device="cuda"))
    pos = torch.cat([torch.arange(n - m, n, device="cuda") for n, m in zip(lens, new)])
    s["slots"] = s["tables"][seq, pos // c["block"]].to(torch.int64) * c["block"] + pos % c["block"]
    s["k_new"] = _normal(g, (sum(new), hkv, d), dt, outliers=True)
    s["v_new"] = _normal(g, (sum(new), hkv, d), dt)
    s["cu"] = torch.tensor(np.cumsum([0] + lens), **i32)
    s["k_out"] = torch.empty((sum(lens), hkv, d), dtype=dt, device="cuda")
    s["v_out"] = torch.empty_like(s["k_out"])
    return s


# ---------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------

ROPE = dict(base=1000000.0, factor=8.0, original=8192.0, alpha=1.0, beta=32.0)


def run(s):
    return (_library if own else _plain)[s["case"]["op"]](s)


def _rotary_plain(s):
    c = s["case"]
    rot, half = c["rot"], c["rot"] // 2
    i = torch.arange(half, dtype=torch.float64, device="cuda")
    base = ROPE["base"]
    if c["scaling"] == "ntk":
        base = base * ROPE["factor"] ** (rot / (rot - 2))
    f = base ** (-2 * i / rot)
    if c["scaling"] == "linear":
        f = f / ROPE["factor"]
    if c["scaling"] == "parts":
        turns = ROPE["original"] * f / (2 * math.pi)
        keep = ((turns - ROPE["alpha"]) / (ROPE["beta"] - ROPE["alpha"])).clamp(0, 1)
        f = f * keep + f / ROPE["factor"] * (1 - keep)
    angle = s["positions"].double()[:, None] * f       # far positions need 64 bits
    mag = 1 + 0.1 * math.log(ROPE["factor"]) if c["scaling"] == "parts" else 1.0
    cos, sin = (mag * angle.cos()).float()[:, None], (mag * angle.sin()).float()[:, None]

    def turn(x, w):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w.float()
        if c["layout"] == "half":
            a, b = y[..., :half], y[..., half:rot]
            parts = [a * cos - b * sin, b * cos + a * sin]
        else:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            parts = [torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)]
        return torch.cat(parts + [y[..., rot:]], -1).to(x.dtype)

    return {"q": turn(s["q"], s.get("q_weight")), "k": turn(s["k"], s.get("k_weight"))}


def _quantise(u):
    """(bytes of codes, bytes of scales) of fp32 rows, 16 elements to a scale."""
    g = u.unflatten(-1, (-1, 16))
    scale = (g.abs().amax(-1) / 6).clamp(2.0 ** -9, 448).to(torch.float8_e4m3fn)
    t, a = scale.float()[..., None], g.abs()
    code = ((a > 0.25 * t).to(torch.uint8) + (a >= 0.75 * t) + (a > 1.25 * t) + (a >= 1.75 * t) + (a > 2.5 * t)
            + (a >= 3.5 * t) + (a > 5 * t)).to(torch.uint8) + 8 * torch.signbit(g).to(torch.uint8)
    code = code.flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], scale.view(torch.uint8)


def _values(codes, scales):
    """fp32 rows of the bytes that _quantise gives."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
    pairs = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    v = table[pairs.int()].unflatten(-1, (-1, 16))
    return (v * scales.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _split(cache, d):
    """The codes and the scales of every row of a pool, [block, head, row, bytes], as views of it."""
    codes = cache[..., : 8 * d].unflatten(-1, (16, d // 2))
    scales = cache[..., 8 * d:].unflatten(-1, (16, d // 16))
    return codes, scales


def _gather(cache, c, blocks, offsets, head_scale):
    """fp32 rows [n, kv_heads, dim] at the given places of a pool."""
    codes, scales = _split(cache, c["dim"])
    at = (blocks, slice(None), offsets // 16, offsets % 16)
    v = _values(codes[at], scales[at])
    return v if head_scale is None else v * head_scale[:, None]


def _cache_plain(s):
    c = s["case"]
    block, offset = s["slots"] // c["block"], s["slots"] % c["block"]
    for name in ("k", "v"):
        x = s[name + "_new"].float()
        if s[name + "_scale"] is not None:
            x = x / s[name + "_scale"][:, None]
        codes, scales = _split(s[name + "_cache"], c["dim"])
        at = (block, slice(None), offset // 16, offset % 16)
        codes[at], scales[at] = _quantise(x)
    row = torch.arange(s["k_out"].shape[0], device="cuda")
    seq = torch.searchsorted(s["cu"][1:].contiguous(), row, right=True)
    pos = row - s["cu"][seq]
    block = s["tables"][seq, pos // c["block"]].long()
    return {n: _gather(s[n + "_cache"], c, block, pos % c["block"], s[n + "_scale"]).to(s["k_new"].dtype) for n in ("k", "v")}


def _decode_plain(s):
    c = s["case"]
    n, longest = len(s["lens"]), max(s["lens"])
    pos = torch.arange(longest, device="cuda")
    seen = pos[None] < s["context_lens"][:, None]
    block = s["tables"][:, pos // c["block"]].long().clamp(min=0)
    q = s["q"].float().view(n, c["kv_heads"], -1, c["dim"])
    k = _gather(s["k_cache"], c, block.flatten(), (pos % c["block"]).repeat(n), s["k_scale"])
    k = k.view(n, longest, c["kv_heads"], c["dim"]).permute(0, 2, 3, 1)
    x = (q @ k) / math.sqrt(c["dim"])
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    v = _gather(s["v_cache"], c, block.flatten(), (pos % c["block"]).repeat(n), s["v_scale"])
    v = v.view(n, longest, c["kv_heads"], c["dim"]).permute(0, 2, 1, 3)
    out = (p @ v) / p.sum(-1, keepdim=True)
    return out.flatten(1, 2).to(s["q"].dtype)


def _padded(x, cu, longest):
    """[sequence, longest, heads, dim] of packed rows, and which of them exist."""
    at = cu[:-1, None] + torch.arange(longest, device="cuda")
    there = at < cu[1:, None]
    return x[at.clamp(max=x.shape[0] - 1)].float() * there[..., None, None], there


def _prompt_plain(s):
    c = s["case"]
    q, there = _padded(s["q"], s["cu_q"], max(s["q_lens"]))
    k, keys = _padded(s["k"], s["cu_k"], max(s["k_lens"]))
    v, _ = _padded(s["v"], s["cu_k"], max(s["k_lens"]))
    q = q.unflatten(2, (c["kv_heads"], -1)).permute(0, 2, 3, 1, 4)
    k, v = k.permute(0, 2, 3, 1)[:, :, None], v.permute(0, 2, 1, 3)[:, :, None]
    last = torch.arange(q.shape[3], device="cuda") + c["before"]           # the last key a row sees
    seen = keys[:, None] & (torch.arange(k.shape[4], device="cuda") <= last[:, None])
    x = (q @ k).div_(math.sqrt(c["dim"])).masked_fill_(~seen[:, None, None], -math.inf)
    p = x.sub_(x.amax(-1, keepdim=True).clamp(min=-3e38)).exp_()
    out = (p @ v) / p.sum(-1, keepdim=True)
    return out.permute(0, 3, 1, 2, 4).flatten(2, 3)[there].to(s["q"].dtype)


_plain = {"rotary": _rotary_plain, "cache": _cache_plain, "decode": _decode_plain, "prompt": _prompt_plain}


def _rotary_library(s):
    import paged_kv_cache_160_gb300 as pkv
    c = s["case"]
    if "table" not in s:                               # a program keeps the frequencies of its model
        s["table"] = pkv.pkv_rope_table(c["rot"], ROPE["base"], c["scaling"], ROPE["factor"], ROPE["original"],
                                        ROPE["alpha"], ROPE["beta"]).cuda()
    mag = 1 + 0.1 * math.log(ROPE["factor"]) if c["scaling"] == "parts" else 1.0
    pkv.pkv_qk_rotary(s["q_out"], s["q"], s["k_out"], s["k"], s["positions"], s["table"], c["layout"], mag,
                      s.get("q_weight"), s.get("k_weight"), 1e-6)
    return {"q": s["q_out"], "k": s["k_out"]}


def _desc(pkv, s):
    if "desc" not in s:
        s["desc"] = pkv.cache_desc_fp4(s["k_cache"], s["k_scale"], s["v_scale"])
    return s["desc"]


def _cache_library(s):
    import paged_kv_cache_160_gb300 as pkv
    desc = _desc(pkv, s)
    pkv.pkv_kv_write(s["k_new"], s["v_new"], s["slots"], s["k_cache"], s["v_cache"], desc)
    pkv.pkv_kv_read(s["k_out"], s["v_out"], s["cu"], s["tables"], s["k_cache"], s["v_cache"], desc)
    return {"k": s["k_out"], "v": s["v_out"]}


def _decode_library(s):
    import paged_kv_cache_160_gb300 as pkv
    c, desc, longest = s["case"], _desc(pkv, s), max(s["lens"])
    if "workspace" not in s:
        n = pkv.pkv_decode_workspace_bytes(len(s["lens"]), c["heads"], c["kv_heads"], c["dim"], c["block"], longest, 0)
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    pkv.pkv_paged_decode(s["out"], s["q"], s["k_cache"], s["v_cache"], desc, s["tables"], s["context_lens"], longest,
                         c["dim"] ** -0.5, 0, s["workspace"])
    return s["out"]


def _prompt_library(s):
    import paged_kv_cache_160_gb300 as pkv
    pkv.pkv_prompt_attention(s["out"], s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], max(s["q_lens"]),
                             s["case"]["dim"] ** -0.5)
    return s["out"]


_library = {"rotary": _rotary_library, "cache": _cache_library, "decode": _decode_library, "prompt": _prompt_library}


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------

def _e4m3_values():
    v = [m / 8 * 2.0 ** -6 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
    return torch.tensor(v[:127], dtype=torch.float64, device="cuda")       # 0 .. 448; the 128th code is NaN


def _nearest(x, grid):
    """Index of the entry of an ascending grid nearest to x >= 0; a tie goes to the even index."""
    hi = torch.searchsorted(grid, x.contiguous()).clamp(1, len(grid) - 1)
    lo = hi - 1
    below, above = x - grid[lo], grid[hi] - x
    return torch.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, lo)


def _exact_rotary(s, c):
    half = c["rot"] // 2
    freq = []
    for i in range(half):
        base = ROPE["base"]
        if c["scaling"] == "ntk":
            base *= ROPE["factor"] ** (c["rot"] / (c["rot"] - 2))
        f = base ** (-2.0 * i / c["rot"])
        turns = ROPE["original"] * f / (2 * math.pi)
        if c["scaling"] == "linear" or (c["scaling"] == "parts" and turns < ROPE["alpha"]):
            f /= ROPE["factor"]
        elif c["scaling"] == "parts" and turns <= ROPE["beta"]:
            w = (turns - ROPE["alpha"]) / (ROPE["beta"] - ROPE["alpha"])
            f = (1 - w) * f / ROPE["factor"] + w * f
        freq.append(f)
    angle = torch.outer(s["positions"].double(), torch.tensor(freq, dtype=torch.float64, device="cuda"))
    mag = 0.1 * math.log(ROPE["factor"]) + 1 if c["scaling"] == "parts" else 1.0
    turn = torch.polar(torch.full_like(angle, mag), angle)[:, None]
    out = {}
    for n in ("q", "k"):
        x = s[n].double()
        if c["norm"]:
            x = x / (x.pow(2).sum(-1, keepdim=True) / c["dim"] + 1e-6).sqrt() * s[n + "_weight"].double()
        y = x.clone()
        if c["layout"] == "half":
            z = torch.complex(x[..., :half], x[..., half:2 * half]) * turn
            y[..., :half], y[..., half:2 * half] = z.real, z.imag
        else:
            z = torch.view_as_complex(x[..., :2 * half].unflatten(-1, (half, 2)).contiguous()) * turn
            y[..., :2 * half] = torch.view_as_real(z).flatten(-2)
        out[n] = y
    return out


def _exact_row(cache, c, block, offset):
    """The stored values of rows, decoded bit by bit."""
    d = c["dim"]
    tile = cache[block, :, offset // 16].to(torch.int64)                   # [n, kv_heads, 9 * dim]
    r = offset % 16
    at = (r * (d // 2))[:, None, None] + torch.arange(d, device="cuda") // 2
    nib = (tile.gather(-1, at.expand(-1, tile.shape[1], -1)) >> (4 * (torch.arange(d, device="cuda") % 2))) & 15
    sat = 8 * d + (r * (d // 16))[:, None, None] + torch.arange(d, device="cuda") // 16
    sc = tile.gather(-1, sat.expand(-1, tile.shape[1], -1))
    e, m = (nib >> 1) & 3, nib & 1
    mag = torch.where(e == 0, 0.5 * m.double(), (1 + 0.5 * m.double()) * 2.0 ** (e.double() - 1))
    return torch.where(nib >= 8, -mag, mag) * _e4m3_values()[sc]


def _exact_cache(s, c):
    out, grid, levels = {}, _e4m3_values(), torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    first = np.cumsum([0] + s["lens"])
    tables = s["tables"].long()
    for n in ("k", "v"):
        x = s[n + "_new"].float()
        head = torch.ones(c["kv_heads"], device="cuda") if s[n + "_scale"] is None else s[n + "_scale"]
        u = (x / head[:, None]).double()                                   # the quotient is defined in 32 bits
        g = u.unflatten(-1, (-1, 16))
        amax = g.abs().amax(-1)
        sixth = (amax.float() / 6).double()                                # as is the scale's
        scale = grid[_nearest(sixth.clamp(2.0 ** -9, 448), grid)]
        val = levels[_nearest((g.abs() / scale[..., None]).clamp(max=6), levels)] * scale[..., None]
        val = torch.where(g < 0, -val, val).flatten(-2)
        rows, at = [], 0
        for i, length in enumerate(s["lens"]):
            pos = torch.arange(length, device="cuda")
            old = length - min(length, c["new"])
            was = _exact_row(s[n + "_cache"], c, tables[i, pos[:old] // c["block"]], pos[:old] % c["block"])
            rows += [was, val[at:at + length - old]]
            at += length - old
        out[n] = torch.cat(rows) * head.double()[:, None]
        assert out[n].shape[0] == first[-1]
    return out


def _exact_decode(s, c):
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    group = c["heads"] // c["kv_heads"]
    for i, length in enumerate(s["lens"]):
        pos = torch.arange(length, device="cuda")
        block = s["tables"][i].long()[pos // c["block"]]
        k = _exact_row(s["k_cache"], c, block, pos % c["block"])
        v = _exact_row(s["v_cache"], c, block, pos % c["block"])
        if c["scaled"]:
            k, v = k * s["k_scale"].double()[:, None], v * s["v_scale"].double()[:, None]
        for h in range(c["kv_heads"]):
            w = torch.softmax(s["q"][i, h * group:(h + 1) * group].double() @ k[:, h].T / math.sqrt(c["dim"]), -1)
            out[i, h * group:(h + 1) * group] = w @ v[:, h]
    return out


def _exact_prompt(s, c):
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    group, q0, k0 = c["heads"] // c["kv_heads"], 0, 0
    for lq, lk in zip(s["q_lens"], s["k_lens"]):
        for h in range(c["heads"]):
            k, v = s["k"][k0:k0 + lk, h // group].double(), s["v"][k0:k0 + lk, h // group].double()
            x = s["q"][q0:q0 + lq, h].double() @ k.T / math.sqrt(c["dim"])
            x += torch.full_like(x, -math.inf).triu(lk - lq + 1)
            out[q0:q0 + lq, h] = torch.softmax(x, -1) @ v
        q0, k0 = q0 + lq, k0 + lk
    return out


def exact(c, seed):
    s = prepare(c, seed)
    return {"rotary": _exact_rotary, "cache": _exact_cache, "decode": _exact_decode, "prompt": _exact_prompt}[c["op"]](s, c)
