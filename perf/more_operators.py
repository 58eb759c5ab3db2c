"""The library's operators around a cache that is kept short, in a plain form and through the library.

What a serving step over a paged cache needs to attend with several new tokens per sequence, and to keep
only the tokens that attention still looks at:

* ``chunk``    attention of each sequence's new tokens (drafts to verify, a prompt's next chunk, or one
               token) over its paged cache of any type, with the log of each row's sum of exponentials
* ``weights``  the attention weight that each cached token got from those rows, added to what it had
* ``select``   the tokens that each (sequence, kv head) keeps: the newest, the first, then the heaviest
* ``compact``  the kept rows moved to the front of the sequence's blocks, with their weights

``run`` computes them with elementary torch operations while ``own`` is false, and with the library's
calls where it is true.

Caches are [blocks, kv heads, rows of a block, dim] in 16 bits or e4m3 (a scale per kv head), or 4-bit
tiles: 16 rows in 16 x dim/2 bytes of e2m1 codes (element 2j of a row in the low nibble of byte j, element
2j+1 in the high one) followed by 16 x dim/16 e4m3 scales, one per 16 elements; an element's value is
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
        # four short sequences verify one to three drafted tokens: pure latency
        dict(name="chunk_small", op="chunk", seqs=4, low=6, high=37, pick=1, new_low=1, new=3, heads=4, kv_heads=4,
             dim=64, dtype="f16", kv="fp4", block=16, scaled=False),
        # a 7B-shaped batch of 64 sequences verifies four drafted tokens each
        dict(name="chunk_draft", op="chunk", seqs=64, low=128, high=2048, pick=2, new_low=4, new=4, heads=28, kv_heads=4,
             dim=128, dtype="bf16", kv="fp4", block=16, scaled=True),
        # few sequences with long contexts verify eight tokens each
        dict(name="chunk_draft_long", op="chunk", seqs=8, low=32768, high=131072, pick=4, new_low=8, new=8, heads=32,
             kv_heads=8, dim=128, dtype="bf16", kv="fp4", block=16, scaled=True),
        # a prompt's last 512-row chunk over its 4-bit cache
        dict(name="chunk_prefill", op="chunk", seqs=1, low=4096, high=4096, pick=1, new_low=512, new=512, heads=28,
             kv_heads=4, dim=128, dtype="bf16", kv="fp4", block=16, scaled=True),
        # the chunks of four long prompts at once, over an 8-bit cache
        dict(name="chunk_prompts", op="chunk", seqs=4, low=5000, high=9216, pick=3, new_low=700, new=1024, heads=32,
             kv_heads=8, dim=128, dtype="bf16", kv="e4m3", block=32, scaled=True),
        # one decode step's weights for the 7B-shaped batch
        dict(name="weights_step", op="weights", seqs=64, low=128, high=2048, pick=2, new_low=1, new=1, heads=28,
             kv_heads=4, dim=128, dtype="bf16", kv="bf16", block=16, scaled=False, prior=True),
        # the last 64 rows of four prompts look at their whole 4-bit caches, before the first eviction
        dict(name="weights_window", op="weights", seqs=4, low=4096, high=16384, pick=5, new_low=64, new=64, heads=32,
             kv_heads=8, dim=128, dtype="bf16", kv="fp4", block=16, scaled=True, prior=False),
        # every row of a prompt's chunk counts
        dict(name="weights_prompt", op="weights", seqs=1, low=8192, high=8192, pick=1, new_low=2048, new=2048, heads=32,
             kv_heads=8, dim=128, dtype="f16", kv="f16", block=16, scaled=False, prior=True),
        # a 7B-shaped batch keeps up to 512 tokens of each sequence
        dict(name="select_batch", op="select", seqs=64, low=128, high=2048, pick=2, kv_heads=4, keep=512, first=4,
             recent=128),
        # few long contexts go down to 8192 tokens
        dict(name="select_long", op="select", seqs=8, low=32768, high=131072, pick=4, kv_heads=8, keep=8192, first=4,
             recent=1024),
        # the batch's kept rows move to the front of blocks of their own (the old ones are shared prefixes)
        dict(name="compact_batch", op="compact", seqs=64, low=128, high=2048, pick=2, kv_heads=4, keep=512, dim=128,
             dtype="bf16", kv="bf16", block=16, scaled=False),
        # long contexts over an 8-bit cache
        dict(name="compact_long", op="compact", seqs=3, low=32768, high=65536, pick=4, kv_heads=8, keep=8192, dim=128,
             dtype="bf16", kv="e4m3", block=16, scaled=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("chunk", "weights", "select", "compact"))
    seqs = _log_int(rng, 1, 64)
    kv_heads = rng.randint(1, 8)
    c = dict(op=op, seqs=seqs, pick=rng.randrange(1 << 20), kv_heads=kv_heads)
    if op == "select":
        high = _log_int(rng, 1, min(131072, 600000 // seqs))
        keep = _log_int(rng, 1, 16384)
        return dict(c, low=max(1, high // rng.randint(1, 8)), high=high, keep=keep, first=rng.randint(0, 8),
                    recent=rng.randint(0, keep))
    c.update(dim=rng.choice((64, 128)), block=rng.choice((16, 32)), dtype=rng.choice(("bf16", "f16")))
    c["kv"] = rng.choice(("fp4", "e4m3", c["dtype"]))
    c["scaled"] = c["kv"] == "e4m3" or (c["kv"] == "fp4" and rng.random() < 0.5)
    if op == "compact":
        high = _log_int(rng, 1, min(65536, 120000 // seqs))
        return dict(c, low=max(1, high // rng.randint(1, 8)), high=high, keep=_log_int(rng, 1, 8192))
    heads = kv_heads * rng.randint(1, 8)
    high = _log_int(rng, 1, min(131072, 400000 // seqs))
    # at most as many pairs of rows and keys as the listed cases have
    new = _log_int(rng, 1, max(1, min(high, 2048, 500000000 // (seqs * high * heads))))
    c.update(low=max(1, high // rng.randint(1, 8)), high=high, heads=heads, new=new, new_low=max(1, new // rng.randint(1, 3)))
    return dict(c, prior=rng.random() < 0.5) if op == "weights" else c


def _lens(c):
    """The sequences' lengths and numbers of new rows (or of rows kept): fixed by the case."""
    r = random.Random(c["pick"])
    lens = [r.randint(c["low"], c["high"]) for _ in range(c["seqs"])]
    if "keep" in c:
        return lens, [min(n, c["keep"]) for n in lens]
    return lens, [min(n, r.randint(c["new_low"], c["new"])) for n in lens]


def _row_bytes(c):
    """Bytes of one cached row of a kv head, K or V."""
    return c["dim"] * 9 // 16 if c["kv"] == "fp4" else c["dim"] * (1 if c["kv"] == "e4m3" else 2)


def work(c):
    lens, new = _lens(c)
    hkv = c["kv_heads"]
    if c["op"] == "select":
        return {"bytes": 4 * hkv * (sum(lens) + sum(new)) + 8 * c["seqs"], "flops": hkv * sum(lens)}
    tables = 4 * sum(-(-n // c["block"]) for n in lens)
    if c["op"] == "compact":
        moved = hkv * sum(new)
        return {"bytes": moved * (2 * (2 * _row_bytes(c) + 4) + 4) + 2 * tables, "flops": moved}
    d = c["dim"]
    pairs = c["heads"] * sum(n * m - m * (m - 1) // 2 for n, m in zip(lens, new))
    rows = c["heads"] * sum(new)
    if c["op"] == "chunk":
        return {"bytes": 2 * _row_bytes(c) * hkv * sum(lens) + rows * (4 * d + 4) + tables, "flops": 4 * d * pairs}
    before = sum(lens) - sum(new) if c["prior"] else 0
    return {"bytes": hkv * (_row_bytes(c) * sum(lens) + 4 * (sum(lens) + before)) + rows * (2 * d + 4) + tables,
            "flops": 2 * d * pairs}


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------

def _pool(g, c, num_blocks):
    """A pool of rows in the cache's type."""
    shape = (num_blocks, c["kv_heads"], c["block"], c["dim"])
    out = None
    for at in range(0, num_blocks, 4096):              # in parts: the fp32 rows are larger than the pool
        n = min(4096, num_blocks - at)
        x = torch.randn((n,) + shape[1:], generator=g, device="cuda", dtype=torch.float32)
        if c["kv"] == "fp4":
            part = _quantise(x)
        elif c["kv"] == "e4m3":
            part = x.to(torch.float8_e4m3fn)
        else:
            part = x.to(DTYPES[c["kv"]])
        if out is None:
            out = torch.empty((num_blocks,) + part.shape[1:], dtype=part.dtype, device="cuda")
        out[at:at + n] = part
    return out


def _quantise(x):
    """4-bit tiles of fp32 rows [blocks, heads, rows, dim]: 16 rows' codes, then their scales."""
    g = x.unflatten(2, (-1, 16)).unflatten(-1, (-1, 16))
    scale = (g.abs().amax(-1) / 6).clamp(2.0 ** -9, 448).to(torch.float8_e4m3fn)
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    code = torch.bucketize(g.abs() / scale.float()[..., None], borders).to(torch.uint8)
    code = (code + 8 * (g < 0).to(torch.uint8)).flatten(-2)
    return torch.cat([(code[..., 0::2] + 16 * code[..., 1::2]).flatten(-2), scale.view(torch.uint8).flatten(-2)], -1)


def _tables(g, counts, order):
    """Tables of the given numbers of blocks from `order`, padded with -1."""
    tables = torch.full((len(counts), max(counts)), -1, dtype=torch.int32, device="cuda")
    used = torch.arange(max(counts), device="cuda")[None] < torch.tensor(counts, device="cuda")[:, None]
    tables[used] = order[: sum(counts)]
    return tables


def _heavy(g, shape):
    """Accumulated weights: many small ones, a few large, and tokens that nothing looked at."""
    w = torch.exp(2.5 * torch.randn(shape, generator=g, device="cuda") - 4)
    return w * (torch.rand(shape, generator=g, device="cuda") > 0.05)


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    i32 = dict(dtype=torch.int32, device="cuda")
    lens, new = _lens(c)
    n, hkv = c["seqs"], c["kv_heads"]
    s = {"case": c, "lens": lens, "new": new}
    if c["op"] == "select":
        s["weights"] = _heavy(g, (n, hkv, c["high"]))
        s["context_lens"], s["keep_lens"] = torch.tensor(lens, **i32), torch.tensor(new, **i32)
        s["kept"] = torch.empty((n, hkv, max(new)), **i32)
        return s
    blocks = [-(-x // c["block"]) for x in lens]
    fresh = [-(-x // c["block"]) for x in new] if c["op"] == "compact" else []
    total = sum(blocks) + sum(fresh)
    num_blocks = total + max(1, total // 10)
    order = torch.randperm(num_blocks, generator=g, device="cuda").to(torch.int32)
    s["tables"] = _tables(g, blocks, order)
    s["k_cache"] = _pool(g, c, num_blocks)
    s["v_cache"] = _pool(g, c, num_blocks) if c["op"] != "weights" else None
    s["k_scale"] = s["v_scale"] = None
    if c["scaled"]:
        s["k_scale"] = 0.5 + torch.rand(hkv, generator=g, device="cuda")
        s["v_scale"] = 0.5 + torch.rand(hkv, generator=g, device="cuda")
    if c["op"] == "compact":
        s["dst_tables"] = _tables(g, fresh, order[sum(blocks):])
        s["keep_lens"] = torch.tensor(new, **i32)
        s["rows"], s["dst_rows"] = torch.arange(n, **i32), torch.arange(n, 2 * n, **i32)
        s["weights"] = _heavy(g, (2 * n, hkv, c["high"]))
        kept = torch.full((n, hkv, max(new)), -1, **i32)
        for i in range(n):                             # a sorted choice of its own for every head
            at = torch.rand((hkv, lens[i]), generator=g, device="cuda").argsort(-1)[:, :new[i]]
            kept[i, :, :new[i]] = at.sort(-1).values.to(torch.int32)
        s["kept"] = kept
        if c["kv"] == "fp4":                           # 4-bit rows are read back as the values they stand for
            s["cu"] = torch.tensor(np.cumsum([0] + new), **i32)
            s["k_out"] = torch.empty((sum(new), hkv, c["dim"]), dtype=DTYPES[c["dtype"]], device="cuda")
            s["v_out"] = torch.empty_like(s["k_out"])
        return s
    s["cu_q"] = torch.tensor(np.cumsum([0] + new), **i32)
    s["start"] = torch.tensor([a - b for a, b in zip(lens, new)], **i32)
    s["q"] = torch.randn((sum(new), c["heads"], c["dim"]), generator=g, device="cuda").to(DTYPES[c["dtype"]])
    if c["op"] == "chunk":
        s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty((sum(new), c["heads"]), device="cuda")
        return s
    s["weights"] = _heavy(g, (n, hkv, c["high"])) if c["prior"] else None
    s["out"] = torch.zeros((n, hkv, c["high"]), device="cuda")
    s["lse"] = torch.empty((sum(new), c["heads"]), device="cuda")
    for i in range(n):                                 # as the attention of the same rows leaves it
        s["lse"][s["cu_q"][i]:s["cu_q"][i + 1]] = torch.logsumexp(_logits(s, i), -1).permute(2, 0, 1).flatten(1)
    return s


# ---------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------

def run(s):
    return (_library if own else _plain)[s["case"]["op"]](s)


def _rows(s, name, i, length):
    """fp32 rows [kv heads, length, dim] of sequence i."""
    c, cache = s["case"], s[name + "_cache"]
    blocks = s["tables"][i, : -(-length // c["block"])].long()
    if c["kv"] == "fp4":
        x = _values(cache[blocks], c["dim"])
    elif c["kv"] == "e4m3":
        x = cache.view(torch.uint8)[blocks].view(torch.float8_e4m3fn)
    else:
        x = cache[blocks]
    x = x.float().transpose(0, 1).flatten(1, 2)[:, :length]
    scale = s[name + "_scale"]
    return x if scale is None else x * scale[:, None, None]


def _values(tiles, d):
    """fp32 rows [blocks, heads, rows, dim] of 4-bit tiles, without the heads' scales."""
    codes = tiles[..., : 8 * d].unflatten(-1, (16, d // 2))
    scales = tiles[..., 8 * d:].unflatten(-1, (16, d // 16)).view(torch.float8_e4m3fn).float()
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
    v = table[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()]
    return (v.unflatten(-1, (-1, 16)) * scales[..., None]).flatten(-2).flatten(2, 3)


def _logits(s, i):
    """Scaled products [kv heads, group, rows, keys] of sequence i's new rows, -inf where a row does not look."""
    c, length, m = s["case"], s["lens"][i], s["new"][i]
    first = sum(s["new"][:i])
    q = s["q"][first:first + m].float().unflatten(1, (c["kv_heads"], -1)).permute(1, 2, 0, 3)
    x = (q.flatten(1, 2) @ _rows(s, "k", i, length).transpose(1, 2)).div_(math.sqrt(c["dim"])).unflatten(1, (-1, m))
    seen = torch.arange(length, device="cuda") <= torch.arange(length - m, length, device="cuda")[:, None]
    return x.masked_fill_(~seen, -math.inf)


def _chunk_plain(s):
    out, lse = [], []
    for i in range(len(s["lens"])):
        x = _logits(s, i)
        top = x.amax(-1, keepdim=True)
        p = x.sub_(top).exp_()
        total = p.sum(-1, keepdim=True)
        o = (p.flatten(1, 2) @ _rows(s, "v", i, s["lens"][i])).unflatten(1, (-1, s["new"][i])) / total
        out.append(o.permute(2, 0, 1, 3).flatten(1, 2))
        lse.append((top + total.log())[..., 0].permute(2, 0, 1).flatten(1))
    return {"out": torch.cat(out).to(s["q"].dtype), "lse": torch.cat(lse)}


def _weights_plain(s):
    first = 0
    for i, (length, m) in enumerate(zip(s["lens"], s["new"])):
        lse = s["lse"][first:first + m].unflatten(1, (s["case"]["kv_heads"], -1)).permute(1, 2, 0)
        w = _logits(s, i).sub_(lse[..., None]).exp_().sum((1, 2))
        if s["weights"] is not None:                   # what the tokens before these had
            w[:, :length - m] += s["weights"][i, :, :length - m]
        s["out"][i, :, :length] = w
        first += m
    return s["out"]


def _select_plain(s):
    c, w = s["case"], s["weights"]
    pos = torch.arange(w.shape[2], device="cuda")
    length, keep = s["context_lens"][:, None, None], s["keep_lens"][:, None, None]
    newest = (pos >= length - c["recent"]) & (pos < length)
    # larger comes first, ties by position; the newest all fit (recent is at most the number to keep)
    rank = torch.where(newest, 3e38 + 0 * w, torch.where(pos < c["first"], 2e38 + 0 * w, w))
    rank = torch.where(pos < length, rank, -1.0)
    order = rank.sort(dim=-1, descending=True, stable=True).indices
    order = order[..., : s["kept"].shape[2]]
    there = torch.arange(order.shape[2], device="cuda") < keep
    order = torch.where(there, order, 1 << 30).sort(-1).values
    return torch.where(there, order, -1).to(torch.int32)


def _compact_plain(s):
    c = s["case"]
    i, h, j = (s["kept"] >= 0).nonzero(as_tuple=True)
    p = s["kept"][i, h, j].long()
    src, dst = s["tables"][i, p // c["block"]].long(), s["dst_tables"][i, j // c["block"]].long()
    for name in ("k_cache", "v_cache"):
        cache = s[name]
        if c["kv"] == "fp4":
            d = c["dim"]
            for part in (cache[..., : 8 * d].unflatten(-1, (16, -1)), cache[..., 8 * d:].unflatten(-1, (16, -1))):
                part[dst, h, j % c["block"] // 16, j % 16] = part[src, h, p % c["block"] // 16, p % 16]
        else:
            flat = cache.view(torch.uint8) if c["kv"] == "e4m3" else cache
            flat[dst, h, j % c["block"]] = flat[src, h, p % c["block"]]
    s["weights"][s["dst_rows"].long()[i], h, j] = s["weights"][s["rows"].long()[i], h, p]
    out = {"weights": s["weights"]}
    if c["kv"] != "fp4":
        return dict(out, k=s["k_cache"], v=s["v_cache"])
    for name in ("k", "v"):
        rows = []
        for at, m in enumerate(s["new"]):
            x = _values(s[name + "_cache"][s["dst_tables"][at, : -(-m // c["block"])].long()], c["dim"])
            rows.append(x.transpose(0, 1).flatten(1, 2)[:, :m].transpose(0, 1))
        x = torch.cat(rows)
        out[name] = (x if s[name + "_scale"] is None else x * s[name + "_scale"][:, None]).to(DTYPES[c["dtype"]])
    return out


_plain = {"chunk": _chunk_plain, "weights": _weights_plain, "select": _select_plain, "compact": _compact_plain}


def _desc(pkv, s):
    if "desc" not in s:                                # a program keeps its pool's description
        make = pkv.cache_desc_fp4 if s["case"]["kv"] == "fp4" else pkv.cache_desc
        s["desc"] = make(s["k_cache"], s["k_scale"], s["v_scale"])
    return s["desc"]


def _chunk_library(s):
    import paged_kv_cache_160_gb300 as pkv
    c = s["case"]
    if "workspace" not in s:
        n = pkv.pkv_chunk_workspace_bytes(s["q"].shape[0], c["heads"], c["kv_heads"], c["dim"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    pkv.pkv_paged_chunk_attention(s["out"], s["q"], s["cu_q"], s["start"], s["k_cache"], s["v_cache"], _desc(pkv, s),
                                  s["tables"], c["dim"] ** -0.5, s["workspace"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _weights_library(s):
    import paged_kv_cache_160_gb300 as pkv
    pkv.pkv_attention_weights(s["out"], s["weights"], 1.0, s["q"], s["lse"], s["cu_q"], s["start"], s["k_cache"],
                              _desc(pkv, s), s["tables"], s["case"]["dim"] ** -0.5)
    return s["out"]


def _select_library(s):
    import paged_kv_cache_160_gb300 as pkv
    c = s["case"]
    pkv.pkv_evict_select(s["kept"], s["weights"], s["context_lens"], s["keep_lens"], c["first"], c["recent"])
    return s["kept"]


def _compact_library(s):
    import paged_kv_cache_160_gb300 as pkv
    c, desc = s["case"], _desc(pkv, s)
    pkv.pkv_evict_compact(s["k_cache"], s["v_cache"], desc, s["kept"], s["keep_lens"], s["tables"], s["dst_tables"],
                          s["weights"], s["rows"], s["dst_rows"])
    if c["kv"] != "fp4":
        return {"weights": s["weights"], "k": s["k_cache"], "v": s["v_cache"]}
    pkv.pkv_kv_read(s["k_out"], s["v_out"], s["cu"], s["dst_tables"], s["k_cache"], s["v_cache"], desc)
    return {"weights": s["weights"], "k": s["k_out"], "v": s["v_out"]}


_library = {"chunk": _chunk_library, "weights": _weights_library, "select": _select_library, "compact": _compact_library}


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------

def _e4m3_values():
    v = [m / 8 * 2.0 ** -6 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
    v = v[:127] + [math.nan]
    return torch.tensor(v + [-x for x in v], dtype=torch.float64, device="cuda")


def _exact_rows(s, c, name, h, table, pos):
    """Values [positions, dim] of kv head h at positions of a table, decoded bit by bit."""
    cache, d = s[name + "_cache"], c["dim"]
    block, offset = table[pos // c["block"]].long(), pos % c["block"]
    if c["kv"] == "fp4":
        tile = cache[block, h, offset // 16].long()
        j = torch.arange(d, device="cuda")
        r = (offset % 16)[:, None]
        code = (tile.gather(1, r * (d // 2) + j // 2) >> (4 * (j % 2))) & 15
        e, m = (code >> 1) & 3, (code & 1).double()
        mag = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * 2.0 ** (e.double() - 1))
        x = torch.where(code >= 8, -mag, mag) * _e4m3_values()[tile.gather(1, 8 * d + r * (d // 16) + j // 16)]
    elif c["kv"] == "e4m3":
        x = _e4m3_values()[cache.view(torch.uint8)[block, h, offset].long()]
    else:
        x = cache[block, h, offset].double()
    return x if s[name + "_scale"] is None else x * s[name + "_scale"][h].double()


def _exact_chunk(s, c):
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["lse"].shape, dtype=torch.float64, device="cuda")
    group, at = c["heads"] // c["kv_heads"], 0
    for i, (length, m) in enumerate(zip(s["lens"], s["new"])):
        pos = torch.arange(length, device="cuda")
        for g in range(c["kv_heads"]):
            k, v = (_exact_rows(s, c, name, g, s["tables"][i], pos) for name in ("k", "v"))
            for h in range(g * group, (g + 1) * group):
                x = s["q"][at:at + m, h].double() @ k.T / math.sqrt(c["dim"])
                x += torch.full_like(x, -math.inf).triu(length - m + 1)
                lse[at:at + m, h] = torch.logsumexp(x, -1)
                out[at:at + m, h] = torch.softmax(x, -1) @ v
        at += m
    return {"out": out, "lse": lse}


def _exact_weights(s, c):
    out = s["out"].double()
    group, at = c["heads"] // c["kv_heads"], 0
    for i, (length, m) in enumerate(zip(s["lens"], s["new"])):
        pos = torch.arange(length, device="cuda")
        for g in range(c["kv_heads"]):
            k = _exact_rows(s, c, "k", g, s["tables"][i], pos)
            w = torch.zeros(length, dtype=torch.float64, device="cuda")
            if c["prior"]:
                w[:length - m] = s["weights"][i, g, :length - m].double()
            for h in range(g * group, (g + 1) * group):
                x = s["q"][at:at + m, h].double() @ k.T / math.sqrt(c["dim"]) - s["lse"][at:at + m, h, None].double()
                w += torch.exp(x).tril(length - m).sum(0)
            out[i, g, :length] = w
        at += m
    return out


def _exact_select(s, c):
    w = s["weights"].double().cpu().numpy()
    kept = np.full(s["kept"].shape, -1, dtype=np.int64)
    for i, (length, keep) in enumerate(zip(s["lens"], s["new"])):
        recent = min(c["recent"], keep)
        first = min(c["first"], keep - recent, length - recent)
        rest = keep - recent - first
        for h in range(c["kv_heads"]):
            middle = np.argsort(-w[i, h, first:length - recent], kind="stable")[:rest] + first
            chosen = np.concatenate([np.arange(first), np.sort(middle), np.arange(length - recent, length)])
            kept[i, h, :keep] = chosen
    return torch.from_numpy(kept).cuda()


def _exact_compact(s, c):
    weights = s["weights"].double()
    out = {}
    if c["kv"] != "fp4":
        for name in ("k", "v"):
            cache = s[name + "_cache"]
            x = _e4m3_values()[cache.view(torch.uint8).long()] if c["kv"] == "e4m3" else cache.double()
            out[name] = x
    else:
        for name in ("k", "v"):
            out[name] = torch.empty(s[name + "_out"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for i, m in enumerate(s["new"]):
        for h in range(c["kv_heads"]):
            pos = s["kept"][i, h, :m].long()
            weights[c["seqs"] + i, h, :m] = s["weights"][i, h].double()[pos]
            j = torch.arange(m, device="cuda")
            for name in ("k", "v"):
                if c["kv"] == "fp4":
                    out[name][at:at + m, h] = _exact_rows(s, c, name, h, s["tables"][i], pos)
                else:                                  # stored values: without the head's scale
                    plain = dict(s, **{name + "_scale": None})
                    rows = _exact_rows(plain, c, name, h, s["tables"][i], pos)
                    out[name][s["dst_tables"][i].long()[j // c["block"]], h, j % c["block"]] = rows
        at += m
    return dict(out, weights=weights)


def exact(c, seed):
    s = prepare(c, seed)
    return {"chunk": _exact_chunk, "weights": _exact_weights, "select": _exact_select, "compact": _exact_compact}[c["op"]](s, c)
