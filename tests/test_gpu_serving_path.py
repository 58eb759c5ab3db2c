"""The operators together, as a server runs them over a 4-bit cache: a prompt (rotation and norms, attention
over its own rows, write), a second chunk (its history read back, attention over both), then decode steps with
the fused append.  Each stage's result is compared with float64 on the inputs that stage had, and the cache with
the bytes the definition gives.
"""
import numpy as np
import pytest
import torch

from oracle import fp4, prompt, rotary

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def _close(got, ref, bound):
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= bound).all(), float(np.nanmax(err / bound))


@pytest.mark.parametrize("dim,hq,hkv,block,dtype", [(128, 4, 2, 16, torch.bfloat16), (64, 3, 1, 32, torch.float16)])
def test_prompt_chunk_and_decode_steps(dim, hq, hkv, block, dtype):
    import paged_kv_cache_160_gb300 as pkv
    u = torch.finfo(dtype).eps / 2
    g = torch.Generator().manual_seed(dim)
    scale, base, rot = dim ** -0.5, 10000.0, dim // 2
    freq = rotary.frequencies(rot, base)
    table = pkv.pkv_rope_table(rot, base).cuda()
    wq, wk = ((1 + 0.2 * torch.randn(dim, generator=g)).to(dtype) for _ in range(2))
    prompts, chunks = [37, 130], [65, 9]
    bm = pkv.BlockManager(64, block)
    k_cache = torch.full(pkv.fp4_cache_shape(64, hkv, block, dim), 0x7F, dtype=torch.uint8, device="cuda")
    v_cache = torch.full_like(k_cache, 0x7F)
    hs = [torch.tensor([0.7 + 0.4 * h for h in range(hkv)], device="cuda") for _ in range(2)]
    desc = pkv.cache_desc_fp4(k_cache, *hs)
    width = 16
    stored = [[], []]                                  # the rows each sequence got, per sequence: (k, v) tensors

    def project(n, starts):
        """A packed projection of n[i] rows of each sequence, rotated: q, k (normed, rotated), v."""
        qkv = torch.randn((sum(n), hq + 2 * hkv, dim), generator=g).to(dtype).cuda()
        pos = np.concatenate([np.arange(s, s + m) for s, m in zip(starts, n)])
        q, k, v = qkv.split([hq, hkv, hkv], 1)
        q0, k0 = q.double().cpu().numpy(), k.double().cpu().numpy()
        pkv.pkv_qk_rotary(q, q, k, k, torch.tensor(pos, dtype=torch.int32, device="cuda"), table, "half", 1.0,
                          wq.cuda(), wk.cuda(), 1e-6)
        for got, x, w in ((q, q0, wq), (k, k0, wk)):
            ref, size = rotary.rotate(rotary.rms_norm(x, w.double().numpy(), 1e-6), pos, freq, "half")
            _close(got, ref, u * np.abs(ref) + 2.0 ** -18 * size + 2.0 ** -25)
        return q, k, v.contiguous()

    def attend(q, k, v, q_lens, k_lens):
        out = torch.empty((sum(q_lens), hq, dim), dtype=dtype, device="cuda")
        cu = [torch.tensor(np.cumsum([0] + n), dtype=torch.int32, device="cuda") for n in (q_lens, k_lens)]
        pkv.pkv_prompt_attention(out, q, k, v, *cu, max(q_lens), scale)
        ref, size = prompt.prompt_attention(*(t.double().cpu().numpy() for t in (q, k, v)), q_lens, k_lens, scale)
        _close(out, ref, (u + 2.0 ** -11) * size + u * np.abs(ref) + 2.0 ** -25)

    def write(k, v, n):
        slots = np.concatenate([bm.append_slots(i, m)[0] for i, m in enumerate(n)])
        pkv.pkv_kv_write(k.contiguous(), v, torch.tensor(slots, dtype=torch.int64, device="cuda"), k_cache, v_cache, desc)
        at = 0
        for i, m in enumerate(n):
            stored[i].append((k[at:at + m].cpu(), v[at:at + m].cpu()))
            at += m

    def history(i):
        """float64 values of what sequence i's cache has to hold."""
        return [fp4.values(*fp4.quantise(torch.cat(part).double().numpy(), s.cpu().numpy()))
                * s.double().cpu().numpy()[:, None] for part, s in zip(zip(*stored[i]), hs)]

    # the prompts attend their own fresh rows, which then go into the cache
    for i in range(2):
        bm.allocate(i, 0)
    q, k, v = project(prompts, [0, 0])
    attend(q, k, v, prompts, prompts)
    write(k, v, prompts)
    # a chunk behind each: its history comes back from the cache and takes the chunk's rows behind it
    tables, lens = bm.export([0, 1], width)
    assert lens == prompts
    q, k, v = project(chunks, prompts)
    hist = [torch.empty((sum(prompts), hkv, dim), dtype=dtype, device="cuda") for _ in range(2)]
    pkv.pkv_kv_read(*hist, torch.tensor(np.cumsum([0] + prompts), dtype=torch.int32, device="cuda"),
                    torch.tensor(tables, dtype=torch.int32, device="cuda"), k_cache, v_cache, desc)
    for got, refs in zip(hist, zip(history(0), history(1))):
        ref = np.concatenate(refs)
        _close(got, ref, u * np.abs(ref) * (1 + 2.0 ** -12) + 2.0 ** -25)
    both = [torch.cat([h[:37], x[:65], h[37:], x[65:]]) for h, x in zip(hist, (k, v))]
    attend(q, *both, chunks, [p + c for p, c in zip(prompts, chunks)])
    write(k, v, chunks)
    # decode steps
    ws = torch.empty(pkv.pkv_decode_workspace_bytes(2, hq, hkv, dim, block, 512, 0), dtype=torch.uint8, device="cuda")
    for step in range(3):
        _, _, tables, lens = bm.step_decode([0, 1], width)
        q, k, v = project([1, 1], [n - 1 for n in lens])
        out = torch.empty((2, hq, dim), dtype=dtype, device="cuda")
        q = q.contiguous()
        pkv.pkv_paged_decode_append(out, q, k.contiguous(), v, k_cache, v_cache, desc,
                                    torch.tensor(tables, dtype=torch.int32, device="cuda"),
                                    torch.tensor(lens, dtype=torch.int32, device="cuda"), 512, scale, 0, ws)
        for i in range(2):
            stored[i].append((k[i:i + 1].cpu(), v[i:i + 1].cpu()))
        kk, vv = (np.concatenate(t) for t in zip(*(history(i) for i in range(2))))
        assert len(kk) == sum(lens)
        ref, size = prompt.prompt_attention(q.double().cpu().numpy(), kk, vv, [1, 1], lens, scale)
        # scores of normed rows: scale * sum |q k| < 32, as for the decode's own tests
        _close(out, ref, 2.0 ** -10 * size + u * np.abs(ref) + 2.0 ** -25)
    assert pkv.pkv_get_device_error() == 0


def test_blocks_past_4_gib_of_a_pool():
    """Written, read back and decoded at the end of a pool of more than 2^32 bytes, as in a small pool."""
    import paged_kv_cache_160_gb300 as pkv
    heads, dim, lens = 8, 128, [40, 100]
    g = torch.Generator().manual_seed(7)
    rows = [torch.randn((sum(lens), heads, dim), generator=g).to(torch.bfloat16).cuda() for _ in range(2)]
    q = torch.randn((2, 4 * heads, dim), generator=g).to(torch.bfloat16).cuda()
    need = [-(-n // 16) for n in lens]
    cu = torch.tensor([0, *np.cumsum(lens)], dtype=torch.int32, device="cuda")
    results = []
    for nb in (sum(need), 480_000):
        pools = [torch.zeros(pkv.fp4_cache_shape(nb, heads, 16, dim), dtype=torch.uint8, device="cuda") for _ in range(2)]
        assert nb < 1000 or pools[0].numel() > 2 ** 32
        ids = list(range(nb - sum(need), nb))
        table = np.full((2, max(need)), -1, dtype=np.int32)
        for i, n in enumerate(need):
            table[i, :n] = [ids.pop() for _ in range(n)]
        slots = np.concatenate([table[i, np.arange(n) // 16].astype(np.int64) * 16 + np.arange(n) % 16
                                for i, n in enumerate(lens)])
        desc, tables = pkv.cache_desc_fp4(pools[0]), torch.from_numpy(table).cuda()
        pkv.pkv_kv_write(*rows, torch.from_numpy(slots).cuda(), *pools, desc)
        back = [torch.zeros_like(rows[0]) for _ in range(2)]
        pkv.pkv_kv_read(*back, cu, tables, *pools, desc)
        out = torch.zeros_like(q)
        ws = torch.empty(pkv.pkv_decode_workspace_bytes(2, 4 * heads, heads, dim, 16, max(lens), 0), dtype=torch.uint8,
                         device="cuda")
        pkv.pkv_paged_decode(out, q, *pools, desc, tables, torch.tensor(lens, dtype=torch.int32, device="cuda"), max(lens),
                             0.09, 0, ws)
        assert pkv.pkv_get_device_error() == 0
        results.append([*back, out])
        del pools
    assert results[0][0].abs().sum() > 0 and results[0][2].abs().sum() > 0
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_two_streams_at_once():
    """The same calls on two streams, with their own tensors, give what they give one after the other."""
    import paged_kv_cache_160_gb300 as pkv
    table = pkv.pkv_rope_table(128).cuda()

    def inputs(seed, lens):
        g = torch.Generator().manual_seed(seed)
        qkv = torch.randn((sum(lens), 12, 128), generator=g).to(torch.bfloat16).cuda()
        cu = torch.tensor([0, *np.cumsum(lens)], dtype=torch.int32, device="cuda")
        pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32).cuda()
        return qkv, cu, pos, max(lens)

    def step(x):
        qkv, cu, pos, longest = x
        q, k, v = (t.clone() for t in qkv.split([8, 2, 2], 1))
        pkv.pkv_qk_rotary(q, q, k, k, pos, table)
        out = torch.zeros_like(q)
        pkv.pkv_prompt_attention(out, q, k, v, cu, cu, longest, 0.09)
        return q, k, out

    # many items on one stream, few with split keys on the other
    sides = [inputs(1, [700, 30, 1, 513]), inputs(2, [1100])]
    alone = [step(x) for x in sides]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sides]
    together = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                together[i].append(step(sides[i]))
    torch.cuda.synchronize()
    assert pkv.pkv_get_device_error() == 0
    for want, runs in zip(alone, together):
        for got in runs:
            assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("longest", [0, 3000])
def test_rows_past_4_gib(longest):
    """Rotation and attention of 65,535 sequences, the most that a call takes, in more than 2^32 bytes of rows: parts
    of them are as alone."""
    import paged_kv_cache_160_gb300 as pkv
    hq, hkv, dim = 14, 2, 128
    rng = np.random.default_rng(12)
    lens = rng.integers(0, 40, 65535)
    if longest:
        lens[50_000] = longest
    start = np.concatenate([[0], np.cumsum(lens)])
    total = int(start[-1])
    g = torch.Generator(device="cuda").manual_seed(3)
    qkv = torch.randn((total, hq + 2 * hkv, dim), generator=g, device="cuda", dtype=torch.bfloat16)
    assert qkv.numel() * 2 > 2 ** 32
    pos = torch.from_numpy(np.arange(total) - np.repeat(start[:-1], lens)).to(torch.int32).cuda()
    table = pkv.pkv_rope_table(dim).cuda()
    parts = [(0, 40), (49_990, 50_010), (65_500, 65_535)]
    before = [qkv[start[a]:start[b]].clone() for a, b in parts]

    def step(x, p, n):
        q, k, v = x.split([hq, hkv, hkv], 1)
        pkv.pkv_qk_rotary(q, q, k, k, p, table)
        out = torch.zeros((len(x), hq, dim), dtype=x.dtype, device="cuda")
        cu = torch.from_numpy(np.concatenate([[0], np.cumsum(n)])).to(torch.int32).cuda()
        pkv.pkv_prompt_attention(out, q, k, v, cu, cu, int(max(n)), dim ** -0.5)
        return out

    whole = step(qkv, pos, lens)
    assert pkv.pkv_get_device_error() == 0
    for (a, b), x in zip(parts, before):
        s, e = start[a], start[b]
        out = step(x, pos[s:e].clone(), lens[a:b])
        assert pkv.pkv_get_device_error() == 0
        assert torch.equal(x, qkv[s:e])
        # Few items may share their keys between CTAs, with sums in another order: each side is within
        # (2^-8 + 2^-11) sum_j p_j |v_j| + 2^-8 |out| of the exact row (tests/test_gpu_prompt.py), and sum_j p_j |v_j| <= max |v|.
        err = (out.double() - whole[s:e].double()).abs()
        most = x[:, hq + hkv:].double().abs().max()
        assert (err <= 2 * ((2.0 ** -8 + 2.0 ** -11) * most + 2.0 ** -8 * out.double().abs())).all() and (out != 0).any()
