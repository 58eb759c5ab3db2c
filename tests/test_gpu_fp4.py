"""GPU parity of the 4-bit cache: written bytes, rows read back, decode over it (plain, fused append,
no-alloc), block copies, against the float64 oracle (oracle/fp4.py).

Written bytes match the definition bit for bit.  A row read back is code * scale (exact) times the head's
scale (one fp32 rounding), rounded once: |err| <= u |v| (1 + 2^-12) + 2^-25 (fp16 subnormals), u = finfo.eps / 2.

Decode, with A = sum_j p_j |v_j|: P is rounded to fp16 (2^-11); scores are fp32 sums of exact fp16 products of
at most 128 terms, scaled: an error of the exponent below 2^-24 * 128 * scale * sum |q k|, under 2^-12 for the
inputs here (scale * sum |q k| < 32); exp2 and the fp32 sums add less than 2^-14; partials merge in fp32.  So
|err| <= 2^-10 A + u |out| + 2^-25.
"""
import numpy as np
import pytest
import torch

from oracle import fp4, prompt
from oracle.formats import e4m3_table

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def _tables(rng, lens, block, num_blocks, extra=1):
    need = [-(-n // block) for n in lens]
    ids = list(rng.permutation(num_blocks)[: sum(need)])
    width = max(need + [1]) + extra
    t = np.full((len(lens), width), -1, dtype=np.int32)
    for i, n in enumerate(need):
        t[i, :n] = [ids.pop() for _ in range(n)]
    return t


def _pool(rng, num_blocks, heads, block, dim):
    if num_blocks > 2000:                                      # codes and scales as they come
        return (rng.integers(0, 16, (num_blocks, heads, block, dim)).astype(np.uint8),
                rng.integers(0x28, 0x34, (num_blocks, heads, block, dim // 16)).astype(np.uint8))
    x = rng.standard_normal((num_blocks, heads, block, dim)) * np.exp(0.3 * rng.standard_normal((num_blocks, heads, 1, 1)))
    return fp4.quantise(x)


def _rows(codes, sc, table, length, block, scale):
    """float64 [length, heads, D] of one sequence."""
    pos = np.arange(length)
    at = (table[pos // block], slice(None), pos % block)
    r = fp4.values(codes[at], sc[at])
    return r if scale is None else r * scale.astype(np.float64)[:, None]


def _close(got, ref, bound):
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= bound).all(), (float(np.nanmax(err / bound)), np.argwhere(~(err <= bound))[:3])


# ---------------------------------------------------------------------------------------
# write
# ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim,heads,block,scaled", [(128, 4, 16, True), (128, 3, 32, False), (64, 5, 16, False),
                                                    (64, 1, 32, True), (96, 2, 48, True), (16, 2, 16, False)])
def test_written_bytes_are_the_definitions(dtype, dim, heads, block, scaled):
    import paged_kv_cache_160_gb300 as pkv
    rng = np.random.default_rng(dim + heads)
    nb, tokens = 9, 61
    pool = [rng.integers(0, 256, pkv.fp4_cache_shape(nb, heads, block, dim)).astype(np.uint8) for _ in range(2)]
    x = [torch.from_numpy(rng.standard_normal((tokens, heads, dim)) * np.exp(2 * rng.standard_normal((tokens, heads, 1))))
         .to(DT[dtype]) for _ in range(2)]
    x[0][0, 0, :5] = torch.tensor([1e30, -1e30, float("inf"), -float("inf"), 0.0])
    x[0][1, 0, 7] = float("nan")
    x[1][2, 0] = 0.0
    x[1][3, 0] = 2.0 ** -14
    x[1][4, 0, 3] = -0.0
    # quotients on the borders between codes: with a 6 in the group and no head scale, u / s = u
    x[0][5, 0, :8] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    x[0][5, 0, 8:16] = -x[0][5, 0, :8]
    slots = rng.permutation(nb * block)[:tokens].astype(np.int64)
    slots[[10, 20]] = -1
    scales = [(0.3 + 2 * rng.random(heads)).astype(np.float32) if scaled else None for _ in range(2)]
    dev = [torch.from_numpy(p).cuda() for p in pool]
    desc = pkv.cache_desc_fp4(dev[0], *(torch.from_numpy(s).cuda() if scaled else None for s in scales))
    pkv.pkv_kv_write(x[0].cuda(), x[1].cuda(), torch.from_numpy(slots).cuda(), *dev, desc)
    assert pkv.pkv_get_device_error() == 0
    live = slots >= 0
    for xs, p, got, hs in zip(x, pool, dev, scales):
        codes, sc = fp4.unpack(p)
        want_c, want_s = fp4.quantise(xs.double().numpy(), hs)
        nan = (want_s == 0x7F)[..., None] & np.ones(16, bool)
        blk, off = slots[live] // block, slots[live] % block
        codes[blk, :, off], sc[blk, :, off] = want_c[live], want_s[live]
        gc, gs = fp4.unpack(got.cpu().numpy())
        assert np.array_equal(gs, sc)
        # the codes of a NaN group stand for nothing
        hole = np.zeros(codes.shape, bool)
        hole[blk, :, off] = nan.reshape(want_c.shape)[live]
        assert np.array_equal(gc[~hole], codes[~hole])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("head_scale", [None, 1.0, 0.3, -1.7, 1e-3, 3e4])
def test_elements_on_and_next_to_the_borders_between_codes(head_scale, dtype):
    """Every scale of the format; elements on each border times the scale, and their neighbours in the type."""
    import paged_kv_cache_160_gb300 as pkv
    dt = DT[dtype]
    hs = 1.0 if head_scale is None else np.float64(np.float32(head_scale))
    s = e4m3_table()[1:0x7F]
    s = s[(6 * s * abs(hs) < 6e4) & (s * abs(hs) > 1e-3)]      # well inside fp16
    borders = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    x = torch.zeros((len(s), 32), dtype=dt)
    x[:, 0] = x[:, 16] = torch.from_numpy(6 * s * hs).to(dt)
    mid = torch.from_numpy(s[:, None] * borders * hs).to(dt)
    step = torch.finfo(dt).eps * mid.float().abs()
    x[:, 1:8], x[:, 8:15], x[:, 17:24], x[:, 24:31] = mid, -(mid.float() + step).to(dt), (mid.float() - step).to(dt), -mid
    n = len(s)
    k = torch.zeros(pkv.fp4_cache_shape(-(-n // 16), 1, 16, 32), dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(k)
    scale = None if head_scale is None else torch.tensor([head_scale], dtype=torch.float32, device="cuda")
    xx = x.view(n, 1, 32)
    pkv.pkv_kv_write(xx.cuda(), xx.flip(0).contiguous().cuda(), torch.arange(n, device="cuda"), k, v,
                     pkv.cache_desc_fp4(k, scale, scale))
    for got, src in ((k, xx), (v, xx.flip(0))):
        gc, gs = fp4.unpack(got.cpu().numpy())
        wc, ws = fp4.quantise(src.double().numpy(), None if head_scale is None else [head_scale])
        at = np.arange(n)
        assert np.array_equal(gs[at // 16, :, at % 16], ws) and np.array_equal(gc[at // 16, :, at % 16], wc)


@pytest.mark.parametrize("head_scale", [0.0, float("inf"), float("nan"), 1e-38, 1e38, -3e-31])
def test_odd_head_scales(head_scale):
    import paged_kv_cache_160_gb300 as pkv
    g = torch.Generator().manual_seed(3)
    x = torch.randn((16, 1, 64), generator=g).to(torch.bfloat16)
    x[3, 0, 5] = float("inf")
    x[4, 0, :20] = 0.0
    x[5] *= 1e-30
    x[6] *= 1e30
    k = torch.zeros(pkv.fp4_cache_shape(1, 1, 16, 64), dtype=torch.uint8, device="cuda")
    scale = torch.tensor([head_scale], dtype=torch.float32, device="cuda")
    pkv.pkv_kv_write(x.cuda(), x.cuda(), torch.arange(16, device="cuda"), k, k.clone(), pkv.cache_desc_fp4(k, scale, scale))
    gc, gs = fp4.unpack(k.cpu().numpy())
    wc, ws = fp4.quantise(x.double().numpy(), [head_scale])
    assert np.array_equal(gs[0].transpose(1, 0, 2), ws)
    live = np.repeat(ws != 0x7F, 16, -1)
    assert np.array_equal(gc[0].transpose(1, 0, 2)[live], wc[live])


@pytest.mark.parametrize("exponent", [-120, -99, -85, -80, -79, -60, 60, 99, 101])
def test_elements_of_the_size_of_a_tiny_or_huge_head_scale(exponent):
    """Elements down to subnormals: u = x / head scale is of ordinary size for the larger ones."""
    import paged_kv_cache_160_gb300 as pkv
    rng = np.random.default_rng(200 + exponent)
    size = np.maximum(exponent + rng.integers(-16, 4, (64, 1, 16)), -133).astype(np.float64)
    x = torch.from_numpy(rng.uniform(-2, 2, (64, 1, 16)) * 2.0 ** size).to(torch.bfloat16)
    x[1] = 0.0
    x[2, 0, 3:] = 0.0
    scale = np.array([1.7 * 2.0 ** exponent], dtype=np.float32)
    pool = torch.zeros(pkv.fp4_cache_shape(4, 1, 16, 16), dtype=torch.uint8, device="cuda")
    dev = torch.from_numpy(scale).cuda()
    pkv.pkv_kv_write(x.cuda(), x.cuda(), torch.arange(64, device="cuda"), pool, pool.clone(),
                     pkv.cache_desc_fp4(pool, dev, dev))
    codes, sc = fp4.unpack(pool.cpu().numpy())
    want, want_sc = fp4.quantise(x.double().numpy(), scale)
    assert (sc.reshape(64, 1, 1) == want_sc).all() and (codes.reshape(64, 1, 16) == want).all()


def test_many_tokens_and_a_bad_slot():
    import paged_kv_cache_160_gb300 as pkv
    rng = np.random.default_rng(1)
    heads, dim, block, nb = 2, 128, 16, 400
    x = torch.randn((6000, heads, dim), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    slots = torch.from_numpy(rng.permutation(nb * block)[:6000].astype(np.int64))
    slots[77] = nb * block
    k = torch.zeros(pkv.fp4_cache_shape(nb, heads, block, dim), dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(k)
    pkv.pkv_kv_write(x.cuda(), x.flip(0).contiguous().cuda(), slots.cuda(), k, v, pkv.cache_desc_fp4(k))
    assert pkv.pkv_get_device_error() == pkv.DEVERR["slot"]
    keep = np.arange(6000) != 77
    blk, off = slots.numpy()[keep] // block, slots.numpy()[keep] % block
    for got, xs in ((k, x), (v, x.flip(0))):
        gc, gs = fp4.unpack(got.cpu().numpy())
        wc, ws = fp4.quantise(xs.double().numpy()[keep])
        assert np.array_equal(gc[blk, :, off], wc) and np.array_equal(gs[blk, :, off], ws)


# ---------------------------------------------------------------------------------------
# read
# ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("out", ["bf16", "f16"])
@pytest.mark.parametrize("dim,heads,block,scaled", [(128, 4, 16, True), (64, 3, 32, False), (96, 2, 16, True)])
@pytest.mark.parametrize("lens", [[1], [0, 17, 0, 16, 300, 1], [33, 64, 5]])
def test_read_back(lens, dim, heads, block, scaled, out):
    import paged_kv_cache_160_gb300 as pkv
    rng = np.random.default_rng(sum(lens) + dim)
    nb = sum(-(-n // block) for n in lens) + 3
    table = _tables(rng, lens, block, nb)
    pools = [_pool(rng, nb, heads, block, dim) for _ in range(2)]
    scales = [(0.3 + 2 * rng.random(heads)).astype(np.float32) if scaled else None for _ in range(2)]
    dev = [torch.from_numpy(fp4.pack(*p)).cuda() for p in pools]
    desc = pkv.cache_desc_fp4(dev[0], *(torch.from_numpy(s).cuda() if scaled else None for s in scales))
    total = sum(lens)
    outs = [torch.full((total + 5, heads, dim), 9.0, dtype=DT[out], device="cuda") for _ in range(2)]
    pkv.pkv_kv_read(*outs, torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device="cuda"),
                    torch.from_numpy(table).cuda(), *dev, desc)
    assert pkv.pkv_get_device_error() == 0
    u = torch.finfo(DT[out]).eps / 2
    for o, p, hs in zip(outs, pools, scales):
        assert (o[total:] == 9.0).all()
        ref = np.concatenate([_rows(*p, table[i], n, block, hs) for i, n in enumerate(lens)])
        _close(o[:total], ref, u * np.abs(ref) * (1 + 2.0 ** -12) + 2.0 ** -25)


@pytest.mark.parametrize("lens,heads,dim", [([9001, 3], 4, 128), ([20001], 2, 128), ([3000, 0, 801], 16, 64)])
def test_read_back_of_many_rows(lens, heads, dim):
    test_read_back(lens, dim, heads, 16, True, "bf16")


def test_read_back_of_16_bit_and_e4m3_caches():
    import paged_kv_cache_160_gb300 as pkv
    rng = np.random.default_rng(8)
    lens, block, heads, dim = [20, 1, 47], 16, 3, 128
    table = _tables(rng, lens, block, 9)
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device="cuda")
    pos = np.concatenate([np.arange(n) for n in lens])
    blk = np.concatenate([table[i, np.arange(n) // block] for i, n in enumerate(lens)])
    for dt in (torch.bfloat16, torch.float16):
        k = torch.randn((9, heads, block, dim), generator=torch.Generator().manual_seed(2)).to(dt)
        v = k.flip(0).contiguous()
        ko, vo = (torch.empty((sum(lens), heads, dim), dtype=dt, device="cuda") for _ in range(2))
        kc = k.cuda()
        pkv.pkv_kv_read(ko, vo, cu, torch.from_numpy(table).cuda(), kc, v.cuda(), pkv.cache_desc(kc))
        assert torch.equal(ko.cpu(), k[blk, :, pos % block]) and torch.equal(vo.cpu(), v[blk, :, pos % block])
    codes = rng.integers(0, 256, (2, 9, heads, block, dim)).astype(np.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0
    hs = (0.5 + rng.random((2, heads))).astype(np.float32)
    kc, vc = (torch.from_numpy(c).cuda() for c in codes)
    desc = pkv.cache_desc(kc, *(torch.from_numpy(s).cuda() for s in hs))
    for dt in (torch.bfloat16, torch.float16):
        outs = [torch.empty((sum(lens), heads, dim), dtype=dt, device="cuda") for _ in range(2)]
        pkv.pkv_kv_read(*outs, cu, torch.from_numpy(table).cuda(), kc, vc, desc)
        for o, c, s in zip(outs, codes, hs):
            ref = e4m3_table()[c][blk, :, pos % block] * s.astype(np.float64)[:, None]
            _close(o, ref, torch.finfo(dt).eps / 2 * np.abs(ref) * (1 + 2.0 ** -12) + 2.0 ** -25)
    assert pkv.pkv_get_device_error() == 0


def test_read_back_reports_bad_blocks_and_lengths():
    import paged_kv_cache_160_gb300 as pkv
    heads, dim = 2, 64
    k = torch.zeros(pkv.fp4_cache_shape(4, heads, 16, dim), dtype=torch.uint8, device="cuda")
    desc = pkv.cache_desc_fp4(k)

    def read(cu, table, total=40):
        o = torch.full((total, heads, dim), 3.0, dtype=torch.bfloat16, device="cuda")
        v = o.clone()
        pkv.pkv_kv_read(o, v, torch.tensor(cu, dtype=torch.int32, device="cuda"),
                        torch.tensor(table, dtype=torch.int32, device="cuda"), k, k, desc)
        err = pkv.pkv_get_device_error()
        assert torch.equal(o, v)
        return (o[:, 0, 0] == 3.0).tolist(), err

    left, err = read([0, 20, 40], [[0, 4], [1, 2]])           # block 4 does not exist: rows 16 .. 19
    assert err == pkv.DEVERR["block_id"] and left == [16 <= i < 20 for i in range(40)]
    left, err = read([0, 40], [[0, 1]])                       # two blocks hold 32 rows
    assert err == pkv.DEVERR["chunk"] and left == [i >= 32 for i in range(40)]
    left, err = read([0, 20, 10, 30], [[0, 1], [1, 2], [2, 3]])
    assert err & pkv.DEVERR["chunk"] and left[30:] == [True] * 10
    left, err = read([0, 50], [[0, 1, 2, 3]])                 # more rows than the output has
    assert err == pkv.DEVERR["chunk"] and not any(left)
    left, err = read([0, 40], [[0, -1, 1]])
    assert err == pkv.DEVERR["block_id"] and left == [16 <= i < 32 for i in range(40)]


# ---------------------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------------------

def _decode_case(seed, lens, hq, hkv, dim, block, scaled, nan_rest=True):
    rng = np.random.default_rng(seed)
    nb = sum(-(-n // block) for n in lens) + 3
    table = _tables(rng, lens, block, nb)
    pools = [_pool(rng, nb, hkv, block, dim) for _ in range(2)]
    if nan_rest:                                               # rows that hold no token are NaN
        used = np.zeros((nb, block), bool)
        for i, n in enumerate(lens):
            pos = np.arange(n)
            used[table[i, pos // block], pos % block] = True
        for codes, sc in pools:
            sc[~used[:, None, :].repeat(hkv, 1)] = 0x7F
    scales = [(0.5 + rng.random(hkv)).astype(np.float32) if scaled else None for _ in range(2)]
    return rng, table, pools, scales


def _bound(out, size, dtype):
    return 2.0 ** -10 * size + torch.finfo(dtype).eps / 2 * np.abs(out) + 2.0 ** -25


def _run_decode(lens, hq, hkv, dim, dtype, block=16, part=0, scaled=True, seed=0, entry="plain", scale=None):
    import paged_kv_cache_160_gb300 as pkv
    rng, table, pools, scales = _decode_case(seed, lens, hq, hkv, dim, block, scaled)
    dev = [torch.from_numpy(fp4.pack(*p)).cuda() for p in pools]
    desc = pkv.cache_desc_fp4(dev[0], *(torch.from_numpy(s).cuda() if scaled else None for s in scales))
    q = torch.from_numpy(rng.standard_normal((len(lens), hq, dim))).to(DT[dtype])
    out = torch.full(q.shape, float("nan"), dtype=DT[dtype], device="cuda")
    longest = max(lens + [1])
    scale = dim ** -0.5 if scale is None else scale
    ws = torch.full((pkv.pkv_decode_workspace_bytes(len(lens), hq, hkv, dim, block, longest, part),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    args = (out, q.cuda(), *dev, desc, torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
            longest, scale, part)
    if entry == "noalloc":
        pkv.pkv_paged_decode_noalloc(*args)
    else:
        pkv.pkv_paged_decode(*args, ws)
    assert pkv.pkv_get_device_error() == 0
    k, v = (np.concatenate([_rows(*p, table[i], n, block, s) for i, n in enumerate(lens)]) for p, s in zip(pools, scales))
    ref, size = prompt.prompt_attention(q.double().numpy(), k, v, [1] * len(lens), lens, scale)
    _close(out, ref, _bound(ref, size, DT[dtype]))
    return out


RAGGED = [1, 15, 16, 17, 31, 32, 33, 255, 700]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(4, 4), (8, 1), (6, 2), (28, 4), (5, 1), (10, 5)])
def test_decode_groups(hq, hkv, dim, dtype):
    _run_decode(RAGGED, hq, hkv, dim, dtype, seed=hq + dim)


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("part", [0, 16, 48, 512])
@pytest.mark.parametrize("dim", [64, 128])
def test_decode_blocks_and_partitions(dim, part, block):
    _run_decode(RAGGED + [2049], 8, 2, dim, "bf16", block=block, part=part, scaled=part % 32 == 0, seed=part)


@pytest.mark.parametrize("lens", [[1], [16], [0], [0, 5, 0], [4000], [3, 9000], [1] * 300, [40] * 65])
def test_decode_lengths(lens):
    _run_decode(lens, 7, 1, 128, "f16", seed=len(lens))


@pytest.mark.parametrize("scale", [0.0, -0.1])
def test_decode_with_a_zero_or_negative_scale(scale):
    _run_decode(RAGGED, 8, 2, 128, "bf16", seed=8, scale=scale)


@pytest.mark.parametrize("lens,hq,hkv,dim", [([20000], 8, 1, 64), ([9001, 17], 4, 2, 128), ([0, 30001, 5], 3, 1, 128),
                                            ([4099] * 9, 6, 3, 64)])
def test_decode_of_few_long_sequences(lens, hq, hkv, dim):
    """Fewer workers than warps, and merges that a CTA's warps share."""
    _run_decode(lens, hq, hkv, dim, "bf16", seed=len(lens) + dim)


def test_decode_large_batch_takes_the_four_warp_layout():
    """12 prefix bytes per sequence next to 12 warps' stages: past about 9,900 sequences four warps run."""
    rng = np.random.default_rng(4)
    _run_decode([int(n) for n in rng.integers(1, 20, 11000)], 1, 1, 128, "bf16", seed=5)


@pytest.mark.parametrize("length", [40, 5000])
@pytest.mark.parametrize("which", ["k", "v"])
def test_a_nan_in_an_attended_row_reaches_its_head_only(which, length):
    """One sequence inside a worker's range, one split over workers and merged."""
    import paged_kv_cache_160_gb300 as pkv
    lens, hq, hkv, dim = [length, 30], 4, 2, 128
    rng, table, pools, _ = _decode_case(31, lens, hq, hkv, dim, 16, False)
    codes, sc = pools[0 if which == "k" else 1]
    j = length // 2
    sc[table[0, j // 16], 1, j % 16, 3] = 0x7F                 # 16 elements of kv head 1
    k, v = (torch.from_numpy(fp4.pack(*p)).cuda() for p in pools)
    q = torch.from_numpy(rng.standard_normal((2, hq, dim))).to(torch.bfloat16).cuda()
    out = torch.empty_like(q)
    ws = torch.empty(pkv.pkv_decode_workspace_bytes(2, hq, hkv, dim, 16, length, 0), dtype=torch.uint8, device="cuda")
    pkv.pkv_paged_decode(out, q, k, v, pkv.cache_desc_fp4(k), torch.from_numpy(table).cuda(),
                         torch.tensor(lens, dtype=torch.int32, device="cuda"), length, 0.09, 0, ws)
    assert pkv.pkv_get_device_error() == 0
    nan = torch.isnan(out).cpu()
    want = torch.zeros_like(nan)
    want[0, 2:] = True if which == "k" else torch.arange(dim) // 16 == 3
    assert torch.equal(nan, want)


def test_decode_no_alloc_is_bit_identical():
    a = _run_decode(RAGGED, 8, 2, 128, "bf16", seed=9)
    b = _run_decode(RAGGED, 8, 2, 128, "bf16", seed=9, entry="noalloc")
    assert torch.equal(a, b)


def test_decode_under_an_sm_budget():
    import paged_kv_cache_160_gb300 as pkv
    try:
        for n in (1, 7, 66):
            pkv.pkv_set_decode_sm_budget(n)
            _run_decode(RAGGED, 8, 2, 128, "f16", seed=10)
    finally:
        pkv.pkv_set_decode_sm_budget(0)


def test_decode_reports_bad_blocks_and_lengths():
    import paged_kv_cache_160_gb300 as pkv
    k = torch.zeros(pkv.fp4_cache_shape(4, 1, 16, 64), dtype=torch.uint8, device="cuda")
    desc = pkv.cache_desc_fp4(k)
    q = torch.ones((2, 1, 64), dtype=torch.float16, device="cuda")
    out = torch.empty_like(q)
    ws = torch.empty(pkv.pkv_decode_workspace_bytes(2, 1, 1, 64, 16, 64, 0), dtype=torch.uint8, device="cuda")
    for table, lens, bit in (([[0, 4], [1, 2]], [20, 20], "block_id"), ([[0, 1], [2, 3]], [33, 5], "context_len")):
        pkv.pkv_paged_decode(out, q, k, k, desc, torch.tensor(table, dtype=torch.int32, device="cuda"),
                             torch.tensor(lens, dtype=torch.int32, device="cuda"), 64, 0.125, 0, ws)
        assert pkv.pkv_get_device_error() == pkv.DEVERR[bit]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim,block,scaled", [(128, 16, True), (128, 32, False), (64, 16, False), (64, 32, True)])
def test_append_equals_write_then_decode(dim, block, scaled, dtype):
    import paged_kv_cache_160_gb300 as pkv
    lens, hq, hkv = [1, 16, 17, 32, 33, 500, 0, 2048], 8, 2
    rng, table, pools, scales = _decode_case(3, lens, hq, hkv, dim, block, scaled)
    host = [torch.from_numpy(fp4.pack(*p)) for p in pools]
    sc = [torch.from_numpy(s).cuda() if scaled else None for s in scales]
    q, kn, vn = (torch.from_numpy(rng.standard_normal((len(lens), h, dim)) * 2).to(DT[dtype]).cuda() for h in (hq, hkv, hkv))
    slots = torch.tensor([int(table[i, (n - 1) // block]) * block + (n - 1) % block if n else -1
                          for i, n in enumerate(lens)], device="cuda")
    tab, ln = torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = torch.empty(pkv.pkv_decode_workspace_bytes(len(lens), hq, hkv, dim, block, 2048, 0), dtype=torch.uint8, device="cuda")
    got = []
    for fused in (False, True):
        k, v = host[0].cuda(), host[1].cuda()
        desc = pkv.cache_desc_fp4(k, *sc)
        out = torch.empty_like(q)
        tail = (tab, ln, 2048, dim ** -0.5, 0, ws)
        if fused:
            pkv.pkv_paged_decode_append(out, q, kn, vn, k, v, desc, *tail)
        else:
            pkv.pkv_kv_write(kn, vn, slots, k, v, desc)
            pkv.pkv_paged_decode(out, q, k, v, desc, *tail)
        assert pkv.pkv_get_device_error() == 0
        got.append((out, k, v))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert torch.isfinite(got[0][0]).all()


def test_copies_and_swaps_move_whole_4_bit_blocks():
    import paged_kv_cache_160_gb300 as pkv
    rng = np.random.default_rng(12)
    shape = pkv.fp4_cache_shape(8, 3, 32, 64)
    k, v = (torch.from_numpy(rng.integers(0, 256, shape).astype(np.uint8)) for _ in range(2))
    dk, dv = k.cuda(), v.cuda()
    desc = pkv.cache_desc_fp4(dk)
    pkv.pkv_copy_blocks(dk, dv, desc, torch.tensor([[0, 5], [7, 2]], dtype=torch.int32, device="cuda"))
    wk, wv = k.clone(), v.clone()
    for t in (wk, wv):
        t[5], t[2] = t[0].clone(), t[7].clone()
    assert torch.equal(dk.cpu(), wk) and torch.equal(dv.cpu(), wv)
    hk, hv = torch.zeros((2,) + shape[1:], dtype=torch.uint8).pin_memory(), torch.zeros((2,) + shape[1:], dtype=torch.uint8).pin_memory()
    pkv.pkv_swap_blocks(hk, hv, dk, dv, desc, torch.tensor([[3, 0], [5, 1]], dtype=torch.int32, device="cuda"))
    assert pkv.pkv_get_device_error() == 0
    assert torch.equal(hk, wk[[3, 5]]) and torch.equal(hv, wv[[3, 5]])


def test_write_read_decode_captured_and_replayed():
    import paged_kv_cache_160_gb300 as pkv
    rng, table, pools, _ = _decode_case(21, [100, 40], 4, 2, 128, 16, False)
    k, v = (torch.from_numpy(fp4.pack(*p)).cuda() for p in pools)
    desc = pkv.cache_desc_fp4(k)
    q, kn, vn = (torch.from_numpy(rng.standard_normal((2, h, 128))).to(torch.bfloat16).cuda() for h in (4, 2, 2))
    tab, lens = torch.from_numpy(table).cuda(), torch.tensor([100, 40], dtype=torch.int32, device="cuda")
    slots = torch.tensor([int(table[0, 6]) * 16 + 3, int(table[1, 2]) * 16 + 7], device="cuda")
    cu = torch.tensor([0, 100, 140], dtype=torch.int32, device="cuda")
    out, ko, vo = torch.empty_like(q), *(torch.empty((140, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = torch.empty(pkv.pkv_decode_workspace_bytes(2, 4, 2, 128, 16, 100, 0), dtype=torch.uint8, device="cuda")

    def step():
        pkv.pkv_kv_write(kn, vn, slots, k, v, desc)
        pkv.pkv_kv_read(ko, vo, cu, tab, k, v, desc)
        pkv.pkv_paged_decode(out, q, k, v, desc, tab, lens, 100, 0.09, 0, ws)

    step()
    torch.cuda.synchronize()
    eager = [t.clone() for t in (out, ko, vo)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for t in (out, ko, vo):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((out, ko, vo), eager))
    assert pkv.pkv_get_device_error() == 0


@pytest.mark.parametrize("dim,dtype,exponent", [(128, "bf16", -20), (64, "bf16", -20), (128, "f16", -20), (128, "bf16", -118),
                                                (64, "bf16", 20), (128, "bf16", 100)])
def test_decode_of_queries_far_below_and_above_one(dim, dtype, exponent):
    """Queries of size 2^exponent under head scales of the inverse size: scores of ordinary size.  Half of the query
    heads are another 2^-9 smaller."""
    import paged_kv_cache_160_gb300 as pkv
    lens, hq, hkv = RAGGED + [3000], 8, 2
    rng, table, pools, scales = _decode_case(200 + exponent, lens, hq, hkv, dim, 16, True)
    scales[0] = scales[0] * np.float32(2.0) ** -exponent
    dev = [torch.from_numpy(fp4.pack(*p)).cuda() for p in pools]
    desc = pkv.cache_desc_fp4(dev[0], *(torch.from_numpy(s).cuda() for s in scales))
    q = rng.standard_normal((len(lens), hq, dim)) * 2.0 ** exponent
    q[:, 1::2] *= 2.0 ** -9 if dtype == "bf16" else 1.0
    q = torch.from_numpy(q).to(DT[dtype])
    out = torch.empty(q.shape, dtype=DT[dtype], device="cuda")
    ws = torch.empty(pkv.pkv_decode_workspace_bytes(len(lens), hq, hkv, dim, 16, 3000, 0), dtype=torch.uint8, device="cuda")
    pkv.pkv_paged_decode(out, q.cuda(), *dev, desc, torch.from_numpy(table).cuda(),
                         torch.tensor(lens, dtype=torch.int32, device="cuda"), 3000, dim ** -0.5, 0, ws)
    assert pkv.pkv_get_device_error() == 0
    k, v = (np.concatenate([_rows(*p, table[i], n, 16, s) for i, n in enumerate(lens)]) for p, s in zip(pools, scales))
    ref, size = prompt.prompt_attention(q.double().numpy(), k, v, [1] * len(lens), lens, dim ** -0.5)
    _close(out, ref, _bound(ref, size, DT[dtype]))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_a_query_that_is_not_finite_reaches_its_own_head_only(dtype):
    import paged_kv_cache_160_gb300 as pkv
    lens, hq, hkv, dim = [70, 2000, 33], 8, 2, 128
    rng, table, pools, _ = _decode_case(33, lens, hq, hkv, dim, 16, False)
    k, v = (torch.from_numpy(fp4.pack(*p)).cuda() for p in pools)
    q = torch.from_numpy(rng.standard_normal((3, hq, dim))).to(DT[dtype])
    q[2, 5] = 0.0                                              # a row of zeros: the mean of its values
    broken = q.clone()
    broken[0, 1, 5], broken[1, 6, 100] = float("inf"), float("nan")
    ws = torch.empty(pkv.pkv_decode_workspace_bytes(3, hq, hkv, dim, 16, 2000, 0), dtype=torch.uint8, device="cuda")
    outs = []
    for x in (q, broken):
        out = torch.empty(q.shape, dtype=DT[dtype], device="cuda")
        pkv.pkv_paged_decode(out, x.cuda(), k, v, pkv.cache_desc_fp4(k), torch.from_numpy(table).cuda(),
                             torch.tensor(lens, dtype=torch.int32, device="cuda"), 2000, dim ** -0.5, 0, ws)
        outs.append(out.cpu())
    assert pkv.pkv_get_device_error() == 0
    hit = torch.zeros((3, hq), dtype=torch.bool)
    hit[0, 1] = hit[1, 6] = True
    assert torch.isnan(outs[1][hit]).all() and torch.equal(outs[1][~hit], outs[0][~hit])
    rows = _rows(*pools[1], table[2], 33, 16, None)[:, 1]
    _close(outs[0][2, 5], rows.mean(0), _bound(rows.mean(0), np.abs(rows).mean(0), DT[dtype]))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("seqs", [1000, 5000, 8000])
def test_decode_and_append_of_large_batches(seqs, dim):
    """12 prefix bytes per sequence beside the warps' stages: 12 warps run up to about 900 sequences, 8 up to about
    7,040, then 4."""
    import paged_kv_cache_160_gb300 as pkv
    rng = np.random.default_rng(seqs + dim)
    lens, hq, hkv = [int(n) for n in rng.integers(0, 40, seqs)], 3, 1
    lens[seqs // 2] = 700
    _run_decode(lens, hq, hkv, dim, "bf16", seed=seqs)
    _, table, pools, _ = _decode_case(seqs + 1, lens, hq, hkv, dim, 16, False)
    host = [torch.from_numpy(fp4.pack(*p)) for p in pools]
    q, kn, vn = (torch.from_numpy(rng.standard_normal((seqs, h, dim))).to(torch.bfloat16).cuda() for h in (hq, hkv, hkv))
    slots = torch.tensor([int(table[i, (n - 1) // 16]) * 16 + (n - 1) % 16 if n else -1 for i, n in enumerate(lens)],
                         device="cuda")
    tail = (torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), 700, dim ** -0.5, 0,
            torch.empty(pkv.pkv_decode_workspace_bytes(seqs, hq, hkv, dim, 16, 700, 0), dtype=torch.uint8, device="cuda"))
    got = []
    for fused in (False, True):
        k, v = host[0].cuda(), host[1].cuda()
        out = torch.empty_like(q)
        if fused:
            pkv.pkv_paged_decode_append(out, q, kn, vn, k, v, pkv.cache_desc_fp4(k), *tail)
        else:
            pkv.pkv_kv_write(kn, vn, slots, k, v, pkv.cache_desc_fp4(k))
            pkv.pkv_paged_decode(out, q, k, v, pkv.cache_desc_fp4(k), *tail)
        assert pkv.pkv_get_device_error() == 0
        got.append((out, k, v))
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_batches_past_the_limit_are_refused():
    import paged_kv_cache_160_gb300 as pkv
    for seqs, dim in ((13100, 64), (13100, 128), (13300, 64), (13300, 128)):
        k = torch.zeros(pkv.fp4_cache_shape(1, 1, 16, dim), dtype=torch.uint8, device="cuda")
        q = torch.ones((seqs, 1, dim), dtype=torch.bfloat16, device="cuda")
        out = torch.full_like(q, 7.0)
        ws = torch.empty(pkv.pkv_decode_workspace_bytes(seqs, 1, 1, dim, 16, 16, 0), dtype=torch.uint8, device="cuda")
        args = (out, q, k, k, pkv.cache_desc_fp4(k), torch.zeros((seqs, 1), dtype=torch.int32, device="cuda"),
                torch.full((seqs,), 3, dtype=torch.int32, device="cuda"), 16, 0.1, 0, ws)
        if seqs < 13150:
            pkv.pkv_paged_decode(*args)
            assert pkv.pkv_get_device_error() == 0 and (out == 0).all()
        else:
            with pytest.raises(pkv.PkvError):
                pkv.pkv_paged_decode(*args)
            assert (out == 7.0).all()


def test_append_from_pinned_host_memory():
    import paged_kv_cache_160_gb300 as pkv
    lens, hq, hkv, dim = [1, 16, 0, 500, 3000], 8, 2, 128
    rng, table, pools, scales = _decode_case(46, lens, hq, hkv, dim, 16, True)
    host = [torch.from_numpy(fp4.pack(*p)) for p in pools]
    x = [torch.from_numpy(rng.standard_normal((len(lens), h, dim))).to(torch.bfloat16) for h in (hq, hkv, hkv)]
    x += [torch.from_numpy(table), torch.tensor(lens, dtype=torch.int32)]
    ws = torch.empty(pkv.pkv_decode_workspace_bytes(len(lens), hq, hkv, dim, 16, 3000, 0), dtype=torch.uint8, device="cuda")
    got = []
    for put in (torch.Tensor.cuda, torch.Tensor.pin_memory):
        k, v = host[0].cuda(), host[1].cuda()
        desc = pkv.cache_desc_fp4(k, *(torch.from_numpy(s).cuda() for s in scales))
        q, kn, vn, tab, ln = (put(t) for t in x)
        out = put(torch.zeros(x[0].shape, dtype=torch.bfloat16))
        pkv.pkv_paged_decode_append(out, q, kn, vn, k, v, desc, tab, ln, 3000, dim ** -0.5, 0, ws)
        assert pkv.pkv_get_device_error() == 0                 # (waits)
        got.append((out.cpu(), k, v))
    for a, b in zip(*got):
        assert torch.equal(a, b)
