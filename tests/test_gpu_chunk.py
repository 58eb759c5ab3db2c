"""GPU parity of pkv_paged_chunk_attention against float64.

With A = sum_j p_j |v_j|, u = finfo.eps / 2 of q's type and w that of the exponentials' type (q's; fp16 over a quantised
cache): the exponentials are rounded to that type (w A; as fp16, those below its least normal, 2^-14, by at most 2^-25 where
the row's largest is 2^7 or more: N 2^-32 max |v| over N keys, under 2^-15 for the N here and small beside w A); scores are fp32 sums of at most
128 exact products, an error of the exponent below 2^-24 * 128 * scale * sum |q k| (under 2^-12 here), and bf16 rows that
are taken as fp16 lose at most 2^-25 of their largest element; exp2 and the fp32 sums add less than 2^-13.  So
|err| <= (w + 2^-11) A + u |out| + 2^-25, and |err| <= 2^-11 + 2^-22 |lse| for the log of the sum.
"""
import numpy as np
import pytest
import torch

from oracle import evict, fp4
from tests.paged import DT, Paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def _kv(kind, dtype):
    return dtype if kind == "same" else kind


class Case:
    def __init__(self, starts, news, hq, hkv, dim, dtype, kind, block=16, seed=0, pad=0, spread=1.0, scaled=True,
                 max_blocks=None):
        import paged_kv_cache_160_gb300 as pkv
        self.pkv, self.starts, self.news, self.hq, self.dtype, self.pad = pkv, starts, news, hq, dtype, pad
        self.cache = Paged([s + n for s, n in zip(starts, news)], _kv(kind, dtype), hkv, dim, block, scaled, seed,
                           max_blocks=max_blocks)
        g = torch.Generator().manual_seed(seed + 7 * sum(news) + hq)
        self.total = sum(news)
        self.q = (spread * torch.randn((self.total + pad, hq, dim), generator=g)).to(DT[dtype])
        self.q[self.total:] = float("nan")
        self.scale = dim ** -0.5
        self.cu = np.cumsum([0] + list(news)).astype(np.int32)
        self.dev()

    def dev(self):
        self.q_dev = self.q.cuda()
        self.cu_dev = torch.from_numpy(self.cu).cuda()
        self.start_dev = torch.tensor(self.starts, dtype=torch.int32, device="cuda")
        self.out = torch.full(self.q.shape, 5.0, dtype=DT[self.dtype], device="cuda")
        self.lse = torch.full(self.q.shape[:2], 7.0, device="cuda")
        c = self.cache
        self.ws = torch.full((self.pkv.pkv_chunk_workspace_bytes(self.q.shape[0], self.hq, c.heads, c.dim),), 0xFF,
                             dtype=torch.uint8, device="cuda")

    def call(self, lse=True, stream=None):
        c = self.cache
        self.pkv.pkv_paged_chunk_attention(self.out, self.q_dev, self.cu_dev, self.start_dev, c.k_cache, c.v_cache, c.desc,
                                           c.dev_tables, self.scale, self.ws, self.lse if lse else None, stream)

    def check(self, lse=True, only=None):
        u = torch.finfo(DT[self.dtype]).eps / 2
        w = 2.0 ** -11 if self.cache.kv not in DT else u
        got, got_lse = self.out.double().cpu().numpy(), self.lse.double().cpu().numpy()
        assert (got[self.total:] == 5.0).all() and (got_lse[self.total:] == 7.0).all()
        q = self.q.double().numpy()
        for i, (s, n) in enumerate(zip(self.starts, self.news)):
            if n == 0 or (only is not None and i not in only):
                continue
            a, b = self.cu[i], self.cu[i + 1]
            k, v = (self.cache.rows(x, i, s + n) for x in "kv")
            ref, ref_lse, size = evict.chunk_attention(q[a:b], k, v, s, self.scale)
            err, bound = np.abs(got[a:b] - ref), (w + 2.0 ** -11) * size + u * np.abs(ref) + 2.0 ** -25
            assert (err <= bound).all(), (i, float(np.nanmax(err / bound)), np.argwhere(~(err <= bound))[:3])
            if lse:
                e = np.abs(got_lse[a:b] - ref_lse)
                assert (e <= 2.0 ** -11 + 2.0 ** -22 * np.abs(ref_lse)).all(), (i, float(np.nanmax(e)))
        if not lse:
            assert (got_lse == 7.0).all()


def _run(*a, lse=True, **k):
    c = Case(*a, **k)
    c.call(lse)
    assert c.pkv.pkv_get_device_error() == 0
    c.check(lse)
    return c


KINDS = ["fp4", "e4m3", "same"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("block", [16, 32])
def test_ragged(kind, dtype, dim, block):
    _run([0, 7, 127, 128, 129, 0, 300, 15], [1, 3, 1, 2, 0, 20, 5, 2], 6, 2, dim, dtype, kind, block=block, pad=3)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 127, 128, 129, 256, 257, 400])
def test_whole_prompt(kind, n):
    _run([0], [n], 2, 1, 128, "bf16", kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("start", [1, 111, 112, 127, 128, 255, 1000, 5000])
@pytest.mark.parametrize("n", [1, 4, 37])
def test_history(kind, start, n):
    _run([start], [n], 7, 1, 128, "bf16", kind)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (5, 5), (8, 1), (28, 4), (40, 1), (129, 1), (300, 2)])
@pytest.mark.parametrize("n", [1, 3, 50])
def test_heads(hq, hkv, n):
    _run([90, 0], [n, 2], hq, hkv, 64, "f16", "fp4", pad=1)


@pytest.mark.parametrize("kind", KINDS)
def test_few_rows_over_many_keys(kind):
    _run([40000], [2], 4, 2, 128, "bf16", kind)
    _run([20011, 3, 9000], [1, 2, 3], 3, 1, 64, "f16", kind)


@pytest.mark.parametrize("kind", KINDS)
def test_many_sequences(kind):
    rng = np.random.default_rng(5)
    starts = [int(x) for x in rng.integers(0, 150, 700)]
    news = [int(x) for x in rng.integers(0, 3, 700)]
    _run(starts, news, 2, 1, 64, "bf16", kind, pad=2)


@pytest.mark.parametrize("kind", KINDS)
def test_long_and_short_together(kind):
    _run([600] + [3] * 20 + [0], [300] + [1] * 20 + [200], 4, 2, 128, "f16", kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows", [600, 300, 90])
def test_many_items_for_every_sm(kind, rows):
    """Blocks of 256 rows and remainders in turn, many for each SM."""
    c = Case([5] * 40, [rows] * 40, 8, 8, 64, "bf16", kind, pad=1)
    for _ in range(5):
        c.out[:c.total] = 5.0
        c.call()
        assert c.pkv.pkv_get_device_error() == 0
        if _ == 0:
            first = c.out.clone()
        assert torch.equal(first, c.out)
    c.check(only=[0, 23] if rows < 600 else [31])


def test_without_lse():
    _run([100, 2000], [5, 5], 4, 2, 128, "bf16", "fp4", lse=False)
    _run([100, 2000], [5, 5], 4, 2, 128, "bf16", "same", lse=False)


@pytest.mark.parametrize("kind", ["fp4", "e4m3"])
@pytest.mark.parametrize("size", [1e-30, 1e-4, 3e4, 1e30])
def test_bf16_queries_of_any_size(kind, size):
    """Rows of very different sizes; the scale keeps the scores of the largest within reach."""
    c = Case([200], [6], 2, 1, 128, "bf16", kind)
    f = torch.tensor([1.0, 2.0 ** -20, 2.0 ** -60, 2.0 ** -3, 1.5, 0.0])[:, None, None]
    c.q = (c.q.float() * f * size).to(torch.bfloat16)
    c.scale = 128 ** -0.5 / size
    c.dev()
    c.call()
    assert c.pkv.pkv_get_device_error() == 0
    c.check()


@pytest.mark.parametrize("size", [1, 60])
def test_scales_far_from_one(size):
    """Scales of 2^123 and 2^-123 between queries and keys of 2^-60 and 2^60 in bf16: the scores are ordinary ones."""
    for e in (size, -size):
        c = Case([200, 3], [6, 40], 2, 1, 128, "bf16", "same")
        k = torch.from_numpy(c.cache.stored[0]).view(torch.bfloat16)
        c.cache.stored[0] = (k.float() * 2.0 ** e).to(torch.bfloat16).view(torch.int16).numpy()
        c.cache.upload()
        c.q = (c.q.float() * 2.0 ** e).to(torch.bfloat16)
        c.scale = 128 ** -0.5 * 2.0 ** (-2 * e)
        c.dev()
        c.call()
        assert c.pkv.pkv_get_device_error() == 0
        c.check()


@pytest.mark.parametrize("kind", ["fp4", "e4m3"])
def test_head_scales_of_any_sign(kind):
    c = Case([150], [9], 8, 4, 64, "f16", kind)
    c.cache.scales = [np.array([-1.2, 0.5, 0.0, 2.0 ** -30], np.float32), np.array([1.0, -3.0, 0.7, 2.0 ** 10], np.float32)]
    c.cache.upload()
    c.dev()
    c.call()
    assert c.pkv.pkv_get_device_error() == 0
    c.check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("start,n", [(70, 6), (0, 300), (250, 20)])
def test_what_a_row_does_not_see(kind, start, n):
    """Infinities and NaN in stale rows, unused blocks and later tokens reach no row that does not see them."""
    c = Case([start], [n], 4, 2, 128, "bf16", kind, seed=3)
    cc, pos = c.cache, start + n - 2                              # the last two tokens are bad
    nan = {"fp4": None, "e4m3": 0x7F, "bf16": 0x7FC0}[cc.kv]
    for which, stored in enumerate(cc.stored):
        rows = {(int(cc.tables[0, p // 16]), p % 16) for p in range(start + n)}
        for b in range(cc.num_blocks):
            for r in range(16):
                if (b, r) in rows and not (cc.tables[0, pos // 16] == b and r == pos % 16):
                    continue
                if cc.kv == "fp4":
                    stored[b, :, 0, 8 * 128 + 8 * r + 3] = 0x7F       # 16 of the row's values
                else:
                    stored[b, :, r, 5::7] = nan
                    if cc.kv == "bf16" and which == 1:
                        stored[b, :, r, 4::7] = 0x7F80            # infinity
    cc.upload()
    c.dev()
    c.call()
    assert c.pkv.pkv_get_device_error() == 0
    got = c.out.double().cpu().numpy()
    q = c.q.double().numpy()
    k, v = (cc.rows(x, 0, start + n) for x in "kv")
    ref, _, size = evict.chunk_attention(q, k, v, start, c.scale)
    m = n - 2
    assert np.isfinite(ref[:m]).all()
    u, w = 2.0 ** -8, 2.0 ** -11 if cc.kv not in DT else 2.0 ** -8
    assert (np.abs(got[:m] - ref[:m]) <= (w + 2.0 ** -11) * size[:m] + u * np.abs(ref[:m]) + 2.0 ** -25).all()
    assert np.isnan(got[m:]).all()                                # NaN scores


@pytest.mark.parametrize("kind", KINDS)
def test_non_finite_values_reach_those_who_see_them(kind):
    c = Case([100], [8], 2, 1, 128, "f16", kind, seed=4)
    cc, pos = c.cache, 104
    b, r = cc.tables[0, pos // 16], pos % 16
    if cc.kv == "fp4":
        cc.stored[1][b, 0, 0, 8 * 128 + 8 * r + 3] = 0x7F
    elif cc.kv == "e4m3":
        cc.stored[1][b, 0, r, 48:64] = 0x7F
    else:
        cc.stored[1][b, 0, r, 48:64] = 0x7C00                     # infinity
    cc.upload()
    c.dev()
    c.call()
    assert c.pkv.pkv_get_device_error() == 0
    got = c.out.float().cpu().numpy()
    assert np.isfinite(got[:4]).all()
    bad = np.isinf if cc.kv in DT else np.isnan
    assert bad(got[4:, :, 48:64]).all()
    assert np.isfinite(got[4:, :, :48]).all() and np.isfinite(got[4:, :, 64:]).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows", [1, 40, 200])
def test_many_small_weights_behind_a_large_one(kind, rows):
    """One key has nearly all of the weight and a value of zero; 2^17 others have e^-18 of it each and values of one.

    As many chunks as SMs over the same blocks, so that no SM sees a part of the keys alone.  An exponential below 2^-14 is
    rounded to a multiple of 2^-24 as fp16, where that of the row's largest key is 2^7 or more: an error of at most 2^-32 of
    that one each, N 2^-32 max |v| in all (2^-15 here)."""
    n, dim, sms = 131072, 64, torch.cuda.get_device_properties(0).multi_processor_count
    c = Case([n - rows], [rows], 1, 1, dim, "f16", kind, scaled=False)
    cc = c.cache
    k, v = np.zeros((cc.num_blocks, 1, 16, dim)), np.ones((cc.num_blocks, 1, 16, dim))
    b = cc.tables[0, 0]
    k[b, 0, 0, 0], v[b, 0, 0] = 6.0, 0.0
    cc.scales = [None, None]
    if kind == "fp4":
        cc.stored = [fp4.pack(*fp4.quantise(x)) for x in (k, v)]
    elif kind == "e4m3":
        cc.scales = [np.ones(1, np.float32)] * 2
        cc.stored = [torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy() for x in (k, v)]
    else:
        cc.stored = [torch.from_numpy(x).to(torch.float16).view(torch.int16).numpy() for x in (k, v)]
    cc.tables = np.repeat(cc.tables, sms, 0)
    cc.upload()
    c.q = torch.zeros((sms * rows, 1, dim), dtype=torch.float16)
    c.q[:, :, 0] = 24.0
    c.cu, c.starts, c.total = np.arange(sms + 1, dtype=np.int32) * rows, [n - rows] * sms, sms * rows
    c.dev()
    c.call()
    assert c.pkv.pkv_get_device_error() == 0
    others = np.arange(n - rows, n) * np.exp(-18.0)
    one = cc.rows("v", 0, 2)[1, 0, 0]                          # (as stored: 1.03125 in 4 bits)
    ref = one * (others / (1 + others))[:, None, None]
    err = np.abs(c.out.double().cpu().numpy().reshape(sms, rows, 1, dim) - ref)
    bound = 2.0 ** -10 * ref + 2.0 ** -11 * ref + one * n * 2.0 ** -32
    worst = float((err / bound).max())
    assert worst <= 1
    e = np.abs(c.lse.double().cpu().numpy().reshape(sms, rows) - (18.0 + np.log1p(others)))
    assert (e <= 2.0 ** -11).all()


@pytest.mark.parametrize("kind", ["e4m3", "same"])
@pytest.mark.parametrize("rows", [8, 40, 200])
@pytest.mark.parametrize("first,apart,steps,alone", [(1024, 6, (2, 5, 5, 3), True), (1024, 6, (2.5, 5, 5, 3.5), True),
                                                     (1024, 1, (2, 6, 6, 3), False), (1024, 1, (7, 5, 8, 3), False),
                                                     (1915, 1, (8, 6, 6, 2), False)])
def test_scores_of_many_millions_that_differ_a_little(kind, rows, first, apart, steps, alone):
    """Scores of 12.6 to 27 million, where fp32 maxima in units of log2 are multiples of 2 or 4: no exponential may leave
    fp16's range because of the maximum's own rounding.  (Not alone: as many chunks as SMs, so that an SM sees all of a
    row's keys.)

    fp32 holds whole numbers up to 2^24 and even ones up to 2^25, as the scores of whole and even steps are: their sums and,
    a fused product less the maximum, the exponentials' arguments are exact.  Other steps and scores may be rounded to such a
    number on either side, at most 2 away: a weight that is wrong by a factor of e^2 at most, |err| <= 2 (e^2 - 1) A."""
    start, dim, n = 700, 64, 1 if alone else torch.cuda.get_device_properties(0).multi_processor_count
    c = Case([start], [rows], 1, 1, dim, "f16", kind)
    cc = c.cache
    h = 32.0 if kind == "e4m3" else 1.0
    k = np.zeros((cc.num_blocks, 1, 16, dim))
    k[..., 0] = 12288.0 / h
    for j, step in zip((300, 450, 460, 600), steps):           # (5 is 7.2 in units of log2)
        k[cc.tables[0, j // 16], 0, j % 16, 1] = step / h
    if kind == "e4m3":
        cc.scales[0] = np.full(1, h, np.float32)
        cc.stored[0] = torch.from_numpy(k).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    else:
        cc.stored[0] = torch.from_numpy(k).to(torch.float16).view(torch.int16).numpy()
    cc.upload()
    assert np.array_equal(cc.k, k * h)
    c.q[:] = 0
    c.q[:, 0, 0] = float(first) + apart * torch.arange(rows)
    c.q[:, 0, 1] = 1.0
    c.scale = 1.0
    q = c.q.double().numpy()
    ref, _, size = evict.chunk_attention(q, cc.rows("k", 0, start + rows), cc.rows("v", 0, start + rows), start, 1.0)
    c.q, cc.tables = c.q.repeat(n, 1, 1), np.repeat(cc.tables, n, 0)
    cc.upload()
    c.cu, c.starts, c.total = np.arange(n + 1, dtype=np.int32) * rows, [start] * n, n * rows
    c.dev()
    c.call()
    assert c.pkv.pkv_get_device_error() == 0
    got = c.out.double().cpu().numpy().reshape(n, rows, 1, dim)
    assert np.isfinite(got).all()
    top = q[:, 0, 0] * 12288 + max(steps)
    exact = (top <= 2.0 ** 24) & all(x == int(x) for x in steps) | (top <= 2.0 ** 25) & all(x % 2 == 0 for x in steps)
    slack = np.where(exact, 2.0 ** -10, 2 * (np.exp(2) - 1))[:, None, None]
    worst = float((np.abs(got - ref) / (slack * size + 2.0 ** -11 * np.abs(ref) + 2.0 ** -25)).max())
    assert worst <= 1


def test_inconsistent_lengths():
    import paged_kv_cache_160_gb300 as pkv
    for what in ("start", "past_table", "descending", "past_total", "first"):
        c = Case([40, 50, 60], [2, 3, 4], 4, 2, 64, "bf16", "fp4", pad=0)
        good = [0, 1, 2]
        if what == "start":
            c.start_dev[1] = -1
            good = [0, 2]
        elif what == "past_table":
            c.start_dev[2] = 62
            good = [0, 1]
        elif what == "descending":
            c.cu_dev[2] = 1
            good = [0]
        elif what == "past_total":
            c.cu_dev[3] = 10
            good = [0, 1]
        else:
            c.cu_dev[0] = 1
            good = [1, 2]
        c.call()
        assert pkv.pkv_get_device_error() == pkv.DEVERR["chunk"], what
        c.check(only=good)
        if what in ("start", "past_table", "past_total"):
            i = ({0, 1, 2} - set(good)).pop()
            assert (c.out[c.cu[i]:c.cu[i + 1]] == 5.0).all() and (c.lse[c.cu[i]:c.cu[i + 1]] == 7.0).all()


@pytest.mark.parametrize("kind", KINDS)
def test_block_ids_outside_the_pool(kind):
    import paged_kv_cache_160_gb300 as pkv
    c = Case([300, 40], [3, 2], 4, 2, 128, "bf16", kind)
    for bad in (-1, c.cache.num_blocks, 1 << 30, -(1 << 31)):
        c.cache.dev_tables[0, 5] = bad
        c.out.fill_(5.0)
        c.call()
        assert pkv.pkv_get_device_error() == pkv.DEVERR["block_id"]
        c.check(only=[1])
        assert torch.isfinite(c.out).all()
    # the block's keys and values count as zeros
    cc = c.cache
    cc.k, cc.v = cc.k.copy(), cc.v.copy()
    b = cc.tables[0, 5]
    cc.k[b] = 0
    cc.v[b] = 0
    c.check(only=[0])


def test_entries_behind_the_sequence_are_not_read():
    c = Case([30], [2], 4, 2, 128, "bf16", "fp4", max_blocks=9)
    c.cache.dev_tables[0, 2:] = 1 << 29
    c.call()
    assert c.pkv.pkv_get_device_error() == 0
    c.check()


def test_same_bits_every_time_and_a_shared_workspace():
    a = Case([5000, 100], [4, 9], 8, 2, 128, "bf16", "fp4")
    b = Case([700, 3000, 9], [200, 1, 9], 4, 1, 128, "f16", "e4m3")
    ws = a.ws if a.ws.numel() >= b.ws.numel() else b.ws
    a.ws = b.ws = ws
    a.call()
    b.call()
    first = [t.clone() for t in (a.out, a.lse, b.out, b.lse)]
    for _ in range(3):
        b.call()
        a.call()
    assert all(torch.equal(x, y) for x, y in zip(first, (a.out, a.lse, b.out, b.lse)))
    a.check()
    b.check()


def test_captured_graphs_and_another_stream():
    a = Case([5000, 100], [4, 9], 8, 2, 128, "bf16", "fp4")
    b = Case([3000, 0], [3, 160], 4, 1, 64, "f16", "same")
    b.ws = a.ws if a.ws.numel() >= b.ws.numel() else b.ws
    a.ws = b.ws
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        for c in (a, b):
            c.call()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                c.call()
            graphs.append(g)
        for c in (a, b):
            c.out.fill_(5.0)
            c.lse.fill_(7.0)
        for _ in range(2):
            for g in graphs:
                g.replay()
    torch.cuda.synchronize()
    assert a.pkv.pkv_get_device_error() == 0
    a.check()
    b.check()
    # new lengths in the captured tensors
    a.starts, a.news = [4000, 105], [9, 4]
    a.cu = np.cumsum([0, 9, 4]).astype(np.int32)
    a.cu_dev.copy_(torch.from_numpy(a.cu))
    a.start_dev.copy_(torch.tensor(a.starts, dtype=torch.int32))
    graphs[0].replay()
    assert a.pkv.pkv_get_device_error() == 0
    a.check()


def test_two_streams_at_once():
    a = Case([9000, 100], [4, 9], 8, 2, 128, "bf16", "fp4")
    b = Case([700, 3000, 9], [200, 1, 9], 4, 1, 128, "f16", "same")
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for c, st in zip((a, b), streams):
            c.call(stream=st)
    torch.cuda.synchronize()
    assert a.pkv.pkv_get_device_error() == 0
    a.check()
    b.check()


def test_host_memory_is_refused():
    import paged_kv_cache_160_gb300 as pkv
    c = Case([30], [2], 4, 2, 128, "bf16", "same")
    host = c.cache.k_cache.cpu().pin_memory()
    import ctypes
    args = (c.out.data_ptr(), 0, c.q_dev.data_ptr(), 1, c.cu_dev.data_ptr(), c.start_dev.data_ptr(), 1, 2, 4, host.data_ptr(),
            c.cache.v_cache.data_ptr(), ctypes.byref(c.cache.desc), c.cache.dev_tables.data_ptr(), 2, 0.1, c.ws.data_ptr(),
            c.ws.numel(), None)
    assert pkv.lib.pkv_paged_chunk_attention(*args) == 1
    torch.cuda.synchronize()
    assert (c.out == 5.0).all()


def test_one_row_agrees_with_the_decode():
    import paged_kv_cache_160_gb300 as pkv
    for kind in KINDS:
        c = _run([0, 77, 400], [1, 1, 1], 8, 2, 128, "bf16", kind)
        out, lens = torch.empty_like(c.q_dev), torch.tensor([1, 78, 401], dtype=torch.int32, device="cuda")
        ws = torch.empty(pkv.pkv_decode_workspace_bytes(3, 8, 2, 128, 16, 401, 0), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        pkv.pkv_paged_decode(out, c.q_dev, c.cache.k_cache, c.cache.v_cache, c.cache.desc, c.cache.dev_tables,
                             lens, 401, c.scale, 0, ws)
        assert (out.float() - c.out.float()).abs().max() <= 2.0 ** -5


@pytest.mark.parametrize("kind", ["fp4", "same"])
def test_blocks_past_4_gib(kind):
    """The last blocks of a pool of more than 2^32 bytes."""
    import paged_kv_cache_160_gb300 as pkv
    c = Case([300], [3], 2, 1, 128, "f16", kind)
    cc = c.cache
    big = (1 << 32) // (cc.k_cache[0].numel() * cc.k_cache.element_size()) + 40
    pools = []
    for x in (cc.k_cache, cc.v_cache):
        p = torch.zeros((big,) + tuple(x.shape[1:]), dtype=x.dtype, device="cuda")
        p[big - cc.num_blocks:] = x
        pools.append(p)
    cc.k_cache, cc.v_cache = pools
    cc.desc = (pkv.cache_desc_fp4 if kind == "fp4" else pkv.cache_desc)(pools[0], *cc.dev_scales)
    cc.dev_tables += big - cc.num_blocks
    c.call()
    assert pkv.pkv_get_device_error() == 0
    c.check()


def test_65535_chunks():
    """As many chunks as a call takes, of zero to two rows over the same few blocks."""
    import paged_kv_cache_160_gb300 as pkv
    n = 65535
    c = Case([40, 7], [1, 1], 2, 1, 64, "bf16", "fp4")
    cc = c.cache
    starts = np.arange(n) % 46
    news = (np.arange(n) * 7 % 13 % 3).astype(int)
    cu = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    total = int(cu[-1])
    g = torch.Generator().manual_seed(3)
    q = torch.randn((total, 2, 64), generator=g).to(torch.bfloat16)
    tables = torch.from_numpy(np.ascontiguousarray(np.broadcast_to(cc.tables[0], (n, cc.tables.shape[1])))).cuda()
    out, lse = torch.full_like(q, 5.0, device="cuda"), torch.empty((total, 2), device="cuda")
    ws = torch.empty(pkv.pkv_chunk_workspace_bytes(total, 2, 1, 64), dtype=torch.uint8, device="cuda")
    dev = [torch.from_numpy(a).cuda() for a in (cu, starts.astype(np.int32))]
    pkv.pkv_paged_chunk_attention(out, q.cuda(), *dev, cc.k_cache, cc.v_cache, cc.desc, tables, 0.125, ws, lse=lse)
    w = torch.full((n, 1, 48), 3.0, device="cuda")
    pkv.pkv_attention_weights(w, None, 1.0, q.cuda(), lse, *dev, cc.k_cache, cc.desc, tables, 0.125)
    assert pkv.pkv_get_device_error() == 0
    j = np.arange(48)
    k, v = (x[cc.tables[0, j // 16], :, j % 16] for x in (cc.k, cc.v))
    sums = w.sum(-1)[:, 0].cpu().numpy()
    for i in list(range(0, n, 4001)) + [n - 1]:
        a, m, s = cu[i], news[i], int(starts[i])
        if m == 0:
            assert (w[i] == 3.0).all()
            continue
        ref, ref_lse, size = evict.chunk_attention(q[a:a + m].double().numpy(), k[:s + m], v[:s + m], s, 0.125)
        err = np.abs(out[a:a + m].double().cpu().numpy() - ref)
        assert (err <= 2.0 ** -10 * size + 2.0 ** -8 * np.abs(ref) + 2.0 ** -25).all()
        assert abs(sums[i] - 2 * m - 3.0 * (48 - s - m)) <= 2.0 ** -9 * m
    assert torch.isfinite(out.float()).all()


def test_nothing_to_do():
    import paged_kv_cache_160_gb300 as pkv
    c = Case([5, 9], [0, 0], 4, 2, 64, "bf16", "fp4", pad=4)
    c.call()
    assert pkv.pkv_get_device_error() == 0 and (c.out == 5.0).all() and (c.lse == 7.0).all()
