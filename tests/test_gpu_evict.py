"""GPU parity of pkv_attention_weights, pkv_evict_select and pkv_evict_compact, and of the four calls in a row.

Weights: each term exp(scale q . k - lse) has a score that is an fp32 sum of at most 128 exact products (an error
below 2^-12 here, as in the attention's tests, bf16 rows taken as fp16 included), an argument rounded to fp32 (2^-18 for
arguments below 64) and exp2's own 2^-22; the sums of positive terms are fp32.  So |err| <= 2^-11 w + 2^-22 |decay in| +
2^-30.  Select and compact are exact.
"""
import numpy as np
import pytest
import torch

from oracle import evict
from tests.paged import DT, Paged
from tests.test_gpu_chunk import KINDS, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


# ---------------------------------------------------------------------------------------
# weights
# ---------------------------------------------------------------------------------------

class Weights(Case):
    def __init__(self, *a, rows=None, num_rows=None, max_len=None, prior=True, decay=1.0, **k):
        super().__init__(*a, **k)
        c = self.cache
        n = len(self.starts)
        self.rows = rows
        num_rows = num_rows or n
        max_len = max_len or max(c.lens)
        g = torch.Generator().manual_seed(n)
        self.prior = torch.rand((num_rows, c.heads, max_len), generator=g) if prior else None
        self.decay = decay
        self.w = torch.full((num_rows, c.heads, max_len), 3.0, device="cuda")
        q = self.q.double().numpy()
        lse = np.full(self.q.shape[:2], np.nan)
        for i, (s, m) in enumerate(zip(self.starts, self.news)):
            if m:
                lse[self.cu[i]:self.cu[i + 1]] = evict.chunk_attention(q[self.cu[i]:self.cu[i + 1]], c.rows("k", i, s + m),
                                                                      c.rows("v", i, s + m), s, self.scale)[1]
        self.lse = torch.from_numpy(lse).float().cuda()
        self.prior_dev = None if self.prior is None else self.prior.cuda()
        self.rows_dev = None if rows is None else torch.tensor(rows, dtype=torch.int32, device="cuda")

    def call_weights(self, in_place=False, stream=None):
        c = self.cache
        if in_place:
            self.w.copy_(self.prior_dev)
        self.pkv.pkv_attention_weights(self.w, self.w if in_place else self.prior_dev, self.decay, self.q_dev, self.lse,
                                       self.cu_dev, self.start_dev, c.k_cache, c.desc, c.dev_tables, self.scale,
                                       self.rows_dev, stream)

    def check_weights(self, in_place=False, only=None):
        c, q, lse = self.cache, self.q.double().numpy(), self.lse.double().cpu().numpy()
        got = self.w.double().cpu().numpy()
        ref = self.prior.double().numpy().copy() if in_place else np.full(got.shape, 3.0)
        size = np.zeros(got.shape)
        for i, (s, n) in enumerate(zip(self.starts, self.news)):
            row = i if self.rows is None else self.rows[i]
            if n == 0 or row < 0 or (only is not None and i not in only):
                continue
            a, b = self.cu[i], self.cu[i + 1]
            w = evict.chunk_weights(q[a:b], lse[a:b], c.rows("k", i, s + n), s, self.scale)
            size[row, :, :s + n] = 2.0 ** -11 * w + 2.0 ** -30
            if self.prior is not None:
                old = self.decay * self.prior[row, :, :s].double().numpy()
                w[:, :s] += old
                size[row, :, :s] += 2.0 ** -22 * np.abs(old)
            ref[row, :, :s + n] = w
        err = np.abs(got - ref)
        assert (err <= size).all(), (float(np.nanmax(err - size)), np.argwhere(~(err <= size))[:3])


def _weights(*a, in_place=False, **k):
    c = Weights(*a, **k)
    c.call_weights(in_place)
    assert c.pkv.pkv_get_device_error() == 0
    c.check_weights(in_place)
    return c


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("block", [16, 32])
def test_weights_ragged(kind, dtype, dim, block):
    _weights([0, 7, 127, 128, 129, 0, 300, 15], [1, 3, 1, 2, 0, 20, 5, 2], 6, 2, dim, dtype, kind, block=block, pad=3)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [1, 2, 16, 17, 64, 65, 128, 129, 257])
@pytest.mark.parametrize("start", [0, 130])
def test_weights_of_prompts(kind, n, start):
    _weights([start], [n], 2, 1, 128, "bf16", kind, max_len=start + n + 9)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 1), (28, 4), (40, 1), (150, 1)])
@pytest.mark.parametrize("n", [1, 5])
def test_weights_of_heads(hq, hkv, n):
    _weights([300, 31], [n, 2], hq, hkv, 128, "f16", "fp4", decay=0.75)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hq,hkv,n", [(28, 4, 60), (5, 1, 100), (3, 1, 200), (130, 1, 7), (96, 1, 4)])
def test_weights_of_many_blocks(kind, dtype, hq, hkv, n):
    """More than two blocks of rows, of sizes that no power of two divides."""
    _weights([200, 0], [n, 3], hq, hkv, 64, dtype, kind)


@pytest.mark.parametrize("kind", KINDS)
def test_weights_of_many_items_for_every_sm(kind):
    """Items of one, two, three and four key tiles, one to five blocks of rows, many for each SM."""
    c = Weights([5 + 37 * (i % 13) for i in range(120)], [1 + (i * 7) % 90 for i in range(120)], 8, 2, 64, "bf16", kind)
    c.call_weights()
    assert c.pkv.pkv_get_device_error() == 0
    first = c.w.clone()
    for _ in range(4):
        c.w.fill_(3.0)
        c.call_weights()
        assert c.pkv.pkv_get_device_error() == 0 and torch.equal(first, c.w)
    c.check_weights()


@pytest.mark.parametrize("kind", KINDS)
def test_weights_of_long_sequences(kind):
    _weights([9000, 40], [3, 200], 4, 2, 128, "bf16", kind, decay=0.5)


@pytest.mark.parametrize("kind,dtype", [("same", "bf16"), ("fp4", "bf16"), ("e4m3", "f16")])
@pytest.mark.parametrize("keys,rows,chunks", [(896, 34, 1), (896, 34, 3), (640, 12, 3), (1100, 7, 2), (384, 17, 4)])
def test_weights_of_uneven_groups_and_many_blocks(kind, dtype, keys, rows, chunks):
    """One to three items for each SM, of seven key tiles (a group of four and one of three), five, nine or three, seen by
    four to 17 blocks of rows: what a group's idle warps have not read yet is not overwritten."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n, heads, dim = chunks * sms, 64, 64
    c = Case([keys - rows] * n, [rows] * n, heads, 1, dim, dtype, kind)
    c.call()
    cc = c.cache
    w = torch.full((n, 1, keys), 3.0, device="cuda")
    call = lambda: c.pkv.pkv_attention_weights(w, None, 1.0, c.q_dev, c.lse, c.cu_dev, c.start_dev, cc.k_cache, cc.desc,  # noqa: E731
                                               cc.dev_tables, c.scale)
    call()
    assert c.pkv.pkv_get_device_error() == 0
    first = w.clone()
    k = torch.from_numpy(cc.k).cuda()                          # float64
    q = c.q_dev.double().view(n, rows, heads, dim)
    lse = c.lse.double().view(n, rows, heads)
    j = torch.arange(keys)
    seen = j.cuda()[None] <= torch.arange(keys - rows, keys, device="cuda")[:, None]
    for i in range(n):
        blocks = torch.from_numpy(cc.tables[i]).long()[j // 16].cuda()
        s = c.scale * torch.einsum("rhd,jd->rhj", q[i], k[blocks, 0, (j % 16).cuda()]) - lse[i][:, :, None]
        ref = (s.exp() * seen[:, None]).sum((0, 1))
        err = (first[i, 0].double() - ref).abs()
        assert (err <= 2.0 ** -11 * ref + 2.0 ** -30).all(), (i, float((err / ref).max()))
    for _ in range(10):
        w.fill_(3.0)
        call()
        assert c.pkv.pkv_get_device_error() == 0 and torch.equal(first, w)


def test_weights_of_many_sequences():
    rng = np.random.default_rng(6)
    _weights([int(x) for x in rng.integers(0, 300, 400)], [int(x) for x in rng.integers(0, 3, 400)], 3, 1, 64, "bf16", "fp4")


@pytest.mark.parametrize("in_place", [False, True])
def test_weights_rows(in_place):
    """Rows in another order; chunks without a row and chunks without query rows change nothing."""
    _weights([20, 30, 200, 10], [2, 1, 3, 0], 4, 2, 128, "bf16", "fp4", rows=[5, -1, 0, 2], num_rows=6, max_len=250,
             in_place=in_place, decay=0.9)


def test_weights_without_earlier_ones():
    _weights([20, 300], [2, 1], 4, 2, 128, "bf16", "fp4", prior=False)


def test_weights_ignore_what_is_stored_for_new_tokens():
    """What a row holds from the chunk's first position on is not read."""
    c = Weights([20, 300], [2, 3], 4, 2, 128, "bf16", "same")
    c.prior_dev[0, :, 20:] = float("nan")
    c.prior_dev[1, :, 300:] = float("inf")
    c.call_weights()
    c.check_weights()


@pytest.mark.parametrize("kind", ["fp4", "e4m3"])
def test_weights_of_any_scale(kind):
    c = Weights([150], [9], 8, 4, 64, "bf16", kind)
    c.cache.scales = [np.array([-1.2, 0.5, 0.0, 2.0 ** -30], np.float32), c.cache.scales[1]]
    c.cache.upload()
    c.q = (c.q.float() * torch.tensor([1.0, 2.0 ** -40, 0.25] * 3)[:, None, None]).to(torch.bfloat16)
    c.q_dev = c.q.cuda()
    lse = evict.chunk_attention(c.q.double().numpy(), c.cache.rows("k", 0, 159), c.cache.rows("v", 0, 159), 150, c.scale)[1]
    c.lse = torch.from_numpy(lse).float().cuda()
    c.call_weights()
    c.check_weights()


@pytest.mark.parametrize("kind", KINDS)
def test_weights_of_stale_and_later_rows(kind):
    """NaN in stale rows of blocks and in keys that only some rows see."""
    c = Weights([70], [6], 4, 2, 128, "bf16", kind, seed=3)
    cc = c.cache
    stored, bad = cc.stored[0], 74
    for p in list(range(76, 80)) + [bad]:
        b, r = cc.tables[0, p // 16], p % 16
        if cc.kv == "fp4":
            stored[b, :, 0, 8 * 128 + 8 * r + 3] = 0x7F
        else:
            stored[b, :, r, 5] = 0x7F if cc.kv == "e4m3" else 0x7FC0
    cc.upload()
    c.call_weights()
    got = c.w.cpu()
    assert torch.isnan(got[0, :, bad]).all()
    got[0, :, bad] = 0
    assert torch.isfinite(got).all()


def test_weights_errors():
    import paged_kv_cache_160_gb300 as pkv
    c = Weights([20, 300, 40], [2, 3, 1], 4, 2, 128, "bf16", "fp4", rows=[0, 1, 2])
    c.rows_dev[1] = 3
    c.call_weights()
    assert pkv.pkv_get_device_error() == pkv.DEVERR["slot"]
    c.check_weights(only=[0, 2])
    c = Weights([20, 300, 40], [2, 3, 1], 4, 2, 128, "bf16", "fp4", max_len=302)
    c.call_weights()
    assert pkv.pkv_get_device_error() == pkv.DEVERR["context_len"]
    c.check_weights(only=[0, 2])
    c = Weights([20, 300, 40], [2, 3, 1], 4, 2, 128, "bf16", "fp4")
    c.start_dev[1] = -5
    c.call_weights()
    assert pkv.pkv_get_device_error() == pkv.DEVERR["chunk"]
    c.check_weights(only=[0, 2])
    c = Weights([20, 300, 40], [2, 3, 1], 4, 2, 128, "bf16", "fp4")
    c.cache.dev_tables[1, 3] = 1 << 28
    c.call_weights()
    assert pkv.pkv_get_device_error() == pkv.DEVERR["block_id"]
    cc = c.cache
    cc.k = cc.k.copy()
    cc.k[cc.tables[1, 3]] = 0
    c.check_weights()


@pytest.mark.parametrize("kind,dtype", [("same", "bf16"), ("same", "f16"), ("e4m3", "f16"), ("fp4", "f16")])
def test_weights_of_log_sum_exps_that_come_late(kind, dtype):
    """Queries and keys are in L2, the rows' log-sum-exps are not: no product may run ahead of them.  (The forms whose
    queries are copied unchanged; the call before leaves other rows' terms in every place.)"""
    c = Weights([700 + 9 * i for i in range(40)], [1 + i % 5 for i in range(40)], 8, 2, 128, dtype, kind)
    cold = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")        # more than L2 holds
    right, wrong = c.lse.clone(), torch.full_like(c.lse, -40.0)
    for _ in range(20):
        c.lse.copy_(wrong)
        c.call_weights()
        c.lse.copy_(right)
        cold.fill_(_)
        c.q_dev.view(torch.uint8).sum()
        c.cache.k_cache.view(torch.uint8).sum()
        c.w.fill_(3.0)
        c.call_weights()
        assert c.pkv.pkv_get_device_error() == 0
        if _ == 0:
            c.check_weights()
            first = c.w.clone()
        assert torch.equal(first, c.w)


def test_weights_in_a_graph_and_twice_the_same():
    c = Weights([900, 30], [3, 2], 8, 2, 128, "bf16", "fp4")
    c.call_weights()
    first = c.w.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            c.call_weights()
        c.w.fill_(3.0)
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, c.w)
    c.check_weights()


# ---------------------------------------------------------------------------------------
# select
# ---------------------------------------------------------------------------------------

def _select(lens, keep, first, recent, heads=2, rows=None, num_rows=None, max_len=None, max_keep=None, make=None, seed=0):
    import paged_kv_cache_160_gb300 as pkv
    n = len(lens)
    max_len, max_keep = max_len or max(max(lens), 1), max_keep or max(max(keep), 1)
    g = torch.Generator().manual_seed(seed + sum(lens))
    w = torch.exp(2 * torch.randn((num_rows or n, heads, max_len), generator=g)) if make is None else make(
        (num_rows or n, heads, max_len), g)
    i32 = dict(dtype=torch.int32, device="cuda")
    kept = torch.full((n, heads, max_keep), 77, **i32)
    pkv.pkv_evict_select(kept, w.cuda(), torch.tensor(lens, **i32), torch.tensor(keep, **i32), first, recent,
                         None if rows is None else torch.tensor(rows, **i32))
    assert pkv.pkv_get_device_error() == 0
    got, wn = kept.cpu().numpy(), w.numpy()
    for i in range(n):
        row = i if rows is None else rows[i]
        for h in range(heads):
            ref = [] if row < 0 else evict.select(wn[row, h], lens[i], keep[i], first, recent)
            assert got[i, h].tolist() == ref + [-1] * (max_keep - len(ref)), (i, h)


@pytest.mark.parametrize("first,recent", [(0, 0), (4, 0), (0, 16), (4, 16), (100, 100), (3, 1000)])
def test_select_ragged(first, recent):
    _select([0, 1, 2, 5, 31, 33, 100, 300, 1000, 1023, 1024, 1025, 2500], [5, 1, 0, 7, 31, 32, 50, 299, 10, 700, 1, 512, 777],
            first, recent, max_len=2601, max_keep=780)


@pytest.mark.parametrize("n,keep", [(5000, 1), (5000, 4999), (20000, 2500), (70000, 9000), (140001, 33333)])
def test_select_long(n, keep):
    _select([n, n // 2], [keep, keep // 3 + 1], 4, min(keep, 128), heads=1)


def test_select_ties():
    """Few distinct weights, zeros of both signs, infinities, NaN, subnormals, negatives."""
    def make(shape, g):
        v = torch.tensor([0.0, -0.0, 1.0, 1.0, 2.0, float("inf"), -float("inf"), float("nan"), 1e-40, -1e-40, -3.0, 3e38])
        return v[torch.randint(0, len(v), shape, generator=g)]
    for keep in (1, 60, 300, 500, 700, 1100, 1200):
        _select([1200, 700], [keep, min(keep, 650)], 2, 5, make=make, seed=keep)
    _select([3000], [1500], 0, 0, make=lambda s, g: torch.zeros(s))
    _select([3000], [1500], 0, 0, make=lambda s, g: torch.full(s, float("nan")))


def test_select_neighbouring_weights():
    """Weights that differ in their last bits only."""
    def make(shape, g):
        return torch.randint(0x3F800000, 0x3F800000 + 600, shape, generator=g, dtype=torch.int32).view(torch.float32)
    _select([4000, 1500], [1000, 700], 0, 3, make=make)


def test_select_rows():
    _select([50, 60, 70], [20, 20, 20], 1, 2, rows=[4, -1, 0], num_rows=5, max_len=80)


def test_select_errors():
    import paged_kv_cache_160_gb300 as pkv
    i32 = dict(dtype=torch.int32, device="cuda")
    w = torch.rand((3, 2, 100)).cuda()
    for lens, keep, rows, bit in (([50, 101, 60], [9, 9, 9], None, "context_len"), ([50, -1, 60], [9, 9, 9], None, "context_len"),
                                  ([50, 60, 60], [9, 11, 9], None, "context_len"), ([50, 60, 60], [9, -2, 9], None, "context_len"),
                                  ([50, 60, 60], [9, 9, 9], [0, 3, 2], "slot")):
        kept = torch.full((3, 2, 10), 77, **i32)
        pkv.pkv_evict_select(kept, w, torch.tensor(lens, **i32), torch.tensor(keep, **i32), 1, 1,
                             None if rows is None else torch.tensor(rows, **i32))
        assert pkv.pkv_get_device_error() == pkv.DEVERR[bit]
        assert (kept[1] == -1).all()
        for i in (0, 2):
            for h in range(2):
                assert kept[i, h].tolist() == evict.select(w[i, h].cpu().numpy(), lens[i], 9, 1, 1) + [-1]


# ---------------------------------------------------------------------------------------
# compact
# ---------------------------------------------------------------------------------------

def _kept(rng, lens, keep, heads, max_keep):
    kept = np.full((len(lens), heads, max_keep), -1, np.int32)
    for i, (n, m) in enumerate(zip(lens, keep)):
        for h in range(heads):
            kept[i, h, :m] = np.sort(rng.choice(n, m, replace=False))
    return kept


def _rows_of(c, stored):
    """The stored bytes row by row: [blocks, heads, block, bytes]."""
    if c.kv != "fp4":
        return stored
    nb, h, tiles, _ = stored.shape
    codes = stored[..., : 8 * c.dim].reshape(nb, h, tiles * 16, c.dim // 2)
    return np.concatenate([codes, stored[..., 8 * c.dim:].reshape(nb, h, tiles * 16, c.dim // 16)], -1)


def _compact(lens, keep, kv, heads=2, dim=128, block=16, fresh=None, weights=True, seed=0, max_keep=None, kept=None,
             dst_rows=None):
    """fresh: (sequence, block) pairs whose destination is a block that nothing reads."""
    import paged_kv_cache_160_gb300 as pkv
    rng = np.random.default_rng(seed + sum(lens))
    c = Paged(lens, kv, heads, dim, block, seed=seed, extra=3 + len(fresh or []))
    max_keep = max_keep or max(max(keep), 1)
    kept = _kept(rng, lens, keep, heads, max_keep) if kept is None else kept
    dst = c.tables.copy()
    unused = [b for b in range(c.num_blocks) if b not in set(c.tables.flatten().tolist())]
    for (i, b), u in zip(fresh or [], unused):
        dst[i, b] = u
    n = len(lens)
    w = rng.random((2 * n, heads, max(lens) + 3)).astype(np.float32)
    dev = torch.from_numpy(w).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    rows = list(range(n))[::-1]
    pkv.pkv_evict_compact(c.k_cache, c.v_cache, c.desc, torch.from_numpy(kept).cuda(), torch.tensor(keep, **i32), c.dev_tables,
                          torch.from_numpy(dst).cuda() if fresh else None, dev if weights else None,
                          torch.tensor(rows, **i32), None if dst_rows is None else torch.tensor(dst_rows, **i32))
    assert pkv.pkv_get_device_error() == 0
    for pool, stored in zip((c.k_cache, c.v_cache), c.stored):
        got = pool.view(torch.int16 if kv in DT else torch.uint8).cpu().numpy()
        ref = evict.compact(_rows_of(c, stored), kept, keep, c.tables, dst, block)
        assert np.array_equal(_rows_of(c, got), ref)
    ref = w.copy()
    if weights:
        for i in range(n):
            for h in range(heads):
                m = int((kept[i, h] >= 0).sum())
                ref[rows[i] if dst_rows is None else dst_rows[i], h, :m] = w[rows[i], h, kept[i, h, :m]]
    assert np.array_equal(dev.cpu().numpy(), ref)


@pytest.mark.parametrize("kv", ["fp4", "e4m3", "bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("block", [16, 32])
def test_compact_ragged(kv, dim, block):
    _compact([1, 5, 16, 33, 100, 300, 700, 64], [1, 0, 3, 32, 50, 299, 257, 64], kv, dim=dim, block=block)


@pytest.mark.parametrize("kv", ["fp4", "e4m3", "bf16"])
@pytest.mark.parametrize("n,keep", [(3000, 2999), (5000, 1300), (9000, 8192), (30000, 25000)])
def test_compact_long(kv, n, keep):
    _compact([n, 40], [keep, 20], kv, heads=1, dim=64)


@pytest.mark.parametrize("kv", ["fp4", "bf16"])
def test_compact_worst_orders(kv):
    """Everything moves by one row; everything stays; the last rows only."""
    n, m = 3000, 2900
    for first in ([1 + j for j in range(m)], list(range(m)), [n - m + j for j in range(m)],
                  list(range(1500)) + [n - m + j for j in range(1500, m)]):
        _compact([n], [m], kv, heads=2, dim=64, kept=np.array([[first, first[::1]]], np.int32))


@pytest.mark.parametrize("kv", ["fp4", "e4m3", "bf16"])
def test_compact_into_other_blocks(kv):
    _compact([100, 70, 300], [60, 70, 100], kv, fresh=[(0, 0), (0, 2), (1, 1), (2, 0), (2, 5)], dst_rows=[4, 1, 5])


@pytest.mark.parametrize("dim", [16, 32, 80, 96, 256])
def test_compact_head_dims(dim):
    for kv in ("fp4", "e4m3", "bf16"):
        _compact([100, 70], [60, 33], kv, heads=3, dim=dim, block=32)


def test_compact_without_weights_and_short_lists():
    _compact([100, 70], [60, 33], "fp4", weights=False)
    rng = np.random.default_rng(0)
    kept = _kept(rng, [100, 70], [50, 20], 2, 64)              # -1 behind the 50 and 20
    _compact([100, 70], [60, 33], "fp4", kept=kept, max_keep=64)


def test_compact_errors():
    import paged_kv_cache_160_gb300 as pkv
    i32 = dict(dtype=torch.int32, device="cuda")
    for what, bit in (("ascend", "chunk"), ("past", "chunk"), ("keep", "context_len"), ("block", "block_id"),
                      ("row", "slot"), ("length", "context_len"), ("early", "chunk")):
        c = Paged([100, 70], "bf16", 2, 64)
        kept = _kept(np.random.default_rng(1), [100, 70], [40, 30], 2, 40)
        w = torch.rand((2, 2, 100)).cuda()
        before, wb = c.k_cache.clone(), w.clone()
        keep, tables, rows = torch.tensor([40, 30], **i32), c.dev_tables, torch.tensor([0, 1], **i32)
        if what == "ascend":
            kept[0, 0, 20] = kept[0, 0, 19]
        elif what == "past":
            kept[0, 0, 39] = 112
            w = torch.rand((2, 2, 200)).cuda()
            wb = w.clone()
        elif what == "early":
            kept[0, 0, 39] = 30
        elif what == "keep":
            keep[0] = 41
        elif what == "block":
            tables[0, 0] = c.num_blocks
        elif what == "row":
            rows[0] = 2
        else:
            w = torch.rand((2, 2, 69)).cuda()
            wb = w.clone()
        pkv.pkv_evict_compact(c.k_cache, c.v_cache, c.desc, torch.from_numpy(kept).cuda(), keep, tables, None, w, rows)
        assert pkv.pkv_get_device_error() == pkv.DEVERR[bit], what
        # the other sequence and, of a bad entry's head, the other entries move
        ref = evict.compact(c.stored[0], kept[1:], [30], c.tables[1:], c.tables[1:], 16)
        mine = c.tables[1]
        got = c.k_cache.view(torch.int16).cpu().numpy()
        assert np.array_equal(got[mine[mine >= 0]], ref[mine[mine >= 0]])
        if what == "keep":
            own = c.tables[0][c.tables[0] >= 0].tolist()
            assert torch.equal(c.k_cache[own], before[own]) and torch.equal(w[0], wb[0])
        if what == "row":
            assert torch.equal(w[0], wb[0])


@pytest.mark.parametrize("kv", ["fp4", "bf16"])
def test_blocks_past_4_gib(kv):
    """Weights and moves in the last blocks of a pool of more than 2^32 bytes."""
    import paged_kv_cache_160_gb300 as pkv
    c = Weights([300], [3], 2, 1, 128, "bf16", kv)
    cc = c.cache
    big = (1 << 32) // (cc.k_cache[0].numel() * cc.k_cache.element_size()) + 40
    pools = []
    for x in (cc.k_cache, cc.v_cache):
        p = torch.zeros((big,) + tuple(x.shape[1:]), dtype=x.dtype, device="cuda")
        p[big - cc.num_blocks:] = x
        pools.append(p)
    cc.k_cache, cc.v_cache = pools
    cc.desc = (pkv.cache_desc_fp4 if kv == "fp4" else pkv.cache_desc)(pools[0], *cc.dev_scales)
    cc.dev_tables += big - cc.num_blocks
    c.call_weights()
    assert pkv.pkv_get_device_error() == 0
    c.check_weights()
    kept = _kept(np.random.default_rng(2), [303], [200], 1, 200)
    pkv.pkv_evict_compact(*pools, cc.desc, torch.from_numpy(kept).cuda(), torch.tensor([200], dtype=torch.int32, device="cuda"),
                          cc.dev_tables)
    assert pkv.pkv_get_device_error() == 0
    for pool, stored in zip(pools, cc.stored):
        got = pool[big - cc.num_blocks:].view(torch.int16 if kv in DT else torch.uint8).cpu().numpy()
        assert np.array_equal(_rows_of(cc, got), evict.compact(_rows_of(cc, stored), kept, [200], cc.tables, cc.tables, 16))


def test_select_and_compact_in_a_graph():
    """The captured calls, with other weights and lengths in the captured tensors."""
    import paged_kv_cache_160_gb300 as pkv
    i32 = dict(dtype=torch.int32, device="cuda")
    c = Paged([3000, 500], "e4m3", 2, 64, max_blocks=200)
    w = torch.rand((2, 2, 3200)).cuda()
    kept = torch.zeros((2, 2, 900), **i32)
    lens, keep = torch.tensor([3000, 500], **i32), torch.tensor([900, 100], **i32)

    def call():
        pkv.pkv_evict_select(kept, w, lens, keep, 3, 10)
        pkv.pkv_evict_compact(c.k_cache, c.v_cache, c.desc, kept, keep, c.dev_tables, None, w)
    captured = c.k_cache, c.v_cache, c.desc, c.dev_tables, c.dev_scales     # kept for as long as the graph
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            call()
    torch.cuda.synchronize()
    for n, m in (([3000, 500], [900, 100]), ([2900, 480], [77, 300])):
        c.upload()
        # the graph works on the tensors that it captured
        pools = c.k_cache, c.v_cache
        w.copy_(torch.rand((2, 2, 3200)))
        lens.copy_(torch.tensor(n))
        keep.copy_(torch.tensor(m))
        before = w.cpu().numpy().copy()
        call()
        got = [p.clone() for p in pools]
        after, list_ = w.clone(), kept.cpu().numpy()
        for i in range(2):
            for h in range(2):
                ref = evict.select(before[i, h], n[i], m[i], 3, 10)
                assert list_[i, h, :m[i]].tolist() == ref
                assert np.array_equal(after[i, h, :m[i]].cpu().numpy(), before[i, h, ref])
        assert np.array_equal(got[0].cpu().numpy(), evict.compact(c.stored[0], list_, m, c.tables, c.tables, 16))
        # the same by the graph
        w.copy_(torch.from_numpy(before))
        kept.zero_()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(kept.cpu().numpy(), list_) and torch.equal(w, after)
    assert pkv.pkv_get_device_error() == 0
    assert captured[0].data_ptr() != c.k_cache.data_ptr()


@pytest.mark.parametrize("kv", ["fp4", "e4m3", "bf16"])
@pytest.mark.parametrize("fresh", [False, True])
def test_a_captured_compaction_moves_the_rows(kv, fresh):
    """Select and compact in a graph, replayed over other rows, weights and lengths: K, V and weights against the oracle."""
    import paged_kv_cache_160_gb300 as pkv
    i32 = dict(dtype=torch.int32, device="cuda")
    c = Paged([3000, 500], kv, 2, 64, max_blocks=200, extra=70)
    dst = c.tables.copy()
    if fresh:                                                  # blocks of their own for the first sequence
        unused = [b for b in range(c.num_blocks) if b not in set(c.tables.flatten().tolist())]
        dst[0, :60] = unused[:60]
    dst_dev = torch.from_numpy(dst).cuda()
    w = torch.rand((2, 2, 3200)).cuda()
    kept = torch.zeros((2, 2, 900), **i32)
    lens, keep = torch.tensor([3000, 500], **i32), torch.tensor([900, 100], **i32)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        pkv.pkv_evict_select(kept, w, lens, keep, 3, 10)
        pkv.pkv_evict_compact(c.k_cache, c.v_cache, c.desc, kept, keep, c.dev_tables, dst_dev, w)
    torch.cuda.synchronize()
    rng = np.random.default_rng(8)
    for n, m in (([3000, 500], [900, 100]), ([2900, 480], [77, 300]), ([31, 1], [0, 1]), ([3000, 500], [900, 499])):
        stored = [rng.permutation(s, axis=0) for s in c.stored]
        for pool, s in zip((c.k_cache, c.v_cache), stored):
            pool.view(torch.int16 if kv in DT else torch.uint8).copy_(torch.from_numpy(s))
        before = rng.random((2, 2, 3200)).astype(np.float32)
        w.copy_(torch.from_numpy(before))
        lens.copy_(torch.tensor(n))
        keep.copy_(torch.tensor(m))
        kept.fill_(77)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.synchronize()
        assert pkv.pkv_get_device_error() == 0
        list_, after = kept.cpu().numpy(), before.copy()
        for i in range(2):
            for h in range(2):
                ref = evict.select(before[i, h], n[i], m[i], 3, 10)
                assert list_[i, h].tolist() == ref + [-1] * (900 - len(ref))
                after[i, h, :m[i]] = before[i, h, ref]
        assert np.array_equal(w.cpu().numpy(), after)
        for pool, s in zip((c.k_cache, c.v_cache), stored):
            got = pool.view(torch.int16 if kv in DT else torch.uint8).cpu().numpy()
            assert np.array_equal(_rows_of(c, got), evict.compact(_rows_of(c, s), list_, m, c.tables, dst, 16))


# ---------------------------------------------------------------------------------------
# the calls in a row
# ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("kind", KINDS)
def test_a_cache_kept_short(kind):
    """Prompts, eviction into new tables, a step over what is left: each call works on what the last one gave."""
    import paged_kv_cache_160_gb300 as pkv
    hq, hkv, dim, dtype = 4, 2, 128, "bf16"
    lens, keep = [210, 77, 130], [64, 77, 50]
    bm = pkv.BlockManager(60, 16)
    for i, n in enumerate(lens):
        bm.allocate(i, n)
    bm.fork(0, 9)                                              # its blocks are shared
    tables, _ = bm.export([0, 1, 2], 14)
    c = Case([0, 0, 0], lens, hq, hkv, dim, dtype, kind)
    cc = c.cache
    cc.tables = np.array(tables, np.int32)
    pools = Paged([16 * 60], cc.kv, hkv, dim, seed=11, extra=0)
    cc.stored, cc.num_blocks, cc.scales = pools.stored, 60, pools.scales
    cc.upload()
    c.call()
    assert pkv.pkv_get_device_error() == 0
    c.check()
    i32 = dict(dtype=torch.int32, device="cuda")
    w = torch.full((5, hkv, 256), float("nan"), device="cuda")
    rows = torch.tensor([3, 0, 4], **i32)
    pkv.pkv_attention_weights(w, None, 1.0, c.q_dev, c.lse, c.cu_dev, c.start_dev, cc.k_cache, cc.desc, cc.dev_tables,
                              c.scale, rows)
    q, ref = c.q.double().numpy(), []
    for i, n in enumerate(lens):
        a = c.cu[i]
        ref.append(evict.chunk_weights(q[a:a + n], c.lse[a:a + n].double().cpu().numpy(), cc.rows("k", i, n), 0, c.scale))
        assert np.abs(w[rows[i], :, :n].double().cpu().numpy() - ref[i]).max() <= 2.0 ** -11 * ref[i].max() + 2.0 ** -30
        assert abs(ref[i].sum() - n * hq) < 1e-2 * n           # every row hands out a weight of one
    kept = torch.empty((3, hkv, 80), **i32)
    pkv.pkv_evict_select(kept, w, torch.tensor(lens, **i32), torch.tensor(keep, **i32), 2, 8, rows)
    src, src_lens, dst = bm.evict([0, 1, 2], keep, 14, 6)
    assert src_lens == lens and src == tables
    assert dst[1][:5] == src[1][:5] and not set(dst[0]) & set(src[0]) - {-1}
    shared = cc.k_cache.clone()
    before = {x: [cc.rows(x, i, n) for i, n in enumerate(lens)] for x in "kv"}
    pkv.pkv_evict_compact(cc.k_cache, cc.v_cache, cc.desc, kept, torch.tensor(keep, **i32), torch.tensor(src, **i32),
                          torch.tensor(dst, **i32), w, rows)
    assert pkv.pkv_get_device_error() == 0
    forked = [b for b in src[0] if b >= 0]
    assert torch.equal(cc.k_cache.view(torch.uint8)[forked], shared.view(torch.uint8)[forked])
    kn = kept.cpu().numpy()
    # one more token each
    slots, cow, tab, now = bm.step_decode([0, 1, 2], 6)
    assert not cow and now == [n + 1 for n in keep]
    new = torch.randn((2, 3, hkv, dim)).to(DT[dtype]).cuda()
    pkv.pkv_kv_write(new[0].contiguous(), new[1].contiguous(), torch.tensor(slots, device="cuda"), cc.k_cache, cc.v_cache, cc.desc)
    cc.stored = [t.view(torch.int16 if cc.kv in DT else torch.uint8).cpu().numpy() for t in (cc.k_cache, cc.v_cache)]
    cc.tables = np.array(tab, np.int32)
    cc.upload()
    for i, n in enumerate(keep):
        for x in "kv":
            got = cc.rows(x, i, n)
            for h in range(hkv):
                assert np.array_equal(got[:, h], before[x][i][kn[i, h, :n], h])
    d = Case([0] * 3, [1] * 3, hq, hkv, dim, dtype, kind, seed=5)
    d.starts, d.cache = list(keep), cc
    d.dev()
    d.call()
    pkv.pkv_attention_weights(w, w, 0.5, d.q_dev, d.lse, d.cu_dev, d.start_dev, cc.k_cache, cc.desc, cc.dev_tables, d.scale,
                              rows)
    assert pkv.pkv_get_device_error() == 0
    d.check()
    for i, n in enumerate(keep):
        got = w[rows[i], :, :n + 1].double().cpu().numpy()
        step = evict.chunk_weights(d.q[i:i + 1].double().numpy(), d.lse[i:i + 1].double().cpu().numpy(),
                                   cc.rows("k", i, n + 1), n, d.scale)
        for h in range(hkv):
            step[h, :n] += 0.5 * ref[i][h, kn[i, h, :n]]
        assert (np.abs(got - step) <= 2.0 ** -10 * step + 2.0 ** -30).all()
