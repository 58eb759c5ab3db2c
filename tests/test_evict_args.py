"""CPU tests of the chunk attention's and the eviction's argument checks, of pkv_bm_evict, and of their oracle on cases
worked out by hand.  Nothing here reaches a GPU."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import evict

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


def _desc(kv=3, heads=4, block=16, dim=128, scales=False):
    from paged_kv_cache_160_gb300._binding import CacheDesc
    s = 16 if scales or kv == 2 else None
    return CacheDesc(64, heads, block, dim, kv, s, s)


def _chunk(desc=None, out=16, lse=4, q=16, qd=1, cu=4, start=4, n=2, total=8, hq=8, k=16, v=16, tables=4, width=8, scale=0.1,
           ws=16, nbytes=1 << 40):
    import paged_kv_cache_160_gb300 as pkv
    return pkv.lib.pkv_paged_chunk_attention(out, lse, q, qd, cu, start, n, total, hq, k, v, ctypes.byref(desc or _desc()),
                                             tables, width, scale, ws, nbytes, None)


def _weights(desc=None, out=4, prior=4, decay=1.0, num_rows=4, max_len=100, rows=4, q=16, qd=1, lse=4, cu=4, start=4, n=2,
             total=8, hq=8, k=16, tables=4, width=8, scale=0.1):
    import paged_kv_cache_160_gb300 as pkv
    return pkv.lib.pkv_attention_weights(out, prior, decay, num_rows, max_len, rows, q, qd, lse, cu, start, n, total, hq, k,
                                         ctypes.byref(desc or _desc()), tables, width, scale, None)


@pytest.mark.parametrize("call", [_chunk, _weights])
def test_refusals_of_chunk_calls(call):
    nan, inf = float("nan"), float("inf")
    for bad in (dict(hq=6), dict(hq=0), dict(hq=-4), dict(n=-1), dict(total=-1), dict(width=-1), dict(qd=2), dict(qd=3),
                dict(scale=0.0), dict(scale=-1.0), dict(scale=nan), dict(scale=inf), dict(q=0), dict(q=8), dict(cu=0),
                dict(cu=2), dict(start=0), dict(start=6), dict(k=0), dict(k=8), dict(tables=0), dict(tables=2), dict(width=0),
                dict(lse=2), dict(out=0)):
        assert call(**bad) == INVALID, bad
    for bad in (_desc(dim=96), _desc(dim=256), _desc(block=48), _desc(kv=0), _desc(kv=1, block=8)):
        assert call(desc=bad) == UNSUPPORTED
    assert call(desc=_desc(kv=1), qd=0) == UNSUPPORTED
    assert call(total=1 << 28, hq=8) == UNSUPPORTED
    assert call(n=70000, total=1 << 20) == UNSUPPORTED
    # positions, rounded up to a key tile, and pieces of work in 32 bits
    assert call(width=(1 << 27) - 7) == UNSUPPORTED and call(width=(1 << 27) - 8) != UNSUPPORTED
    assert call(total=1 << 20, hq=1024, width=1 << 20) == UNSUPPORTED
    e4m3 = _desc(kv=2)
    e4m3.k_scale = None
    assert call(desc=e4m3) == INVALID
    assert call(n=0) == OK and call(total=0) == OK


@pytest.mark.parametrize("call", [_chunk, _weights])
def test_scales_whose_product_with_log2_e_has_no_fp32(call):
    """scale * 1.4427 has to stay finite: a score of zero times infinity would be NaN."""
    other = dict(desc=_desc(dim=96))                           # looked at later
    assert call(scale=2.5e38, **other) == INVALID and call(scale=2.0 ** 127 * 1.01, **other) == INVALID
    assert call(scale=2.0 ** 127, **other) == UNSUPPORTED and call(scale=1e-40, **other) == UNSUPPORTED


def test_refusals_of_the_chunk_attention():
    for bad in (dict(out=8), dict(v=0), dict(v=8)):
        assert _chunk(**bad) == INVALID, bad
    for bad in (dict(ws=0), dict(ws=8), dict(nbytes=16)):
        assert _chunk(**bad) == WORKSPACE, bad


def test_refusals_of_the_weights():
    nan, inf = float("nan"), float("inf")
    for bad in (dict(lse=0), dict(out=2), dict(prior=2), dict(rows=2), dict(decay=-0.5), dict(decay=nan), dict(decay=inf),
                dict(num_rows=0), dict(num_rows=-1), dict(max_len=0), dict(max_len=-3)):
        assert _weights(**bad) == INVALID, bad


def test_refusals_of_select_and_compact():
    import paged_kv_cache_160_gb300 as pkv
    names = ("kept", "max_keep", "weights", "num_rows", "max_len", "rows", "lens", "keep", "n", "heads", "first", "recent")
    good = dict(kept=4, max_keep=8, weights=4, num_rows=2, max_len=9, rows=4, lens=4, keep=4, n=2, heads=4, first=1, recent=1)
    call = lambda **k: pkv.lib.pkv_evict_select(*[dict(good, **k)[x] for x in names], None)  # noqa: E731
    for bad in (dict(kept=0), dict(kept=2), dict(weights=0), dict(weights=6), dict(rows=2), dict(lens=0), dict(lens=1),
                dict(keep=0), dict(keep=2), dict(max_keep=-1), dict(num_rows=0), dict(num_rows=-1), dict(max_len=0),
                dict(n=-1), dict(heads=0), dict(first=-1), dict(recent=-1)):
        assert call(**bad) == INVALID, bad
    assert call(n=1 << 20, heads=1 << 12) == UNSUPPORTED
    assert call(max_len=(1 << 30) + 1) == UNSUPPORTED and call(max_keep=(1 << 30) + 1) == UNSUPPORTED
    assert call(n=0) == OK and call(max_keep=0) == OK
    names = ("k", "v", "desc", "kept", "max_keep", "keep", "src", "sb", "dst", "db", "w", "num_rows", "max_len", "rows",
             "dst_rows", "n")
    good = dict(k=16, v=32, desc=_desc(), kept=4, max_keep=8, keep=4, src=4, sb=3, dst=4, db=3, w=4, num_rows=2, max_len=9,
                rows=4, dst_rows=4, n=2)

    def move(**k):
        a = dict(good, **k)
        a["desc"] = ctypes.byref(a["desc"])
        return pkv.lib.pkv_evict_compact(*[a[x] for x in names], None)
    for bad in (dict(k=0), dict(k=8), dict(v=0), dict(v=24), dict(k=32), dict(kept=0), dict(kept=2), dict(keep=0), dict(keep=2),
                dict(src=0), dict(src=3), dict(dst=0), dict(dst=2), dict(sb=0), dict(db=0), dict(sb=-1), dict(db=-1),
                dict(w=2), dict(num_rows=0), dict(max_len=0), dict(rows=1), dict(dst_rows=1), dict(n=-1), dict(max_keep=-1)):
        assert move(**bad) == INVALID, bad
    assert move(desc=_desc(kv=1, dim=40)) == UNSUPPORTED and move(desc=_desc(dim=272)) == UNSUPPORTED
    assert move(desc=_desc(block=8)) == UNSUPPORTED
    assert move(n=1 << 30) == UNSUPPORTED and move(max_keep=(1 << 30) + 1) == UNSUPPORTED
    assert move(n=0) == OK and move(max_keep=0) == OK and move(w=0, num_rows=0, max_len=0, n=0) == OK


def test_refusals_of_the_python_calls():
    import paged_kv_cache_160_gb300 as pkv
    i32 = torch.int32
    q, cu, start, tables = torch.zeros((3, 8, 128)), torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros((2, 4), dtype=i32)
    ws, lse = torch.zeros(64), torch.zeros((3, 8))
    desc = _desc()
    with pytest.raises(ValueError):                            # one chunk too many
        pkv.pkv_paged_chunk_attention(q, q, torch.zeros(4, dtype=i32), start, q, q, desc, tables, 0.1, ws)
    with pytest.raises(ValueError):
        pkv.pkv_paged_chunk_attention(q, q, cu, start, q, q, desc, tables, 0.1, ws, lse=torch.zeros((3, 7)))
    with pytest.raises(ValueError):
        pkv.pkv_paged_chunk_attention(q[:2], q, cu, start, q, q, desc, tables, 0.1, ws)
    with pytest.raises(ValueError):
        pkv.pkv_paged_chunk_attention(q, q, cu, start, q, q, _desc(dim=64), tables, 0.1, ws)
    with pytest.raises(ValueError):                            # a CPU tensor
        pkv.pkv_paged_chunk_attention(q, q, cu, start, q, q, desc, tables, 0.1, ws)
    w = torch.zeros((2, 4, 50))
    for out, prior, rows in ((w[:1], None, None), (w[:, :3], None, None), (w, w[:, :, :40], None), (w.double(), None, None),
                             (w, None, torch.zeros(3, dtype=i32)), (w, None, torch.zeros(2, dtype=torch.int64))):
        with pytest.raises(ValueError):
            pkv.pkv_attention_weights(out, prior, 1.0, q, lse, cu, start, q, desc, tables, 0.1, rows)
    kept, n = torch.zeros((2, 4, 8), dtype=i32), torch.zeros(2, dtype=i32)
    for bad in ((kept.long(), w, n, n), (kept[:1], w, n, n), (kept, w[:, :3], n, n), (kept, w[:1], n, n), (kept, w, n, n[:1])):
        with pytest.raises(ValueError):
            pkv.pkv_evict_select(*bad)
    for bad in (dict(kept=kept[:, :3]), dict(kept=kept.long()), dict(weights=w[:1]), dict(weights=w[:, :2])):
        a = dict(dict(kept=kept, weights=None), **bad)
        with pytest.raises(ValueError):
            pkv.pkv_evict_compact(q, q, desc, a["kept"], n, tables, None, a["weights"])


def test_block_manager_eviction():
    import paged_kv_cache_160_gb300 as pkv
    bm = pkv.BlockManager(12, 16)
    bm.allocate(0, 70)                                         # 0 .. 4
    bm.allocate(1, 20)                                         # 5, 6
    bm.fork(1, 2)
    src, lens, dst = bm.evict([0, 1], [33, 10], 5, 4)
    assert src == [[0, 1, 2, 3, 4], [5, 6, -1, -1, -1]] and lens == [70, 20]
    assert dst == [[0, 1, 2, -1], [7, -1, -1, -1]]             # block 5 is shared with sequence 2: a new one
    assert bm.export([0, 1, 2], 3) == ([[0, 1, 2], [7, -1, -1], [5, 6, -1]], [33, 10, 20])
    assert bm.free_queue() == [8, 9, 10, 11, 3, 4] and [bm.ref_cnt(b) for b in (5, 6, 7, 3)] == [1, 1, 1, 0]
    # unchanged lengths keep shared blocks; down to nothing releases all
    bm.fork(2, 3)
    assert bm.evict([2, 0], [20, 0], 3, 3) == ([[5, 6, -1], [0, 1, 2]], [20, 33], [[5, 6, -1], [-1, -1, -1]])
    assert bm.ref_cnt(5) == 2 and bm.free_queue() == [8, 9, 10, 11, 3, 4, 0, 1, 2]
    assert bm.append_slot(0) == (8 * 16, None)


def test_block_manager_eviction_of_both_holders():
    """Both sequences of a fork are cut in one call: neither writes the block that the other reads."""
    import paged_kv_cache_160_gb300 as pkv
    bm = pkv.BlockManager(8, 16)
    bm.allocate(0, 40)
    bm.fork(0, 1)
    _, _, dst = bm.evict([0, 1], [20, 17], 3, 2)
    assert dst == [[3, 4], [5, 6]]
    assert [bm.ref_cnt(b) for b in range(8)] == [0, 0, 0, 1, 1, 1, 1, 0]
    assert bm.free_queue() == [7, 0, 1, 2]


def test_block_manager_eviction_drops_hashes():
    import paged_kv_cache_160_gb300 as pkv
    bm = pkv.BlockManager(8, 16)
    tokens = list(range(48))
    assert bm.allocate_cached(0, tokens) == 0 and bm.num_cached() == 3
    assert bm.evict([0], [20], 3, 2)[2] == [[0, 1]]
    assert [bm.block_hash(b) is None for b in range(3)] == [True, True, False]
    assert bm.allocate_cached(1, tokens) == 0                  # nothing of the old prefix is found
    # a shared cached prefix stays
    assert bm.allocate_cached(2, tokens) == 48
    _, _, dst = bm.evict([2], [20], 3, 2)
    assert not set(dst[0]) & set(bm.export([1], 3)[0][0])
    bm.free(2)
    assert bm.allocate_cached(3, tokens) == 48


def test_block_manager_eviction_refusals():
    import paged_kv_cache_160_gb300 as pkv
    bm = pkv.BlockManager(4, 16)
    bm.allocate(0, 40)
    bm.fork(0, 1)
    state = (bm.export([0, 1], 3), bm.free_queue())
    for seqs, lens, a, b in (([0, 0], [5, 5], 3, 3), ([7], [1], 3, 3), ([0], [41], 3, 3), ([0], [-1], 3, 3), ([0], [20], 2, 3),
                             ([0], [20], 3, 1)):
        with pytest.raises(pkv.PkvError):
            bm.evict(seqs, lens, a, b)
    with pytest.raises(pkv.NoBlocksError):
        bm.evict([0], [20], 3, 2)                              # two shared blocks, one free
    with pytest.raises(ValueError):
        bm.evict([0], [20, 3], 3, 3)
    assert (bm.export([0, 1], 3), bm.free_queue()) == state
    bm.set_host_pool(4)
    bm.swap_out(0)
    with pytest.raises(pkv.PkvError):
        bm.evict([0], [5], 3, 3)
    assert bm.evict([], [], 0, 0) == ([], [], [])
    assert bm.evict([1], [0], 3, 0)[2] == [[]]


# ---------------------------------------------------------------------------------------
# the oracle, by hand
# ---------------------------------------------------------------------------------------

def test_oracle_chunk_and_weights():
    ln2 = float(np.log(2.0))
    q = np.zeros((2, 2, 16))
    q[:, :, 0] = [[ln2, 0.0], [2 * ln2, ln2]]
    k = np.zeros((3, 1, 16))
    k[:, 0, 0] = [0.0, 1.0, 2.0]
    v = np.zeros((3, 1, 16))
    v[:, 0, 0], v[:, 0, 1] = [1.0, 2.0, 4.0], [0.0, -3.0, 0.0]
    out, lse, size = evict.chunk_attention(q, k, v, 1, 1.0)
    # row 0 sees two keys: head 0 weighs them 1 : 2, head 1 evenly; row 1 sees three: 1 : 4 : 16 and 1 : 2 : 4
    assert np.allclose(out[:, :, 0], [[5 / 3, 1.5], [73 / 21, 3.0]]) and np.allclose(out[:, :, 1], [[-2, -1.5], [-12 / 21, -6 / 7]])
    assert np.allclose(np.exp(lse), [[3, 2], [21, 7]]) and np.allclose(size[:, :, 1], -out[:, :, 1])
    w = evict.chunk_weights(q, lse, k, 1, 1.0)
    assert np.allclose(w, [[1 / 3 + 1 / 2 + 1 / 21 + 1 / 7, 2 / 3 + 1 / 2 + 4 / 21 + 2 / 7, 16 / 21 + 4 / 7]])


def test_oracle_select_and_compact():
    nan, inf = float("nan"), float("inf")
    w = np.array([0.0, 5.0, 1.0, 5.0, nan, -inf, 7.0, 0.0, 2.0, 9.0])
    assert evict.select(w, 10, 3, 0, 0) == [1, 6, 9]
    assert evict.select(w, 9, 3, 0, 0) == [1, 3, 6] and evict.select(w, 9, 2, 0, 0) == [1, 6]     # the lower of two 5
    assert evict.select(w, 9, 4, 1, 1) == [0, 1, 6, 8] and evict.select(w, 9, 2, 2, 5) == [7, 8]
    assert evict.select(w, 9, 8, 0, 0) == [0, 1, 2, 3, 5, 6, 7, 8] and evict.select(w, 3, 9, 1, 1) == [0, 1, 2]
    cache = np.arange(2 * 1 * 2 * 1).reshape(2, 1, 2, 1)
    assert evict.compact(cache, [[[1, 2, 3]]], [3], [[1, 0]], [[1, 0]], 2).flatten().tolist() == [1, 1, 3, 0]
