"""GPU parity of pkv_prompt_attention against float64.

With A = sum_j p_j |v_j| and u = finfo.eps / 2 of the type: P is rounded to the type (u A); scores are fp32 sums of
at most 128 exact products, an error of the exponent below 2^-24 * 128 * scale * sum |q k| (under 2^-12 here); the
row maximum may trail by 2^8, which costs nothing in floating point; exp2 and the fp32 sums add less than 2^-13.
So |err| <= (u + 2^-11) A + u |out| + 2^-25.
"""
import numpy as np
import pytest
import torch

from oracle import prompt

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def _run(q_lens, k_lens, hq, hkv, dim, dtype, packed=False, seed=0, pad=0, scale=None, spread=1.0):
    import paged_kv_cache_160_gb300 as pkv
    dt = DT[dtype]
    g = torch.Generator().manual_seed(seed + sum(q_lens))
    tq, tk = sum(q_lens), sum(k_lens)
    scale = dim ** -0.5 if scale is None else scale
    if packed:
        assert q_lens == k_lens
        qkv = (spread * torch.randn((tq + pad, hq + 2 * hkv, dim), generator=g)).to(dt)
        qkv[tq:] = float("nan")
        dev = qkv.cuda().split([hq, hkv, hkv], 1)
        q, k, v = (t[:tq] for t in qkv.split([hq, hkv, hkv], 1))
    else:
        q, k, v = ((spread * torch.randn((n + pad, h, dim), generator=g)).to(dt)
                   for n, h in ((tq, hq), (tk, hkv), (tk, hkv)))
        q[tq:] = float("nan")
        k[tk:] = float("nan")
        v[tk:] = float("inf")
        dev = [t.cuda() for t in (q, k, v)]
        q, k, v = q[:tq], k[:tk], v[:tk]
    out = torch.full((tq + pad, hq, dim), 5.0, dtype=dt, device="cuda")
    cu = [torch.tensor(np.cumsum([0] + n), dtype=torch.int32, device="cuda") for n in (q_lens, k_lens)]
    pkv.pkv_prompt_attention(out, *dev, *cu, max(q_lens + [1]), scale)
    assert pkv.pkv_get_device_error() == 0
    assert (out[tq:] == 5.0).all()
    ref, size = prompt.prompt_attention(*(t.double().numpy() for t in (q, k, v)), q_lens, k_lens, scale)
    u = torch.finfo(dt).eps / 2
    err = np.abs(out[:tq].double().cpu().numpy() - ref)
    bound = (u + 2.0 ** -11) * size + u * np.abs(ref) + 2.0 ** -25
    assert (err <= bound).all(), (float(np.nanmax(err / bound)), np.argwhere(~(err <= bound))[:3])
    return out


@pytest.mark.parametrize("n", [1, 2, 127, 128, 129, 255, 256, 257, 400])
@pytest.mark.parametrize("dim", [64, 128])
def test_one_prompt(n, dim):
    _run([n], [n], 4, 2, dim, "bf16", pad=3)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (3, 1), (4, 4), (7, 1), (6, 2), (9, 3)])
def test_groups(hq, hkv, dim, dtype):
    _run([300, 1, 129], [300, 1, 129], hq, hkv, dim, dtype, packed=True, seed=hq)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_packed_sequences_with_empty_ones(dtype):
    lens = [0, 5, 0, 0, 130, 64, 1, 200, 0]
    _run(lens, lens, 3, 1, 128, dtype, pad=70)
    _run(lens, lens, 4, 2, 64, dtype, packed=True, pad=200)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_lens,k_lens", [([1], [1000]), ([7], [300]), ([128, 3], [256, 131]), ([140], [500]),
                                           ([1, 1, 1], [1, 128, 129]), ([200], [201])])
def test_chunks_after_a_history(q_lens, k_lens, dim):
    _run(q_lens, k_lens, 6, 2, dim, "bf16", pad=9)
    _run(q_lens, k_lens, 3, 3, dim, "f16")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_lens,k_lens,hq,hkv", [([1], [2100], 8, 1), ([1], [700], 4, 4), ([130], [1500], 3, 1),
                                                  ([5, 0, 40], [2300, 2500, 1], 4, 2), ([300], [1900], 2, 2),
                                                  ([2, 150], [2600, 1300], 1, 1)])
def test_few_rows_over_many_keys(q_lens, k_lens, hq, hkv, dim, dtype):
    """Few enough items that clusters of 2, 4 or 8 CTAs share the keys of each."""
    _run(q_lens, k_lens, hq, hkv, dim, dtype, pad=5)


def test_split_keys_with_a_block_that_has_none():
    # 200 rows over 2100 keys and 2 rows over none: some parts and some blocks are empty
    out = _run([200, 2], [4100, 0], 1, 1, 128, "bf16")
    assert (out[200:] == 0).all()
    out = _run([2400], [2100], 1, 1, 64, "f16")                # the first 300 rows see nothing
    assert (out[:300] == 0).all()


@pytest.mark.parametrize("dim", [64, 128])
def test_rows_without_keys_are_zero(dim):
    out = _run([10, 300, 4], [3, 40, 0], 2, 1, dim, "bf16")
    assert (out[:7] == 0).all() and (out[10:270] == 0).all() and (out[310:] == 0).all()
    out = _run([300, 150], [40, 0], 1, 1, dim, "f16")
    assert (out[:260] == 0).all() and (out[300:] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim,q_lens,k_lens,hq,hkv", [(128, [200, 90], [200, 90], 4, 2), (64, [130, 3], [330, 200], 3, 1),
                                                      (128, [300], [333], 1, 1), (64, [40], [900], 2, 2),
                                                      (128, [150], [1600], 3, 1)])
def test_only_what_a_row_attends_reaches_it(dim, q_lens, k_lens, hq, hkv, dtype):
    """Infinities and NaN in K and V rows: rows before them are as if they were not there, rows that attend
    them are not finite where float64 says so."""
    import paged_kv_cache_160_gb300 as pkv
    dt = DT[dtype]
    g = torch.Generator().manual_seed(dim + sum(q_lens))
    q, k, v = (torch.randn((n, h, dim), generator=g).to(dt) for n, h in ((sum(q_lens), hq), (sum(k_lens), hkv), (sum(k_lens), hkv)))
    # the second sequence's first key, a key in the middle of the first one's last tile, and its last key
    bad = [(k_lens[0] - 1, 0, 5, float("nan")), (k_lens[0] - min(40, q_lens[0] - 1), hkv - 1, 7, float("inf")),
           (k_lens[0] - min(30, q_lens[0] - 1), hkv - 1, dim - 1, -float("inf"))]
    if len(k_lens) > 1:
        bad.append((sum(k_lens) - 2, 0, 0, -float("inf")))
    for j, h, d, x in bad:
        v[j, h, d] = x
    kbad = k_lens[0] - min(20, q_lens[0] - 1)
    cu = [torch.tensor(np.cumsum([0] + n), dtype=torch.int32, device="cuda") for n in (q_lens, k_lens)]

    def run(kk):
        out = torch.empty((sum(q_lens), hq, dim), dtype=dt, device="cuda")
        pkv.pkv_prompt_attention(out, q.cuda(), kk.cuda(), v.cuda(), *cu, max(q_lens), dim ** -0.5)
        assert pkv.pkv_get_device_error() == 0
        return out.double().cpu().numpy()

    with np.errstate(all="ignore"):
        ref, size = prompt.prompt_attention(*(t.double().numpy() for t in (q, k, v)), q_lens, k_lens, dim ** -0.5)
        got = run(k)
        fine = np.isfinite(ref)
        assert (~fine).any() and np.array_equal(np.isnan(got), np.isnan(ref))
        assert np.array_equal(got[~fine & ~np.isnan(ref)], ref[~fine & ~np.isnan(ref)])
        u = torch.finfo(dt).eps / 2
        assert (np.abs(got - ref)[fine] <= ((u + 2.0 ** -11) * size + u * np.abs(ref) + 2.0 ** -25)[fine]).all()
        # a NaN key: rows from it on are NaN throughout (in the heads that see it), the others as before
        k2 = k.clone()
        k2[kbad, 0, 3] = float("nan")
        again = run(k2)
        first = kbad - (k_lens[0] - q_lens[0])                 # the first row that attends it
        heads = np.arange(hq) // (hq // hkv) == 0
        rows = np.arange(sum(q_lens))
        hit = (rows >= max(first, 0)) & (rows < q_lens[0])
        assert np.isnan(again[hit][:, heads]).all()
        assert np.array_equal(again[~hit], got[~hit], equal_nan=True)
        assert np.array_equal(again[:, ~heads], got[:, ~heads], equal_nan=True)


@pytest.mark.parametrize("dim,hq,hkv", [(128, 3, 1), (64, 4, 2), (128, 1, 1)])
def test_one_long_prompt_among_many_short_ones(dim, hq, hkv):
    """Skewed lengths: the items are numbered sequence by sequence."""
    rng = np.random.default_rng(dim + hq)
    lens = [int(n) for n in rng.integers(0, 12, 90)]
    lens[37] = 1500
    _run(lens, lens, hq, hkv, dim, "bf16", seed=3)
    lens[37], lens[89] = 5, 1030
    _run(lens, [n + 3 for n in lens], hq, hkv, dim, "f16", seed=4)


def test_a_grid_dimension_does_not_bound_the_length():
    """max_q_len may be any bound, even one whose blocks no grid dimension holds."""
    import paged_kv_cache_160_gb300 as pkv
    g = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn((300, h, 64), generator=g).to(torch.bfloat16).cuda() for h in (4, 2, 2))
    cu = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")
    outs = []
    for bound in (200, 20_000_000):
        out = torch.empty_like(q)
        pkv.pkv_prompt_attention(out, q, k, v, cu, cu, bound, 0.1)
        assert pkv.pkv_get_device_error() == 0
        outs.append(out)
    assert torch.equal(*outs)


def test_no_keys_at_all():
    _run([5, 0], [0, 0], 4, 2, 128, "bf16")


def test_large_scores_and_growing_maxima():
    """Rows whose maximum rises tile after tile (every rescaling path), and scores of several hundred."""
    import paged_kv_cache_160_gb300 as pkv
    n, dim = 700, 128
    q = torch.ones((n, 2, dim))
    k = (torch.arange(n).view(n, 1, 1) / 64.0 + 0.125 * torch.randn((n, 1, dim), generator=torch.Generator().manual_seed(3)))
    v = torch.randn((n, 1, dim), generator=torch.Generator().manual_seed(4))
    q, k, v = (t.to(torch.bfloat16).contiguous() for t in (q, k, v))
    ref, size = prompt.prompt_attention(*(t.double().numpy() for t in (q, k, v)), [n], [n], 0.25)
    out = torch.empty((n, 2, dim), dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    pkv.pkv_prompt_attention(out, q.cuda(), k.cuda(), v.cuda(), cu, cu, n, 0.25)
    assert pkv.pkv_get_device_error() == 0
    # the exponent's error: 2^-24 * 128 * 0.25 * 128 * 11 (the largest |q k| sums) < 2^-8.5
    u = torch.finfo(torch.bfloat16).eps / 2
    err = np.abs(out.double().cpu().numpy() - ref)
    assert (err <= (u + 2.0 ** -8) * size + u * np.abs(ref)).all()


def test_a_rows_result_does_not_depend_on_its_neighbours():
    """A sequence alone, and between others in one batch, bit for bit; and twice the same."""
    import paged_kv_cache_160_gb300 as pkv
    g = torch.Generator().manual_seed(9)
    lens = [77, 333, 260]
    q, k, v = (torch.randn((sum(lens), h, 128), generator=g).to(torch.bfloat16).cuda() for h in (4, 2, 2))

    def run(a, b):
        n = [x for x in lens[a:b]]
        s, e = sum(lens[:a]), sum(lens[:b])
        cu = torch.tensor(np.cumsum([0] + n), dtype=torch.int32, device="cuda")
        out = torch.empty_like(q[s:e])
        pkv.pkv_prompt_attention(out, q[s:e], k[s:e], v[s:e], cu, cu, max(n), 0.1)
        return out

    whole = run(0, 3)
    assert torch.equal(whole, run(0, 3))
    assert torch.equal(whole[77:410], run(1, 2)) and torch.equal(whole[410:], run(2, 3))


def test_inconsistent_lengths_are_flagged():
    import paged_kv_cache_160_gb300 as pkv
    q = torch.randn((300, 2, 64), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    k = q[:, :1].contiguous()

    def run(cu_q, cu_k, max_q=300):
        out = torch.full_like(q, 4.0)
        pkv.pkv_prompt_attention(out, q, k, k, *(torch.tensor(c, dtype=torch.int32, device="cuda") for c in (cu_q, cu_k)),
                                 max_q, 0.125)
        return (out[:, 0, 0] != 4.0).tolist(), pkv.pkv_get_device_error()

    good, err = run([0, 100, 300], [0, 100, 300])
    assert err == 0 and all(good)
    wrote, err = run([0, 100, 301], [0, 100, 300])             # past total_q: that sequence is left
    assert err == pkv.DEVERR["chunk"] and wrote == [i < 100 for i in range(300)]
    wrote, err = run([0, 100, 300], [0, 100, 50])
    assert err == pkv.DEVERR["chunk"] and wrote == [i < 100 for i in range(300)]
    wrote, err = run([0, 300], [0, 300], max_q=128)            # rows past the promised bound stay unwritten
    assert err == pkv.DEVERR["chunk"] and wrote == [i < 128 for i in range(300)]


def test_host_memory_is_refused():
    import paged_kv_cache_160_gb300 as pkv
    q = torch.zeros((4, 1, 64), dtype=torch.bfloat16, device="cuda")
    h = torch.zeros((4, 1, 64), dtype=torch.bfloat16).pin_memory()
    cu = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    a = (1, cu.data_ptr(), cu.data_ptr(), 1, 4, 4, 4, 1, 1, 64, 64, 64, 64, 64, 0.1, 0)
    L = pkv.lib.pkv_prompt_attention
    assert L(q.data_ptr(), h.data_ptr(), q.data_ptr(), q.data_ptr(), *a) == 1
    assert L(q.data_ptr(), q.data_ptr(), h.data_ptr(), q.data_ptr(), *a) == 1
    assert L(q.data_ptr(), q.data_ptr(), q.data_ptr(), h.data_ptr(), *a) == 1


def test_captured_and_replayed():
    import paged_kv_cache_160_gb300 as pkv
    g = torch.Generator().manual_seed(11)
    lens = [200, 64, 391]
    q, k, v = (torch.randn((sum(lens), h, 128), generator=g).half().cuda() for h in (6, 2, 2))
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    pkv.pkv_prompt_attention(out, q, k, v, cu, cu, 391, 0.09)
    torch.cuda.synchronize()
    eager, graph = out.clone(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):
            pkv.pkv_prompt_attention(out, q, k, v, cu, cu, 391, 0.09)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


@pytest.mark.parametrize("hq,hkv,dim", [(4, 1, 128), (7, 1, 128), (6, 2, 64), (28, 4, 128), (5, 1, 64), (40, 2, 128), (128, 1, 64),
                                        (131, 1, 128)])
@pytest.mark.parametrize("q_lens,k_lens", [([1, 2, 17, 18, 19, 0, 25], [40, 2, 17, 300, 129, 5, 20]), ([8] * 6, [700] * 6),
                                           ([1], [2049]), ([33, 70, 64], [33, 70, 200])])
def test_short_sequences_share_blocks_between_heads(q_lens, k_lens, hq, hkv, dim):
    """Few rows per sequence: a block holds them for all query heads of a kv head, whatever their number."""
    _run(q_lens, k_lens, hq, hkv, dim, "bf16", seed=hq + len(q_lens))


def test_blocks_shared_between_heads_in_rows_of_a_packed_projection():
    lens = [20, 1, 33, 7]
    _run(lens, lens, 14, 2, 128, "f16", packed=True, pad=3)


@pytest.mark.parametrize("dim,hq,hkv,longest", [(128, 4, 4, 0), (64, 4, 4, 1500), (128, 6, 3, 1500), (64, 6, 3, 0)])
def test_many_items_for_each_resident_cta(dim, hq, hkv, longest):
    """About 1,700 items, at least ten for each CTA that the GPU holds, numbered level by level and (with one long
    sequence among the short ones) sequence by sequence; infinities and NaN in V rows of scattered sequences."""
    import paged_kv_cache_160_gb300 as pkv
    rng = np.random.default_rng(dim + hq)
    n = 1700 // hkv
    q_lens = [int(x) for x in rng.integers(0, 50, n)]
    if longest:
        q_lens[n // 3] = longest
    k_lens = [x + int(rng.integers(0, 40)) for x in q_lens]
    tq, tk, starts = sum(q_lens), sum(k_lens), np.cumsum([0] + k_lens)
    g = torch.Generator().manual_seed(dim)
    q, k, v = (torch.randn((rows, h, dim), generator=g).to(torch.bfloat16) for rows, h in ((tq, hq), (tk, hkv), (tk, hkv)))
    for i in rng.permutation(n)[:60]:
        if k_lens[i]:
            j = starts[i] + int(rng.integers(0, k_lens[i]))
            v[j, int(rng.integers(0, hkv)), int(rng.integers(0, dim))] = rng.choice([float("nan"), float("inf"), -float("inf")])
    cu = [torch.tensor(np.cumsum([0] + x), dtype=torch.int32, device="cuda") for x in (q_lens, k_lens)]
    out = torch.full((tq, hq, dim), 5.0, dtype=torch.bfloat16, device="cuda")
    pkv.pkv_prompt_attention(out, q.cuda(), k.cuda(), v.cuda(), *cu, max(q_lens), dim ** -0.5)
    assert pkv.pkv_get_device_error() == 0
    got = out.double().cpu().numpy()
    with np.errstate(all="ignore"):
        ref, size = prompt.prompt_attention(*(t.double().numpy() for t in (q, k, v)), q_lens, k_lens, dim ** -0.5)
        fine = np.isfinite(ref)
        assert np.isnan(ref).any() and np.isinf(ref).any() and np.array_equal(np.isnan(got), np.isnan(ref))
        assert np.array_equal(got[np.isinf(ref)], ref[np.isinf(ref)])
        u = torch.finfo(torch.bfloat16).eps / 2
        err, bound = np.abs(got - ref)[fine], ((u + 2.0 ** -11) * size + u * np.abs(ref) + 2.0 ** -25)[fine]
    assert (err <= bound).all(), float((err / bound).max())


@pytest.mark.parametrize("dim,hq,hkv", [(128, 2, 2), (64, 8, 2)])
def test_many_long_items_for_each_resident_cta(dim, hq, hkv):
    """The same with several key tiles per item, so that stages and barriers wrap at every phase: one sequence's rows
    are those of the sequence alone."""
    import paged_kv_cache_160_gb300 as pkv
    rng = np.random.default_rng(hq)
    lens = [int(x) for x in rng.integers(1, 700, 900)]
    q, k, v = (torch.randn((sum(lens), h, dim), generator=torch.Generator().manual_seed(h + i)).to(torch.bfloat16).cuda()
               for i, h in enumerate((hq, hkv, hkv)))
    starts = np.cumsum([0] + lens)

    def run(a, b):
        n, s, e = lens[a:b], starts[a], starts[b]
        cu = torch.tensor(np.cumsum([0] + n), dtype=torch.int32, device="cuda")
        out = torch.empty_like(q[s:e])
        pkv.pkv_prompt_attention(out, q[s:e], k[s:e], v[s:e], cu, cu, max(n), dim ** -0.5)
        return out

    whole = run(0, 900)
    assert torch.equal(whole, run(0, 900))
    for a in (0, 150, 300, 450, 600, 750):                     # fewer items each, in other CTAs
        assert torch.equal(whole[starts[a]:starts[a + 150]], run(a, a + 150))
    assert pkv.pkv_get_device_error() == 0
    for i in (3, 444, 899):
        s, e = starts[i], starts[i + 1]
        ref, size = prompt.prompt_attention(*(t[s:e].double().cpu().numpy() for t in (q, k, v)), [e - s], [e - s], dim ** -0.5)
        u = torch.finfo(torch.bfloat16).eps / 2
        err = np.abs(whole[s:e].double().cpu().numpy() - ref)
        assert (err <= (u + 2.0 ** -11) * size + u * np.abs(ref) + 2.0 ** -25).all()
