"""CPU tests of the argument checks of the 4-bit cache, kv_read, prompt_attention and qk_rotary, and of
pkv_rope_table (host only).  Nothing here reaches a GPU."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import rotary

OK, INVALID, UNSUPPORTED = 0, 1, 2


def _fp4(nb=64, heads=4, block=16, dim=128):
    from paged_kv_cache_160_gb300._binding import CacheDesc
    return CacheDesc(nb, heads, block, dim, 3, None, None)


def test_fp4_descriptors():
    import paged_kv_cache_160_gb300 as pkv
    assert pkv.fp4_cache_shape(10, 4, 32, 128) == (10, 4, 2, 1152)
    for bad in ((10, 4, 8, 128), (10, 4, 16, 40)):
        with pytest.raises(ValueError):
            pkv.fp4_cache_shape(*bad)
    d = pkv.cache_desc_fp4(torch.zeros((10, 4, 2, 576), dtype=torch.uint8))
    assert (d.num_blocks, d.num_kv_heads, d.block_size, d.head_dim, d.kv_dtype) == (10, 4, 32, 64, 3)
    assert d.k_scale is None and d.v_scale is None
    for bad in (torch.zeros((10, 4, 2, 570), dtype=torch.uint8), torch.zeros((10, 4, 2, 576)),
                torch.zeros((10, 4, 576), dtype=torch.uint8)):
        with pytest.raises(ValueError):
            pkv.cache_desc_fp4(bad)
    L = pkv.lib
    # 16-row tiles and 16-element scales
    for desc in (_fp4(block=8), _fp4(dim=40)):
        assert L.pkv_copy_blocks(16, 16, ctypes.byref(desc), 16, 1, None) == UNSUPPORTED
    assert L.pkv_copy_blocks(16, 16, ctypes.byref(_fp4()), 16, 0, None) == OK
    # ready 4-bit rows are not taken
    assert L.pkv_kv_write(16, 16, 3, 4, 16, 16, 16, ctypes.byref(_fp4()), None) == UNSUPPORTED
    # the tile stream and the paged prefill have no 4-bit path
    assert L.pkv_stream_tiles(16, 16, ctypes.byref(_fp4()), 16, 4, 16, None) == UNSUPPORTED
    assert L.pkv_paged_prefill_chunk(16, 16, 1, 16, 16, 1, 8, 8, 8, 16, 16, ctypes.byref(_fp4()), 16, 8, 0.1,
                                     None) == UNSUPPORTED


def test_fp4_decode_checks():
    import paged_kv_cache_160_gb300 as pkv
    L = pkv.lib

    def both(desc, hq=8, qd=1, out=16, part=0):
        args = (out, 16, qd, 4, hq, 16, 16, ctypes.byref(desc), 16, 8, 16, 128, 0.1, part)
        a = L.pkv_paged_decode(*args, 16, 1 << 30, None)
        assert a == L.pkv_paged_decode_noalloc(*args, None)
        return a

    assert both(_fp4(), hq=6) == INVALID
    assert both(_fp4(), hq=36) == UNSUPPORTED               # nine query heads per kv head
    assert both(_fp4(dim=96)) == UNSUPPORTED
    assert both(_fp4(block=48)) == UNSUPPORTED
    assert both(_fp4(), qd=2) == INVALID
    assert both(_fp4(), qd=3) == INVALID
    assert both(_fp4(), out=24) == INVALID
    assert both(_fp4(), part=24) == INVALID


def test_kv_read_checks():
    import paged_kv_cache_160_gb300 as pkv
    from paged_kv_cache_160_gb300._binding import CacheDesc

    def read(ko=16, vo=16, dt=1, total=8, cu=16, seqs=1, tab=16, width=4, k=16, v=16, desc=None):
        return pkv.lib.pkv_kv_read(ko, vo, dt, total, cu, seqs, tab, width, k, v, ctypes.byref(desc or _fp4()), None)

    assert read(total=0) == OK and read(seqs=0) == OK
    assert read(total=-1) == INVALID and read(seqs=-1) == INVALID and read(width=0) == INVALID
    assert read(dt=2) == INVALID and read(dt=3) == INVALID
    for name in ("ko", "vo", "cu", "tab", "k", "v"):
        assert read(**{name: None}) == INVALID, name
    for name in ("ko", "vo", "k", "v"):
        assert read(**{name: 24}) == INVALID, name
    assert read(cu=18) == INVALID and read(tab=18) == INVALID
    assert read(desc=CacheDesc(64, 4, 16, 128, 0, None, None)) == UNSUPPORTED      # bf16 rows of an f16 cache
    assert read(desc=CacheDesc(64, 4, 16, 24, 1, None, None)) == UNSUPPORTED
    assert read(desc=CacheDesc(64, 4, 16, 128, 2, None, None)) == INVALID          # e4m3 without scales


def test_prompt_attention_checks():
    import paged_kv_cache_160_gb300 as pkv
    base = dict(out=16, q=16, k=16, v=16, dt=1, cq=16, ck=16, seqs=1, tq=8, tk=8, mq=8, hq=4, hkv=2, dim=128, so=512, sq=512,
                sk=256, sv=256, scale=0.1)

    def call(**kw):
        a = {**base, **kw}
        return pkv.lib.pkv_prompt_attention(*a.values(), None)

    for name in ("seqs", "tq", "mq"):
        assert call(**{name: 0}) == OK, name
    for name in ("seqs", "tq", "tk", "mq"):
        assert call(**{name: -1}) == INVALID, name
    for bad in (dict(hq=3), dict(hq=0), dict(hkv=0), dict(dt=2), dict(dt=3), dict(scale=0.0), dict(scale=-1.0),
                dict(scale=float("nan")), dict(out=None), dict(q=None), dict(k=None), dict(v=None), dict(cq=None),
                dict(ck=None), dict(out=24), dict(q=24), dict(k=8), dict(v=8), dict(cq=18), dict(ck=18), dict(sq=511),
                dict(sq=504), dict(so=500), dict(sk=248), dict(sv=255), dict(so=-512)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(dim=96, so=4096, sq=4096, sk=4096, sv=4096), dict(seqs=65536),
                dict(hq=65536, hkv=1, so=1 << 24, sq=1 << 24), dict(sq=1 << 38)):
        assert call(**bad) == UNSUPPORTED, bad


def test_qk_rotary_checks():
    import paged_kv_cache_160_gb300 as pkv
    base = dict(qo=16, q=16, ko=16, k=16, dt=1, t=4, hq=4, hkv=2, dim=128, sqo=512, sq=512, sko=256, sk=256, pos=16, tab=16,
                rot=128, layout=0, mag=1.0, qw=None, kw=None, eps=1e-6)

    def call(**kw):
        a = {**base, **kw}
        return pkv.lib.pkv_qk_rotary(*a.values(), None)

    assert call(t=0) == OK and call(hq=0, hkv=0) == OK
    for bad in (dict(t=-1), dict(hq=-1), dict(hkv=-1), dict(dim=0), dict(rot=0), dict(rot=144), dict(dt=2), dict(dt=3),
                dict(layout=2), dict(qo=None), dict(q=None), dict(ko=None), dict(k=None), dict(pos=None), dict(tab=None),
                dict(q=24), dict(ko=8), dict(pos=18), dict(tab=12), dict(sq=500), dict(sq=504), dict(sk=248), dict(qw=8),
                dict(kw=24), dict(qw=16, eps=-1.0), dict(qw=16, eps=float("nan"))):
        assert call(**bad) == INVALID, bad
    for bad in (dict(dim=100, rot=16, sq=800, sqo=800, sk=800, sko=800), dict(rot=24), dict(dim=272, sq=2048, sqo=2048)):
        assert call(**bad) == UNSUPPORTED, bad


@pytest.mark.parametrize("scaling,kw", [("none", {}), ("linear", dict(factor=8.0)), ("ntk", dict(factor=2.5)),
                                        ("parts", dict(factor=8.0, original_context=8192.0, alpha=1.0, beta=32.0)),
                                        ("parts", dict(factor=4.0, original_context=300.0, alpha=1.0, beta=4.0))])
@pytest.mark.parametrize("rot,base", [(128, 10000.0), (16, 1e6), (64, 500.0)])
def test_rope_table_is_turns_in_2_to_minus_64(rot, base, scaling, kw):
    """Each entry is f_i / 2 pi to 2^-64 and double's rounding (a few 2^-53 of it)."""
    import paged_kv_cache_160_gb300 as pkv
    t = pkv.pkv_rope_table(rot, base, scaling, **kw)
    assert t.shape == (rot // 2,) and (t >= 0).all()
    want = rotary.frequencies(rot, base, scaling, **kw) / (2 * np.pi)
    got = t.numpy().astype(np.float64) * 2.0 ** -64
    assert (np.abs(got - want) <= 2.0 ** -48 * want + 2.0 ** -64).all()


def test_rope_table_refusals():
    import paged_kv_cache_160_gb300 as pkv
    for a in ((0,), (15,), (16, 1.0), (16, float("nan")), (16, float("inf")), (16, 1e4, "linear", 0.5),
              (16, 1e4, "linear", float("nan")), (2, 1e4, "ntk", 2.0), (16, 1e4, "parts", 2.0, 0.0),
              (16, 1e4, "parts", 2.0, 4096.0, 4.0, 4.0), (16, 1e4, "parts", 2.0, 4096.0, float("nan"), 4.0)):
        with pytest.raises(pkv.PkvError):
            pkv.pkv_rope_table(*a)
    with pytest.raises(KeyError):
        pkv.pkv_rope_table(16, 1e4, "dynamic")
    assert pkv.lib.pkv_rope_table(None, 16, 1e4, 0, 1.0, 0.0, 0.0, 0.0) == INVALID
    buf = (ctypes.c_uint64 * 8)()
    assert pkv.lib.pkv_rope_table(buf, 16, 1e4, 4, 1.0, 0.0, 0.0, 0.0) == INVALID


def test_binding_refuses_cpu_tensors_and_split_heads():
    import paged_kv_cache_160_gb300 as pkv
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    pos, cu = torch.zeros(2, dtype=torch.int32), torch.tensor([0, 2], dtype=torch.int32)
    with pytest.raises(ValueError):
        pkv.pkv_qk_rotary(q, q, q, q, pos, pkv.pkv_rope_table(64))
    with pytest.raises(ValueError):
        pkv.pkv_prompt_attention(q, q, q, q, cu, cu, 2, 0.1)
    with pytest.raises(ValueError):
        pkv.pkv_kv_read(q, q, cu, torch.zeros((1, 1), dtype=torch.int32), q, q, _fp4(heads=4, dim=64))
