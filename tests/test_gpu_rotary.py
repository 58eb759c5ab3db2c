"""GPU parity of pkv_qk_rotary against the float64 definition.

Bound per element, with u the half step of the type (finfo.eps / 2): the last rounding is u |y|; before
it everything is fp32.  The phase keeps 31 bits of half a turn and is rounded to 24 (pi 2^-24 rad),
sincospi adds 2 ulp: together below 2^-21 on each of cos and sin, times |a| + |b| of the pair.  The norm:
a sum of at most 256 squares in a tree with chains of 8 (16 roundings), a division, rsqrt (2 ulp) and two
products stay below 2^-19 of the element.  The reference's own angles (fp64, positions below 2^31) are
good to 2^-21.  So |err| <= u |y| + 2^-18 (|a| + |b|), and 2^-25 more for fp16's subnormals.
"""
import numpy as np
import pytest
import torch

from oracle import rotary

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


SCALING = {"none": {}, "linear": dict(factor=8.0), "ntk": dict(factor=3.5),
           "parts": dict(factor=8.0, original_context=4096.0, alpha=1.0, beta=32.0)}


def _check(got, x, weight, eps, positions, freq, layout, mag, dtype):
    ref, size = rotary.rotate(rotary.rms_norm(x, weight, eps), positions, freq, layout, mag)
    u = torch.finfo(dtype).eps / 2
    err = np.abs(got.double().cpu().numpy() - ref)
    bound = u * np.abs(ref) + 2.0 ** -18 * size + 2.0 ** -25
    assert (err <= bound).all(), (float((err / bound).max()), np.argwhere(~(err <= bound))[:3])


def _run(tokens, hq, hkv, dim, rot, layout, scaling, dtype, norm, positions, packed=True, in_place=False, seed=0):
    import paged_kv_cache_160_gb300 as pkv
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn((tokens, hq + 2 * hkv, dim), generator=g).to(dtype)
    w = [(1 + 0.3 * torch.randn(dim, generator=g)).to(dtype) if norm else None for _ in range(2)]
    mag = 1.25 if scaling == "parts" else 1.0
    args = SCALING[scaling]
    table = pkv.pkv_rope_table(rot, 10000.0, scaling, **args).cuda()
    freq = rotary.frequencies(rot, 10000.0, scaling, **args)
    dev = qkv.cuda()
    q, k = dev[:, :hq], dev[:, hq:hq + hkv]
    if not packed:
        q, k = q.contiguous(), k.contiguous()
    v0 = dev[:, hq + hkv:].clone()
    qo, ko = (q, k) if in_place else (torch.full((tokens, hq, dim), 7.0, dtype=dtype, device="cuda"),
                                      torch.full((tokens, hkv, dim), 7.0, dtype=dtype, device="cuda"))
    pkv.pkv_qk_rotary(qo, q, ko, k, torch.tensor(positions, dtype=torch.int32, device="cuda"), table, layout, mag,
                      *(t.cuda() if t is not None else None for t in w), 1e-5)
    torch.cuda.synchronize()
    x = qkv.double().numpy()
    pos = np.array(positions)
    live = pos >= 0
    for o, part, wt in ((qo, x[:, :hq], w[0]), (ko, x[:, hq:hq + hkv], w[1])):
        _check(o[torch.from_numpy(live)], part[live], None if wt is None else wt.double().numpy(), 1e-5, pos[live], freq,
               layout, mag, dtype)
        pad = o[torch.from_numpy(~live)]
        if len(pad):
            want = torch.from_numpy(part[~live]).to(dtype).cuda() if in_place else torch.full_like(pad, 7.0)
            assert torch.equal(pad, want)
    if in_place and packed:
        assert torch.equal(dev[:, hq + hkv:], v0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dim,rot", [(64, 64), (64, 16), (80, 48), (96, 96), (128, 128), (128, 64), (256, 256), (256, 32),
                                     (16, 16), (144, 80)])
def test_dims_and_layouts(dim, rot, layout, dtype):
    rng = np.random.default_rng(dim + rot)
    _run(5, 6, 2, dim, rot, layout, "none", dtype, True, rng.integers(0, 5000, 5), seed=dim)
    _run(3, 3, 1, dim, rot, layout, "none", dtype, False, rng.integers(0, 5000, 3), packed=False, seed=rot)


@pytest.mark.parametrize("scaling", ["linear", "ntk", "parts"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_scaled_frequencies(scaling, layout):
    _run(7, 4, 4, 128, 128, layout, scaling, torch.bfloat16, False, [0, 1, 17, 4095, 4096, 32767, 131071])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_far_positions(dtype):
    _run(6, 2, 1, 64, 64, "half", "none", dtype, False, [0, 1, 1 << 20, (1 << 24) + 1, (1 << 30) + 12345, (1 << 31) - 1])


@pytest.mark.parametrize("hq,hkv", [(1, 1), (28, 4), (40, 40), (71, 1), (1, 16)])
def test_head_counts(hq, hkv):
    _run(4, hq, hkv, 128, 128, "half", "none", torch.bfloat16, True, [3, 0, 99, 2048])


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("tokens,hq,hkv,dim,rot,layout", [
    (2500, 1, 1, 64, 64, "half"), (2501, 2, 1, 128, 32, "interleaved"), (3001, 5, 1, 256, 256, "half"),
    (1400, 40, 8, 96, 80, "half"), (1399, 33, 8, 80, 80, "interleaved"), (457, 3, 1, 128, 128, "half")])
def test_tiles_of_several_tokens(tokens, hq, hkv, dim, rot, layout, norm):
    """More tokens than CTAs, few heads and many, padding tokens among them."""
    g = np.random.default_rng(tokens + dim)
    positions = np.where(g.random(tokens) < 0.1, -1, g.integers(0, 1 << 18, tokens)).tolist()
    _run(tokens, hq, hkv, dim, rot, layout, "none", torch.bfloat16, norm, positions, in_place=norm, seed=3)


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_in_place_and_padding_tokens(layout, norm):
    _run(6, 5, 3, 96, 64, layout, "none", torch.float16, norm, [4, -1, 0, 300, -7, 12], in_place=True)
    _run(6, 5, 3, 96, 64, layout, "none", torch.float16, norm, [4, -1, 0, 300, -7, 12])


def test_one_side_only_and_one_weight_only():
    import paged_kv_cache_160_gb300 as pkv
    g = torch.Generator().manual_seed(5)
    q = torch.randn((3, 4, 64), generator=g).to(torch.bfloat16)
    k = torch.randn((3, 2, 64), generator=g).to(torch.bfloat16)
    w = (1 + 0.3 * torch.randn(64, generator=g)).to(torch.bfloat16)
    pos = torch.tensor([5, 9, 11], dtype=torch.int32, device="cuda")
    table, freq = pkv.pkv_rope_table(64).cuda(), rotary.frequencies(64, 10000.0)
    qo, ko = torch.empty_like(q, device="cuda"), torch.empty_like(k, device="cuda")
    none = torch.empty((3, 0, 64), dtype=torch.bfloat16, device="cuda")
    pkv.pkv_qk_rotary(qo, q.cuda(), none, none, pos, table)
    _check(qo, q.double().numpy(), None, 0, np.array([5, 9, 11]), freq, "half", 1.0, torch.bfloat16)
    pkv.pkv_qk_rotary(qo, q.cuda(), ko, k.cuda(), pos, table, k_weight=w.cuda(), eps=1e-5)
    _check(qo, q.double().numpy(), None, 0, np.array([5, 9, 11]), freq, "half", 1.0, torch.bfloat16)
    _check(ko, k.double().numpy(), w.double().numpy(), 1e-5, np.array([5, 9, 11]), freq, "half", 1.0, torch.bfloat16)


def test_zero_rows_and_a_nan_stay_in_their_head():
    import paged_kv_cache_160_gb300 as pkv
    q = torch.zeros((2, 3, 64), dtype=torch.bfloat16, device="cuda")
    q[0, 1] = 1.0
    q[0, 1, 5] = float("nan")
    k = torch.ones((2, 1, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    pkv.pkv_qk_rotary(qo, q, ko, k, torch.tensor([1, 2], dtype=torch.int32, device="cuda"),
                      pkv.pkv_rope_table(64).cuda(), q_weight=w, k_weight=w, eps=1e-6)
    assert (qo[0, 0] == 0).all() and (qo[0, 2] == 0).all() and (qo[1] == 0).all()
    assert torch.isnan(qo[0, 1]).all() and torch.isfinite(ko).all()


def test_captured_and_replayed_on_a_side_stream():
    import paged_kv_cache_160_gb300 as pkv
    g = torch.Generator().manual_seed(6)
    q, k = torch.randn((9, 4, 128), generator=g).half().cuda(), torch.randn((9, 2, 128), generator=g).half().cuda()
    pos = torch.arange(9, dtype=torch.int32, device="cuda")
    table = pkv.pkv_rope_table(128).cuda()
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    pkv.pkv_qk_rotary(qo, q, ko, k, pos, table)
    torch.cuda.synchronize()
    eager = qo.clone(), ko.clone()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        pkv.pkv_qk_rotary(qo, q, ko, k, pos, table)
    for step in range(3):
        qo.zero_()
        ko.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(qo, eager[0]) and torch.equal(ko, eager[1])
