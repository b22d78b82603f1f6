"""Attention of new (drafted) tokens over a key/value cache against float64: trees, chains and single tokens,
ragged lengths, empty prefixes and rows, every cache type, both head dims."""
import math

import pytest
import torch

import cache_util as cu
import sequence_sharded_exact_gb300 as ra
from sequence_sharded_exact_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def _clean_status():
    torch.cuda.set_device(0)
    ra.device_status()
    yield
    assert ra.device_status() == 0


def _i32(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device=DEV)


def _randn(*shape, seed, dtype=F32, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype).to(DEV)


def _cache(B, Hkv, cap, d, dtype, cdt, seed, scale=1.0):
    """A full cache; with e4m3, of rows of very different scales in v."""
    cache = ra.cache_alloc(B, Hkv, cap, d, cdt)
    k, v = _randn(B, Hkv, cap, d, seed=seed, scale=scale), _randn(B, Hkv, cap, d, seed=seed + 1)
    if cdt == E4M3:
        v *= 2.0 ** torch.randint(-6, 6, (B, Hkv, cap, 1), generator=torch.Generator().manual_seed(seed + 2)).to(DEV)
    ra.cache_write(cache, k.to(dtype), v.to(dtype))
    return cache


def _weight_eps(dtype):
    return 2.0 ** -8 if dtype == BF else 0.0  # the weights are held in bfloat16 for the tensor cores' product


def _check(q, cache, lens, mask, ntok, out_dtype=None, what=""):
    got = ra.tree_fwd(q, cache, _i32(lens), mask=None if mask is None else mask.to(DEV), ntok=_i32(ntok), out_dtype=out_dtype)
    assert got[0].dtype == (out_dtype or q.dtype) and got[1].dtype == F32
    k, v = cu.cache_values(cache)
    cu.check_tree(got, cu.tree(q, k, v, lens, mask, ntok), _weight_eps(q.dtype), got[0].dtype, what)
    return got


CASES = [
    # B, H, Hkv, T, d, cap, lens, ntok, tree
    (1, 1, 1, 1, 64, 1, [0], None, False),                       # one key
    (1, 4, 1, 1, 128, 130, [129], None, False),                  # one token, a tile and a row
    (2, 8, 2, 5, 64, 640, [500, 0], [5, 3], True),               # ragged, an empty prefix
    (3, 8, 8, 7, 128, 300, [1, 127, 250], [7, 1, 0], True),      # a sequence without tokens
    (1, 32, 8, 16, 128, 2000, [1900], None, True),               # 64 query rows, split over CTAs
    (4, 8, 1, 9, 128, 1000, [0, 5, 640, 991], None, True),       # 72 rows, the last row of the cache
    (1, 16, 2, 33, 64, 700, [513], [31], True),                  # 264 rows
    (2, 6, 3, 1, 128, 4500, [4321, 17], None, False),
    (5, 2, 2, 3, 64, 129, [126, 125, 0, 64, 1], None, False),    # the chain without a mask
    (37, 4, 4, 2, 64, 40, [(7 * b) % 38 for b in range(37)], [b % 3 for b in range(37)], True),  # more than a warp of sequences
    (2, 64, 8, 17, 128, 400, [300, 383], None, True),            # 136 rows per kv head
]
TYPES = [(F32, F32), (F32, E4M3), (BF, BF), (BF, E4M3)]


@pytest.mark.parametrize("dtype,cdt", TYPES)
@pytest.mark.parametrize("B,H,Hkv,T,d,cap,lens,ntok,tree", CASES)
def test_against_float64(B, H, Hkv, T, d, cap, lens, ntok, tree, dtype, cdt):
    cache = _cache(B, Hkv, cap, d, dtype, cdt, seed=cap + T)
    q = _randn(B, H, T, d, seed=T, dtype=dtype)
    _check(q, cache, lens, cu.random_tree(B, T, cap) if tree else None, ntok)


@pytest.mark.parametrize("dtype,cdt", TYPES)
@pytest.mark.parametrize("B,H,Hkv,T,d,cap,lens", [
    (1, 16, 4, 8, 128, 20000, [19000]),         # several tiles per CTA, the last with rows past the end
    (1, 2, 1, 3, 64, 60000, [59001]),
    (1, 32, 1, 5, 128, 30000, [29995]),         # two query tiles
    (40, 4, 4, 2, 128, 700, [601 + b for b in range(40)]),  # several items per CTA
    (16, 20, 2, 15, 64, 500, [30 * b for b in range(16)]),  # and two query tiles
])
def test_several_tiles_and_items_per_cta(B, H, Hkv, T, d, cap, lens, dtype, cdt):
    cache = _cache(B, Hkv, cap, d, dtype, cdt, seed=cap)
    q = _randn(B, H, T, d, seed=T, dtype=dtype)
    first = _check(q, cache, lens, cu.random_tree(B, T, cap), None)
    mask = cu.random_tree(B, T, cap).to(DEV)
    for _ in range(20):
        again = ra.tree_fwd(q, cache, _i32(lens), mask=mask)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("dtype,cdt", TYPES)
def test_peaked_scores_and_a_maximum_that_grows(dtype, cdt):
    """Large keys: the running maximum grows over the tiles, by more than any rescale threshold; then one key far
    above all others, at the end, in the middle, at the start."""
    B, H, Hkv, T, d, cap = 1, 4, 2, 3, 128, 1500
    cache = ra.cache_alloc(B, Hkv, cap, d, cdt)
    k, v = _randn(B, Hkv, cap, d, seed=1), _randn(B, Hkv, cap, d, seed=2)
    q = _randn(B, H, T, d, seed=3, dtype=dtype)
    ramp = (torch.arange(cap, device=DEV) / cap * 6)[:, None]
    for at in (None, 1400, 700, 0):
        kk = k * (ramp if at is None else 1.0)
        if at is not None:
            kk[:, :, at] = 3 * q.float()[:, ::2, 0]
        ra.cache_write(cache, kk.to(dtype), v.to(dtype))
        _check(q, cache, [1490], None, None, what=f"at {at}")


@pytest.mark.parametrize("dtype,cdt", TYPES)
def test_rows_that_see_nothing_and_masks_of_zeros(dtype, cdt):
    B, H, Hkv, T, d, cap = 2, 4, 2, 6, 64, 300
    cache = _cache(B, Hkv, cap, d, dtype, cdt, seed=7)
    q = _randn(B, H, T, d, seed=8, dtype=dtype)
    mask = cu.random_tree(B, T, 9)
    mask[0, 2] = False
    mask[1, 0] = False
    out, lse = _check(q, cache, [0, 0], mask, None)
    assert torch.isinf(lse[0, :, 2]).all() and torch.isinf(lse[1, :, 0]).all() and (out[0, :, 2] == 0).all()
    _check(q, cache, [200, 0], torch.zeros(B, T, T, dtype=torch.bool), None)
    _check(q, cache, [200, 294], torch.zeros(T, T, dtype=torch.bool), [0, 6])


@pytest.mark.parametrize("dtype,cdt", TYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_what_a_query_does_not_see_has_no_part(dtype, cdt, bad):
    """NaN and infinities behind the sequence, and in drafted tokens that some queries do not see; those that do
    see one get what the formula gives (NaN)."""
    B, H, Hkv, T, d, cap = 2, 4, 2, 5, 128, 400
    k, v = _randn(B, Hkv, cap, d, seed=21), _randn(B, Hkv, cap, d, seed=22)
    lens, ntok = [200, 126], [5, 4]
    for b in range(B):
        k[b, :, lens[b] + ntok[b]:] = bad
        v[b, :, lens[b] + ntok[b]:] = bad
    q = _randn(B, H, T, d, seed=23, dtype=dtype)
    mask = torch.eye(T, dtype=torch.bool).repeat(B, 1, 1)
    mask[:, 4, 1] = True
    clean = ra.cache_alloc(B, Hkv, cap, d, cdt)
    ra.cache_write(clean, k.to(dtype), v.to(dtype))
    _check(q, clean, lens, mask, ntok, what="behind the end")
    ref, ref_lse = ra.tree_fwd(q, clean, _i32(lens), mask=mask.to(DEV), ntok=_i32(ntok))
    for which in ("k", "v"):
        kk, vv = k.clone(), v.clone()
        for b in range(B):
            (kk if which == "k" else vv)[b, :, lens[b] + 1, 3::7] = bad
        cache = ra.cache_alloc(B, Hkv, cap, d, cdt)
        ra.cache_write(cache, kk.to(dtype), vv.to(dtype))
        out, lse = ra.tree_fwd(q, cache, _i32(lens), mask=mask.to(DEV), ntok=_i32(ntok))
        for t in (0, 2, 3, 4):
            if t != 4:
                assert torch.equal(out[:, :, t], ref[:, :, t]) and torch.equal(lse[:, :, t], ref_lse[:, :, t]), (which, t)
        if which == "v":  # the columns that hold it, in the queries that see it (token 1; token 4 of the first sequence)
            seen = out[0][:, [1, 4]].float()
            assert not torch.isfinite(seen[:, :, 3::7]).any() and torch.equal(lse[:, :, 1], ref_lse[:, :, 1])
            cols = torch.ones(d, dtype=torch.bool)
            cols[3::7] = False
            if cdt != E4M3 or not math.isinf(bad):  # (an infinite element takes the whole row's scale)
                assert torch.equal(out[0][:, [1, 4]][:, :, cols], ref[0][:, [1, 4]][:, :, cols])


def test_the_same_from_run_to_run_and_for_any_workspace():
    B, H, Hkv, T, d, cap = 3, 8, 2, 12, 128, 3000
    cache = _cache(B, Hkv, cap, d, BF, E4M3, seed=31)
    q = _randn(B, H, T, d, seed=32, dtype=BF)
    lens, mask = _i32([2988, 1, 1500]), cu.random_tree(B, T, 33).to(DEV)
    first = ra.tree_fwd(q, cache, lens, mask=mask)
    need = ra.tree_workspace_size(B, H, Hkv, T, d, cap, BF, E4M3)
    for fill in (0, 255, 127):
        ws = torch.full((need,), fill, dtype=torch.uint8, device=DEV)
        again = ra.tree_fwd(q, cache, lens, mask=mask, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("cdt", [BF, E4M3])
def test_parts_of_a_sharded_cache_fold_together(cdt):
    """The prefix dealt out over three caches, the drafted tokens in the last: the parts' float32 outputs and lse
    merge into the whole cache's."""
    B, H, Hkv, T, d = 2, 8, 2, 4, 128
    lens = [700, 333]
    whole = _cache(B, Hkv, 710, d, BF, cdt, seed=41)
    q = _randn(B, H, T, d, seed=42, dtype=BF)
    mask = cu.random_tree(B, T, 43).to(DEV)
    ref_k, ref_v = cu.cache_values(whole)
    o, l = None, None
    for i in range(3):
        idx = [torch.arange(i, lens[b], 3) for b in range(B)]
        part = ra.cache_alloc(B, Hkv, 300, d, cdt)
        for t, src in zip(part, whole):
            if t is None:
                continue
            for b in range(B):
                rows = idx[b] if i < 2 else torch.cat([idx[b], lens[b] + torch.arange(T)])
                t[b].view(torch.uint8)[:, :len(rows)] = src[b].view(torch.uint8)[:, rows.to(DEV)]
        m = mask if i == 2 else torch.zeros(T, T, dtype=torch.bool, device=DEV)
        po, pl = ra.tree_fwd(q, part, _i32([len(x) for x in idx]), mask=m, out_dtype=F32)
        if o is None:
            o, l = po, pl
        else:
            ra.lse_merge(o, l, po, pl)
    cu.check_tree((o, l), cu.tree(q, ref_k, ref_v, lens, mask.cpu(), None), 2.0 ** -8, F32, "merged")


def test_lengths_outside_the_cache_are_clamped_and_reported():
    B, H, Hkv, T, d, cap = 3, 2, 1, 4, 64, 50
    cache = _cache(B, Hkv, cap, d, BF, BF, seed=51)
    q = _randn(B, H, T, d, seed=52, dtype=BF)
    got = ra.tree_fwd(q, cache, _i32([48, -3, 99]), ntok=_i32([4, 9, 2]))
    assert ra.device_status() == binding.RA_DEVICE_RANGE
    ref = ra.tree_fwd(q, cache, _i32([48, 0, 50]), ntok=_i32([2, 4, 0]))
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_captured_graph_replays_with_new_lengths_and_tokens():
    B, H, Hkv, T, d, cap = 2, 8, 2, 6, 128, 1200
    cache = _cache(B, Hkv, cap, d, BF, E4M3, seed=61)
    q = _randn(B, H, T, d, seed=62, dtype=BF)
    lens, mask = _i32([3, 900]), cu.random_tree(B, T, 63).to(DEV)
    ra.tree_fwd(q, cache, lens, mask=mask)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ra.tree_fwd(q, cache, lens, mask=mask)
    for new in ([1190, 0], [0, 17], [500, 501]):
        lens.copy_(torch.tensor(new))
        q.copy_(_randn(B, H, T, d, seed=sum(new), dtype=BF))
        graph.replay()
        ref = ra.tree_fwd(q, cache, lens, mask=mask)
        assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_two_streams_with_a_workspace_each():
    B, H, Hkv, T, d, cap = 1, 16, 4, 8, 128, 20000
    streams = [torch.cuda.Stream() for _ in range(2)]
    cache = _cache(B, Hkv, cap, d, BF, BF, seed=71)
    qs = [_randn(B, H, T, d, seed=72 + i, dtype=BF) for i in range(2)]
    lens = _i32([19000])
    refs = [ra.tree_fwd(q, cache, lens) for q in qs]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = ra.tree_fwd(qs[i], cache, lens)
    torch.cuda.synchronize()
    for a, b in zip(got, refs):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_offsets_beyond_32_bits():
    """A cache of more than 2^32 bytes per tensor: the last sequence's rows lie behind that offset."""
    B, H, Hkv, T, d, cap = 5, 4, 2, 2, 128, 1 << 21
    cache = ra.cache_alloc(B, Hkv, cap, d, BF)
    tail = 300
    k, v = _randn(B, Hkv, tail + T, d, seed=81, dtype=BF), _randn(B, Hkv, tail + T, d, seed=82, dtype=BF)
    lens = [tail] * B
    ra.cache_write(cache, k, v)
    q = _randn(B, H, T, d, seed=83, dtype=BF)
    got = ra.tree_fwd(q, cache, _i32(lens))
    ref = cu.tree(q, k.cpu().double(), v.cpu().double(), lens, None, None)
    cu.check_tree(got, ref, 2.0 ** -8, BF)
    rk, rv = ra.cache_read(cache, tail + T)
    assert torch.equal(rk, k) and torch.equal(rv, v)
    # tokens at the far end of the last sequence
    at = _i32([cap - T] * B)
    ra.cache_write(cache, k[:, :, :T].contiguous(), v[:, :, :T].contiguous(), at)
    rk, _ = ra.cache_read(cache, T, row0=cap - T)
    assert torch.equal(rk, k[:, :, :T])
    # all but the last prefix empty: 2^21 rows of zeros, and the tokens
    cache.k[4, :, :tail + T] = 0
    cache.v[4, :, :tail + T] = 0
    out, lse = ra.tree_fwd(q, cache, _i32([0, 0, 0, 0, cap - T]))
    s = torch.einsum("hgtd,hjd->hgtj", q[4].view(Hkv, H // Hkv, T, d).double(), k[4, :, :T].double()) / math.sqrt(d)
    e = s.exp() * torch.ones(T, T, device=DEV).tril().double()
    ref_l = (e.sum(-1) + cap - T).log()
    assert float((lse[4].view(Hkv, H // Hkv, T).double() - ref_l).abs().max()) <= 1e-4
    ref_o = torch.einsum("hgtj,hjd->hgtd", e, v[4, :, :T].double()) / (e.sum(-1, keepdim=True) + cap - T)
    assert float((out[4].view(Hkv, H // Hkv, T, d).double() - ref_o).abs().max()) <= 2.0 ** -7 * float(ref_o.abs().max())
