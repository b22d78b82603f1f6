"""Attention over a cache (tree_fwd) where its kernels' variants differ: few and many query rows per kv head, non-finite
queries, keys and values, growing maxima, far-apart row scales, unaligned index and mask tensors, memory around the outputs."""
import pytest
import torch

import cache_util as cu
import sequence_sharded_exact_gb300 as ra
from sequence_sharded_exact_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn

# H, Hkv, T, d: 2, 8 and 8 query rows per kv head, 20, 128, 256, 16 and 10
ROWS = [(2, 1, 1, 128), (4, 2, 4, 64), (8, 1, 1, 128), (8, 2, 5, 128), (4, 1, 32, 64), (4, 1, 64, 128),
        (8, 2, 4, 128), (2, 1, 5, 64)]
TYPES = [(F32, F32), (F32, E4M3), (BF, BF), (BF, E4M3)]


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


def _cache_of(k, v, dtype, cdt):
    cache = ra.cache_alloc(*k.shape, cdt)
    ra.cache_write(cache, k.to(dtype), v.to(dtype))
    return cache


def _check(q, cache, lens, mask, what=""):
    got = ra.tree_fwd(q, cache, _i32(lens), mask=None if mask is None else mask.to(DEV))
    k, v = cu.cache_values(cache)
    # bfloat16 queries' weights are rounded to bfloat16, or to a float16 that is finer, for the product
    cu.check_tree(got, cu.tree(q, k, v, lens, mask, None), 2.0 ** -8 if q.dtype == BF else 0.0, got[0].dtype, what)
    return got


@pytest.mark.parametrize("cdt", [BF, E4M3])
@pytest.mark.parametrize("H,Hkv,T,d", [r for r in ROWS if r[2] > 1] + [(6, 2, 2, 128)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_hidden_tokens_and_a_spoilt_prefix(H, Hkv, T, d, cdt, bad):
    """A drafted token's value that is not finite reaches the queries that see it, bit for bit no others; one in the
    prefix reaches every query of its kv head, in its columns."""
    B, lens = 2, [250, 131]
    cap = 256 + T
    k, v = _randn(B, Hkv, cap, d, seed=1), _randn(B, Hkv, cap, d, seed=2)
    q = _randn(B, H, T, d, seed=3, dtype=BF)
    mask = torch.eye(T, dtype=torch.bool)
    ref, ref_lse = ra.tree_fwd(q, _cache_of(k, v, BF, cdt), _i32(lens), mask=mask.to(DEV))
    vv = v.clone()
    for b in range(B):
        vv[b, :, lens[b] + 1, 3::7] = bad
    out, lse = ra.tree_fwd(q, _cache_of(k, vv, BF, cdt), _i32(lens), mask=mask.to(DEV))
    rest = [t for t in range(T) if t != 1]
    assert torch.equal(out[:, :, rest], ref[:, :, rest]) and torch.equal(lse, ref_lse)
    assert not torch.isfinite(out[:, :, 1, 3::7]).any()
    vv = v.clone()
    vv[1, 0, 70, 5::16] = bad
    out, lse = ra.tree_fwd(q, _cache_of(k, vv, BF, cdt), _i32(lens), mask=mask.to(DEV))
    G = H // Hkv
    assert torch.equal(lse, ref_lse) and torch.equal(out[0], ref[0]) and torch.equal(out[1, G:], ref[1, G:])
    assert not torch.isfinite(out[1, :G, :, 5::16]).any()
    if not (cdt == E4M3 and bad == float("inf")):  # (an infinite element takes the whole row's scale)
        cols = [c for c in range(d) if c % 16 != 5]
        assert torch.isfinite(out[1, :G][:, :, cols]).all()


@pytest.mark.parametrize("dtype,cdt", TYPES)
@pytest.mark.parametrize("H,Hkv,T,d", ROWS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_query_that_is_not_finite_spoils_its_own_row(H, Hkv, T, d, dtype, cdt, bad):
    B, lens, cap = 2, [300, 40], 300 + T
    k, v, q = _randn(B, Hkv, cap, d, seed=11), _randn(B, Hkv, cap, d, seed=12), _randn(B, H, T, d, seed=13, dtype=dtype)
    cache = _cache_of(k, v, dtype, cdt)
    ref, ref_lse = ra.tree_fwd(q, cache, _i32(lens))
    qq = q.clone()
    qq[0, H - 1, T - 1, 5] = bad
    qq[1, 0, 0, 7] = bad
    out, lse = ra.tree_fwd(qq, cache, _i32(lens))
    spoilt = torch.zeros(B, H, T, dtype=torch.bool, device=DEV)
    spoilt[0, H - 1, T - 1] = spoilt[1, 0, 0] = True
    assert torch.equal(out[~spoilt], ref[~spoilt]) and torch.equal(lse[~spoilt], ref_lse[~spoilt])
    assert not torch.isfinite(out[spoilt]).any()


@pytest.mark.parametrize("dtype,cdt", TYPES)
@pytest.mark.parametrize("H,Hkv,T,d", ROWS)
@pytest.mark.parametrize("down", [False, True])
def test_maxima_that_grow_and_shrink_along_the_cache(H, Hkv, T, d, dtype, cdt, down):
    """Scores that climb by some 40 binades over the cache, in steps within a tile and from tile to tile, or fall."""
    B, n = 1, 900
    cap = n + T
    ramp = torch.linspace(0, 28, cap)
    ramp = (ramp.flip(0) if down else ramp).view(1, 1, cap, 1).to(DEV)
    u = torch.ones(d, device=DEV)
    k = ramp / d ** 0.5 * u + 0.05 * _randn(B, Hkv, cap, d, seed=21)
    v = _randn(B, Hkv, cap, d, seed=22)
    q = (u + 0.1 * _randn(B, H, T, d, seed=23)).to(dtype)  # scores of some ramp * (1 +- 0.1)
    _check(q, _cache_of(k, v, dtype, cdt), [n], None)


@pytest.mark.parametrize("cdt", [BF, E4M3])
@pytest.mark.parametrize("masked", [False, True])
def test_more_than_256_query_rows_and_64_tokens(cdt, masked):
    B, H, Hkv, T, d, cap = 2, 4, 1, 100, 64, 330
    k, v, q = _randn(B, Hkv, cap, d, seed=31), _randn(B, Hkv, cap, d, seed=32), _randn(B, H, T, d, seed=33, dtype=BF)
    _check(q, _cache_of(k, v, BF, cdt), [230, 90], cu.random_tree(B, T, 34) if masked else None)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("H,Hkv,T,d", ROWS[:4] + ROWS[6:])
def test_rows_of_far_apart_scales(H, Hkv, T, d, dtype):
    """e4m3 rows whose scales lie up to 36 binades apart, the largest anywhere along the cache.  (With up to 16 query rows
    a weight times its row's scale is held to 2^-32 of the largest scale: 2^-32 * 448 * 2^E per key, at most 2^-18 of the
    largest row's |v| for these 600 keys and weights above 2^-12, far below the 2^-8 of sum w |v| that is allowed.)"""
    B, n = 2, 600
    cap = n + T
    k = _randn(B, Hkv, cap, d, seed=41) * 2.0 ** torch.randint(-3, 2, (B, Hkv, cap, 1), generator=torch.Generator().manual_seed(42)).to(DEV)
    v = _randn(B, Hkv, cap, d, seed=43) * 2.0 ** torch.randint(-18, 19, (B, Hkv, cap, 1), generator=torch.Generator().manual_seed(44)).to(DEV)
    q = _randn(B, H, T, d, seed=45, dtype=dtype, scale=0.25)
    _check(q, _cache_of(k, v, dtype, E4M3), [n, 333], None)


@pytest.mark.parametrize("dtype,cdt", TYPES)
@pytest.mark.parametrize("H,Hkv,T,d", [(4, 2, 4, 64), (4, 1, 16, 128), (4, 1, 64, 64)])
def test_unaligned_lengths_and_masks(H, Hkv, T, d, dtype, cdt):
    B, lens, cap = 3, [100, 0, 333], 333 + T
    k, v, q = _randn(B, Hkv, cap, d, seed=51), _randn(B, Hkv, cap, d, seed=52), _randn(B, H, T, d, seed=53, dtype=dtype)
    cache = _cache_of(k, v, dtype, cdt)
    mask, ntok = cu.random_tree(B, T, 54).to(DEV), _i32([T, T - 1, 1])
    ref, ref_lse = ra.tree_fwd(q, cache, _i32(lens), mask=mask, ntok=ntok)
    for off in (1, 3):
        ints = torch.zeros(2 * B + 8, dtype=torch.int32, device=DEV)
        ints[off:off + B], ints[off + B:off + 2 * B] = _i32(lens), ntok
        flat = torch.zeros(B * T * T + 8, dtype=torch.bool, device=DEV)
        flat[off:off + B * T * T] = mask.flatten()
        out, lse = ra.tree_fwd(q, cache, ints[off:off + B], mask=flat[off:off + B * T * T].view(B, T, T), ntok=ints[off + B:off + 2 * B])
        assert torch.equal(out, ref) and torch.equal(lse, ref_lse)


def _guarded(shape, dtype, seed):
    """A contiguous tensor in the middle of a buffer of a known pattern, and a check that the rest keeps it."""
    n = torch.Size(shape).numel() * torch.empty(0, dtype=dtype).element_size()
    pad = 4096
    buf = torch.randint(0, 256, (n + 2 * pad,), generator=torch.Generator().manual_seed(seed), dtype=torch.uint8).to(DEV)
    keep = buf.clone()

    def untouched():
        return torch.equal(buf[:pad], keep[:pad]) and torch.equal(buf[pad + n:], keep[pad + n:])

    return buf[pad:pad + n].view(dtype).view(shape), untouched


@pytest.mark.parametrize("dtype,cdt", TYPES)
@pytest.mark.parametrize("H,Hkv,T,d", ROWS + [(3, 3, 3, 64)])
@pytest.mark.parametrize("lens", [[1000, 77, 0], [5, 0, 3]])
def test_nothing_is_written_around_the_outputs(H, Hkv, T, d, dtype, cdt, lens):
    B, cap = len(lens), max(lens) + T
    k, v, q = _randn(B, Hkv, cap, d, seed=61), _randn(B, Hkv, cap, d, seed=62), _randn(B, H, T, d, seed=63, dtype=dtype)
    cache = _cache_of(k, v, dtype, cdt)
    ref, ref_lse = ra.tree_fwd(q, cache, _i32(lens))
    out, out_ok = _guarded((B, H, T, d), dtype, 64)
    lse, lse_ok = _guarded((B, H, T), F32, 65)
    ws, ws_ok = _guarded((ra.tree_workspace_size(B, H, Hkv, T, d, cap, dtype, cdt),), torch.uint8, 66)
    ra.tree_fwd(q, cache, _i32(lens), out=out, lse=lse, workspace=ws)
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    assert out_ok() and lse_ok() and ws_ok()


@pytest.mark.parametrize("dtype,cdt", TYPES)
@pytest.mark.parametrize("d", [64, 128])
def test_nothing_is_written_around_a_cache(d, dtype, cdt):
    B, Hkv, T, cap = 2, 3, 37, 40
    parts = [_guarded((B, Hkv, cap, d), cdt, 71), _guarded((B, Hkv, cap, d), cdt, 72)]
    if cdt == E4M3:
        parts += [_guarded((B, Hkv, cap), torch.uint8, 73), _guarded((B, Hkv, cap), torch.uint8, 74)]
    cache = ra.KVCache(*([p[0] for p in parts] + [None] * (4 - len(parts))))
    before = [p[0].clone() for p in parts]
    k, v = _randn(B, Hkv, T, d, seed=75, dtype=dtype), _randn(B, Hkv, T, d, seed=76, dtype=dtype)
    ra.cache_write(cache, k, v, _i32([3, 0]), ntok=_i32([T, 5]))
    assert all(ok() for _, ok in parts)
    for (x, _), was in zip(parts, before):
        x, was = x.view(torch.uint8), was.view(torch.uint8)
        assert torch.equal(x[0, :, :3], was[0, :, :3]) and torch.equal(x[1, :, 5:], was[1, :, 5:])
    want = ra.cache_alloc(B, Hkv, T, d, cdt)
    ra.cache_write(want, k, v)
    got, exp = ra.cache_read(cache, T, row0=3, dtype=dtype), ra.cache_read(want, T, dtype=dtype)
    assert torch.equal(got[0][0], exp[0][0]) and torch.equal(got[1][0], exp[1][0])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("B,H,Hkv,L,d", [(2, 4, 2, 33, 64), (1, 5, 1, 130, 128)])
def test_nothing_is_written_around_rotated_heads_and_their_gradients(B, H, Hkv, L, d, dtype):
    q, k = _randn(B, H, L, d, seed=81, dtype=dtype), _randn(B, Hkv, L, d, seed=82, dtype=dtype)
    wq, wk = _randn(d, seed=83), _randn(d, seed=84)
    dq, dk = _randn(B, H, L, d, seed=85, dtype=dtype), _randn(B, Hkv, L, d, seed=86, dtype=dtype)
    outs = [_guarded(t.shape, dtype, 87 + i) for i, t in enumerate((q, k))]
    ra.qk_norm_rope(q, k, wq, wk, q_out=outs[0][0], k_out=outs[1][0])
    ref = ra.qk_norm_rope(q, k, wq, wk)
    assert all(torch.equal(o, r) and ok() for (o, ok), r in zip(outs, ref))
    ref = ra.qk_norm_rope_bwd(q, k, wq, wk, dq, dk)
    grads = [_guarded(t.shape, dtype, 89 + i) for i, t in enumerate((q, k))]
    ws, ws_ok = _guarded((binding.library().ring_attn_qk_norm_rope_bwd_workspace_size(d),), torch.uint8, 91)
    got = ra.qk_norm_rope_bwd(q, k, wq, wk, dq, dk, dq=grads[0][0], dk=grads[1][0], workspace=ws)
    assert all(torch.equal(x, y) for x, y in zip(got, ref))
    assert ws_ok() and all(ok() for _, ok in grads)


def test_scratch_stays_with_the_stream_that_uses_it():
    """Given another stream than the current one, the call's own workspace is not given out again while that stream works."""
    B, H, Hkv, T, d, cap = 1, 4, 1, 64, 128, 2000
    cache = _cache_of(_randn(B, Hkv, cap, d, seed=1), _randn(B, Hkv, cap, d, seed=2), BF, BF)
    q, lens = _randn(B, H, T, d, seed=3, dtype=BF), _i32([1900])
    ref = ra.tree_fwd(q, cache, lens)
    need = ra.tree_workspace_size(B, H, Hkv, T, d, cap, BF, BF)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    at = torch.empty(need, dtype=torch.uint8, device=DEV).data_ptr()
    assert torch.empty(need, dtype=torch.uint8, device=DEV).data_ptr() == at  # a free block is given out again
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)
    out = ra.tree_fwd(q, cache, lens, stream=s)
    after = torch.empty(need, dtype=torch.uint8, device=DEV).data_ptr()
    assert s.query() or after != at
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(out, ref))


@pytest.mark.parametrize("cdt", [BF, E4M3])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [1, 2])
def test_many_short_sequences(T, d, cdt):
    """More (sequence, kv head) pairs than CTAs, of up to two tiles; some without tokens, some without a prefix."""
    B, H, Hkv, cap = 500, 4, 2, 150
    k, v, q = _randn(B, Hkv, cap, d, seed=101), _randn(B, Hkv, cap, d, seed=102), _randn(B, H, T, d, seed=103, dtype=BF)
    cache = _cache_of(k, v, BF, cdt)
    lens, ntok = [(37 * b) % (cap - T + 1) for b in range(B)], [T if b % 7 else b % 2 for b in range(B)]
    got = ra.tree_fwd(q, cache, _i32(lens), ntok=_i32(ntok))
    kk, vv = cu.cache_values(cache)
    cu.check_tree(got, cu.tree(q, kk, vv, lens, None, ntok), 2.0 ** -8, BF)
    again = ra.tree_fwd(q, cache, _i32(lens), ntok=_i32(ntok))
    assert all(torch.equal(x, y) for x, y in zip(got, again))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("H,Hkv,T,d", ROWS)
@pytest.mark.parametrize("at", [0, 130, 419])
def test_a_row_of_huge_values_that_hardly_counts(H, Hkv, T, d, dtype, at):
    """One row of v is 2^40 times the others and weighs e^-50 or less of them (2^-72: its contribution is 2^-32 of theirs):
    the others keep their precision, wherever it lies."""
    B, n = 1, 420
    cap = n + T
    u = torch.ones(d, device=DEV)
    k, v = 0.3 * _randn(B, Hkv, cap, d, seed=111), _randn(B, Hkv, cap, d, seed=112)
    k[:, :, at] = -60 / d ** 0.5 * u
    v[:, :, at] *= 2.0 ** 40
    q = (u + 0.05 * _randn(B, H, T, d, seed=113)).to(dtype)
    _check(q, _cache_of(k, v, dtype, E4M3), [n], None)


@pytest.mark.parametrize("cdt,T,cap", [(E4M3, 2, 1 << 22), (E4M3, 6, 1 << 22), (E4M3, 20, 1 << 22), (BF, 20, 1 << 21)])
def test_the_far_end_of_a_cache_of_more_than_32_bits(cdt, T, cap):
    """The last sequence of a cache of more than 2^32 bytes per tensor, its prefix all zeros (each weighs 1) up to the
    last T rows; 4, 12 and 40 query rows per kv head."""
    B, H, Hkv, d = 5, 4, 2, 128
    cache = ra.cache_alloc(B, Hkv, cap, d, cdt)
    k, v, q = _randn(B, Hkv, T, d, seed=121, dtype=BF), _randn(B, Hkv, T, d, seed=122, dtype=BF), _randn(B, H, T, d, seed=123, dtype=BF)
    lens = _i32([0, 0, 0, 0, cap - T])
    ra.cache_write(cache, k, v, lens)
    out, lse = ra.tree_fwd(q, cache, lens)
    kk, vv = (x[4].double() for x in ra.cache_read(cache, T, row0=cap - T))
    s = torch.einsum("hgtd,hjd->hgtj", q[4].view(Hkv, H // Hkv, T, d).double(), kk) / d ** 0.5
    e = s.exp() * torch.ones(T, T, device=DEV).tril().double()
    total = e.sum(-1) + cap - T
    assert float((lse[4].view(Hkv, H // Hkv, T).double() - total.log()).abs().max()) <= 1e-4
    ref = torch.einsum("hgtj,hjd->hgtd", e, vv) / total.unsqueeze(-1)
    mag = torch.einsum("hgtj,hjd->hgtd", e, vv.abs()) / total.unsqueeze(-1)
    # a weight's rounding to bfloat16 and the output's, 2^-8 each of the sum of magnitudes, and 2^-12 for the rest
    assert float(((out[4].view(Hkv, H // Hkv, T, d).double() - ref).abs() - (2.0 ** -7 + 2.0 ** -12) * mag).max()) <= 0
    assert torch.isfinite(out[:4]).all()
