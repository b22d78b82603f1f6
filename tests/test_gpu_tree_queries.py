"""Queries of the attention over a cache that ask much of their form in the products: not finite in a row that sees
nothing, or with one element far above the others."""
import pytest
import torch

import cache_util as cu
import sequence_sharded_exact_gb300 as ra

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
TYPES = [(F32, F32), (F32, E4M3), (BF, BF), (BF, E4M3)]
# H, Hkv, T, d: 4, 8, 16, 20, 128, 136 and 256 query rows per kv head
ROWS = [(4, 2, 2, 128), (8, 1, 1, 64), (4, 2, 8, 128), (8, 2, 5, 64), (4, 1, 32, 128), (8, 1, 17, 64), (4, 1, 64, 128)]


@pytest.fixture(autouse=True)
def _clean_status():
    torch.cuda.set_device(0)
    ra.device_status()
    yield
    assert ra.device_status() == 0


def _randn(*shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed))


def _cache_of(k, v, dtype, cdt):
    cache = ra.cache_alloc(*k.shape, cdt)
    ra.cache_write(cache, k.to(dtype).to(DEV), v.to(dtype).to(DEV))
    return cache


@pytest.mark.parametrize("dtype,cdt", TYPES)
@pytest.mark.parametrize("H,Hkv,T,d", ROWS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_row_that_sees_nothing_is_empty_whatever_its_query_holds(H, Hkv, T, d, dtype, cdt, bad):
    """Two sequences without a prefix, the second's tokens 0 see nothing, nor do the first's last ones: 0 and -infinity."""
    B, cap = 2, T + 3
    cache = _cache_of(_randn(B, Hkv, cap, d, seed=1), _randn(B, Hkv, cap, d, seed=2), dtype, cdt)
    q = _randn(B, H, T, d, seed=3).to(dtype).to(DEV)
    mask = torch.eye(T, dtype=torch.bool).repeat(B, 1, 1)
    mask[0, T - 1] = False
    mask[1, 0] = False
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    ref, ref_lse = ra.tree_fwd(q, cache, lens, mask=mask.to(DEV))
    q[0, :, T - 1, 5] = bad
    q[1, 0, 0] = bad
    out, lse = ra.tree_fwd(q, cache, lens, mask=mask.to(DEV))
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    assert bool((out[1, 0, 0] == 0).all()) and float(lse[1, 0, 0]) == -float("inf")
    assert bool((out[0, :, T - 1] == 0).all()) and bool((lse[0, :, T - 1] == -float("inf")).all())


@pytest.mark.parametrize("dtype,cdt", TYPES)
@pytest.mark.parametrize("H,Hkv,T,d", ROWS)
def test_a_query_with_one_element_far_above_the_others(H, Hkv, T, d, dtype, cdt):
    """Element 0 of every query is 2^12 times the others' size, and the keys have 0 there: the scores are the other
    elements'.  One to three keys, so that lse, which no rounding of weights touches, shows a score's error.

    bfloat16 queries of more than 16 rows per kv head over e4m3 are two 8-bit parts: exact down to 2^-13 of the row's
    largest, below that off by at most 2^-21 of it, so a score is off by sum_i e_i |k_i| / sqrt(d) with e_i that for the small
    elements alone.  Everything else holds them exactly."""
    B = 3
    k, v = _randn(B, Hkv, T + 3, d, seed=11), _randn(B, Hkv, T + 3, d, seed=12)
    k[..., 0] = 0
    cache = _cache_of(k, v, dtype, cdt)
    q = _randn(B, H, T, d, seed=13)
    q[..., 0] = 2.0 ** 12
    q = q.to(dtype)
    lens, mask = [1, 2, 3], torch.zeros(T, T, dtype=torch.bool)
    out, lse = ra.tree_fwd(q.to(DEV), cache, torch.tensor(lens, dtype=torch.int32, device=DEV), mask=mask.to(DEV), out_dtype=F32)
    kk, vv = cu.cache_values(cache)
    ref, ref_lse, mag, big = cu.tree(q, kk, vv, lens, mask, None)
    split = dtype == BF and cdt == E4M3 and H // Hkv * T > 16
    a = q.double().abs()
    top = a.amax(-1, keepdim=True)
    e = torch.where(a < 2.0 ** -13 * top, 2.0 ** -21 * top, torch.zeros_like(top)) if split else torch.zeros_like(a)
    most = kk.abs()[:, :, :3].amax(2).repeat_interleave(H // Hkv, 1).unsqueeze(2)  # of the (at most three) keys, per element
    s_err = (e * most).sum(-1) / d ** 0.5 + 2.0 ** -18 * (1 + big)
    over = (lse.cpu().double() - ref_lse).abs() - s_err - 2.0 ** -22 * ref_lse.abs()
    assert float(over.max()) <= 0, f"lse off by {float(over.max()):.3e} beyond its bound"
    weight_eps = 2.0 ** -8 if dtype == BF else 0.0
    over = (out.cpu().double() - ref).abs() - mag * (weight_eps + 2 * (s_err + 2.0 ** -20)).unsqueeze(-1) - 2.0 ** -23 * ref.abs()
    assert float(over.max()) <= 0, f"out off by {float(over.max()):.3e} beyond its bound"


@pytest.mark.parametrize("dtype,cdt", TYPES)
@pytest.mark.parametrize("H,Hkv,T,d", [r for r in ROWS if r[2] > 1])
def test_queries_of_tokens_that_a_sequence_does_not_have(H, Hkv, T, d, dtype, cdt):
    """Rows behind ntok[b] of a padded batch hold NaN: they come back empty, the others as ever."""
    B, cap = 3, 300 + T
    cache = _cache_of(_randn(B, Hkv, cap, d, seed=31), _randn(B, Hkv, cap, d, seed=32), dtype, cdt)
    q = _randn(B, H, T, d, seed=33).to(dtype).to(DEV)
    lens, ntok = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([300, 17, 0], [1, T - 1, T // 2]))
    ref, ref_lse = ra.tree_fwd(q, cache, lens, ntok=ntok)
    for b in range(B):
        q[b, :, int(ntok[b]):] = float("nan")
    out, lse = ra.tree_fwd(q, cache, lens, ntok=ntok)
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse) and bool(torch.isfinite(out.float()).all())
    for b in range(B):
        assert bool((out[b, :, int(ntok[b]):] == 0).all()) and bool((lse[b, :, int(ntok[b]):] == -float("inf")).all())
