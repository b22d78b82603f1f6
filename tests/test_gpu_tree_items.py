"""The tensor-core kernels of the attention over a cache where a CTA goes from item to item: many short sequences of odd and even
tile counts, ragged tokens, both cache types and head dims, and hidden values in each of many items."""
import pytest
import torch

import cache_util as cu
import sequence_sharded_exact_gb300 as ra

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
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _randn(*shape, seed, dtype=F32):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


def _cache_of(k, v, cdt):
    cache = ra.cache_alloc(*k.shape, cdt)
    ra.cache_write(cache, k.to(BF), v.to(BF))
    return cache


@pytest.mark.parametrize("cdt", [BF, E4M3])
@pytest.mark.parametrize("H,Hkv,T,d", [(4, 2, 10, 128), (4, 2, 10, 64), (4, 2, 64, 64), (4, 2, 64, 128), (4, 2, 66, 64), (4, 2, 66, 128),
                                       (4, 1, 64, 128), (4, 1, 64, 64)])
def test_several_items_per_cta(H, Hkv, T, d, cdt):
    """20, 128, 132 and 256 query rows per kv head; more than three tiles for each of 152 CTAs, in items of one to five tiles."""
    B = 162 if Hkv == 2 else 324
    assert torch.cuda.get_device_properties(0).multi_processor_count * 3 < 3 * B * Hkv
    cap = 4 * 128 + 2 * T
    lens = [(97 * b) % (4 * 128 + T) for b in range(B)]
    ntok = [T - (b % 3) * (T // 3) if b % 11 else b % 2 for b in range(B)]
    k, v, q = _randn(B, Hkv, cap, d, seed=1), _randn(B, Hkv, cap, d, seed=2), _randn(B, H, T, d, seed=3, dtype=BF)
    cache, mask = _cache_of(k, v, cdt), cu.random_tree(B, T, 4)
    got = ra.tree_fwd(q, cache, _i32(lens), mask=mask.to(DEV), ntok=_i32(ntok))
    again = ra.tree_fwd(q, cache, _i32(lens), mask=mask.to(DEV), ntok=_i32(ntok), out_dtype=F32)
    assert torch.equal(again[1], got[1])
    kk, vv = cu.cache_values(cache)
    for b0 in range(0, B, 27):  # every third of each part, in float64
        at = list(range(b0, min(b0 + 27, B)))[::3]
        part = cu.tree(q[at], kk[at], vv[at], [lens[b] for b in at], mask[at], [ntok[b] for b in at])
        cu.check_tree((got[0][at], got[1][at]), part, 2.0 ** -8, BF, f"from sequence {b0}")
        # (weights as two bfloat16 parts, 2^-15 of them apart, and sums of up to 700 terms)
        cu.check_tree((again[0][at], again[1][at]), part, 2.0 ** -15 + 60 * 2.0 ** -23, F32, f"from sequence {b0}, float32")


@pytest.mark.parametrize("cdt", [BF, E4M3])
@pytest.mark.parametrize("H,Hkv,T,d", [(8, 2, 5, 128), (8, 2, 5, 64), (4, 1, 40, 128), (4, 1, 40, 64)])
def test_a_hidden_value_in_each_of_many_items(H, Hkv, T, d, cdt):
    """More than eight items of one tile for each CTA, every one with a value that is not finite in a token that its own
    query alone sees, in a column of its own: no other query, and no other item, has a part of it."""
    B = -(-152 * 10 // Hkv)
    cap = 128
    lens = [(29 * b) % (cap - T + 1) for b in range(B)]
    k, v, q = _randn(B, Hkv, cap, d, seed=11), _randn(B, Hkv, cap, d, seed=12), _randn(B, H, T, d, seed=13, dtype=BF)
    mask = torch.eye(T, dtype=torch.bool)
    clean = _cache_of(k, v, cdt)
    ref, ref_lse = ra.tree_fwd(q, clean, _i32(lens), mask=mask.to(DEV))
    some = list(range(0, B, 41))
    kk, vv = cu.cache_values(clean)
    cu.check_tree((ref[some], ref_lse[some]), cu.tree(q[some], kk[some], vv[some], [lens[b] for b in some], mask, None), 2.0 ** -8, BF)
    every = torch.arange(B, device=DEV)
    token, col = every % T, every * 7 % d
    for only in (1, 2):  # every item, and every second sequence's
        has = every % only == 0
        spoilt = v.clone()
        spoilt[every[has], :, (_i32(lens).long() + token)[has], col[has]] = float("nan")
        out, lse = ra.tree_fwd(q, _cache_of(k, spoilt, cdt), _i32(lens), mask=mask.to(DEV))
        assert torch.equal(lse, ref_lse)
        hit = torch.zeros(B, H, T, d, dtype=torch.bool, device=DEV)
        hit[every[has], :, token[has], col[has]] = True
        assert torch.isnan(out[hit]).all() and torch.equal(out[~hit], ref[~hit])


@pytest.mark.parametrize("cdt", [BF, E4M3])
@pytest.mark.parametrize("H,Hkv,T,d", [(2, 1, 1, 128), (4, 2, 4, 64), (4, 2, 4, 128), (8, 2, 4, 128), (2, 1, 5, 64), (8, 2, 5, 128),
                                       (4, 1, 32, 64), (4, 1, 64, 128), (4, 1, 64, 64)])
@pytest.mark.parametrize("B,n", [(1, 100), (3, 1700)])
def test_float32_output_of_every_kernel(H, Hkv, T, d, B, n, cdt):
    """2, 8, 16, 10, 20, 128 and 256 query rows per kv head, items that one CTA holds whole and items in parts.  (Weights go into
    the product as two bfloat16 parts, 2^-15 of them apart, with up to 16 rows over e4m3 as one float16, 2^-11; the sums of n
    terms are float32's.)  The output in bfloat16 holds one bfloat16 part."""
    cap = n + T
    lens = [n - 611 * b for b in range(B)]
    cache = _cache_of(_randn(B, Hkv, cap, d, seed=21), _randn(B, Hkv, cap, d, seed=22), cdt)
    q, mask = _randn(B, H, T, d, seed=23, dtype=BF), cu.random_tree(B, T, 24)
    out, lse = ra.tree_fwd(q, cache, _i32(lens), mask=mask.to(DEV), out_dtype=F32)
    assert out.dtype == F32
    ref = cu.tree(q, *cu.cache_values(cache), lens, mask, None)
    weight_eps = 2.0 ** -11 if cdt == E4M3 and H // Hkv * T <= 16 else 2.0 ** -15
    cu.check_tree((out, lse), ref, weight_eps + (n / 16 + 16) * 2.0 ** -23, F32)
    rounded, lse2 = ra.tree_fwd(q, cache, _i32(lens), mask=mask.to(DEV))
    cu.check_tree((rounded, lse2), ref, 2.0 ** -8, BF)
    assert torch.equal(lse, lse2)
