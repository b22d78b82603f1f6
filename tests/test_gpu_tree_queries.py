"""Queries of the attention over a cache that ask much of their form in the products: not finite in a row that sees
nothing."""
import pytest
import torch

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
