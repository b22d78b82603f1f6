"""Attention over an e4m3 cache whose rows of v have one element far above the others, which takes the row's scale up: the other
columns are the other rows' and keep their precision."""
import pytest
import torch

import cache_util as cu
import sequence_sharded_exact_gb300 as ra

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
# H, Hkv, T, d: 1, 4, 8, 8, 16, 10, 20, 128 and 256 query rows per kv head
ROWS = [(2, 2, 1, 128), (8, 2, 1, 64), (8, 1, 1, 128), (4, 2, 4, 64), (8, 2, 4, 128), (2, 1, 5, 64), (8, 2, 5, 128), (4, 1, 32, 64), (4, 1, 64, 128)]


@pytest.fixture(autouse=True)
def _clean_status():
    torch.cuda.set_device(0)
    ra.device_status()
    yield
    assert ra.device_status() == 0


def _randn(*shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed))


def _run(q, k, v, lens, mask=None):
    cache = ra.cache_alloc(*k.shape, E4M3)
    ra.cache_write(cache, k.to(q.dtype).to(DEV), v.to(q.dtype).to(DEV))
    got = ra.tree_fwd(q.to(DEV), cache, torch.tensor(lens, dtype=torch.int32, device=DEV), mask=None if mask is None else mask.to(DEV), out_dtype=F32)
    # weights are rounded to bfloat16, or to a float16 that is finer, for the product: every column on its own
    cu.check_tree(got, cu.tree(q, *cu.cache_values(cache), lens, mask, None), 2.0 ** -8 if q.dtype == BF else 0.0, F32)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("H,Hkv,T,d", ROWS)
@pytest.mark.parametrize("up", [12, 24, 40, 90])
@pytest.mark.parametrize("at", [(0,), (37,), (130,), (419,), (5, 37, 300)])
def test_one_element_of_a_row_far_above_the_others(H, Hkv, T, d, up, at, dtype):
    B, n = 2, 420
    cap = n + T
    k, v, q = _randn(B, Hkv, cap, d, seed=1), _randn(B, Hkv, cap, d, seed=2), _randn(B, H, T, d, seed=3).to(dtype)
    for i, row in enumerate(at):
        v[:, :, row, (7 * i + 3) % d] = 2.0 ** (up - 10 * i)
    _run(q, k, v, [n, 333])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("H,Hkv,T,d", ROWS)
def test_scales_of_every_size_in_different_columns(H, Hkv, T, d, dtype):
    """Rows of zeros but for one element, of 2^-30 to 2^30, each column with one size: every column is as exact as any other."""
    B, n = 1, 600
    cap = n + T
    k, q = _randn(B, Hkv, cap, d, seed=11), _randn(B, H, T, d, seed=13).to(dtype)
    col = torch.arange(cap) % d
    size = torch.linspace(-30, 30, d).round()[col]
    v = torch.zeros(B, Hkv, cap, d)
    v[:, :, torch.arange(cap), col] = _randn(B, Hkv, cap, seed=12).abs().clamp(0.1, 3.9) * 2.0 ** size
    _run(q, k, v, [n])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("H,Hkv,T,d", ROWS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_beside_hidden_values_and_rows_of_zeros(H, Hkv, T, d, bad, dtype):
    """Such a row among the drafted tokens, whose own query sees it; one with a value that is not finite, that nobody sees;
    rows of zeros and rows behind the sequence."""
    B, n = 2, 140
    cap = n + T + 20
    k, v, q = _randn(B, Hkv, cap, d, seed=21), _randn(B, Hkv, cap, d, seed=22), _randn(B, H, T, d, seed=23).to(dtype)
    v[:, :, 60:90] = 0
    v[:, :, 10, 1] = 2.0 ** 35
    mask = torch.eye(T, dtype=torch.bool)
    lens = [n, 77]
    for b in range(B):
        v[b, :, lens[b], 2] = 2.0 ** 38
        if T > 1:
            mask[1] = False
            mask[1, 0] = True
            v[b, :, lens[b] + 1, 3] = bad
        v[b, :, lens[b] + T:] = bad
    cache = ra.cache_alloc(B, Hkv, cap, d, E4M3)
    ra.cache_write(cache, k.to(dtype).to(DEV), v.to(dtype).to(DEV))
    got = ra.tree_fwd(q.to(DEV), cache, torch.tensor(lens, dtype=torch.int32, device=DEV), mask=mask.to(DEV), out_dtype=F32)
    kk, vv = cu.cache_values(cache)
    cu.check_tree(got, cu.tree(q, kk, vv, lens, mask, None), 2.0 ** -8 if dtype == BF else 0.0, F32)
