"""The cache's writes and reads at sizes where a block takes several turns: many rows, and more heads than a grid has."""
import pytest
import torch

import cache_util as cu
import sequence_sharded_exact_gb300 as ra
from test_gpu_cache import _same, _stale

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def _clean_status():
    torch.cuda.set_device(0)
    ra.device_status()
    yield
    assert ra.device_status() == 0


@pytest.mark.parametrize("dtype,cdt", [(BF, E4M3), (F32, E4M3), (BF, BF), (F32, F32)])
@pytest.mark.parametrize("B,Hkv,T,d,cap,start", [
    (1, 8, 12013, 128, 12100, 41),  # two and a half turns of the grid's 76 blocks of 64 rows per head
    (1, 8, 24013, 64, 24100, 3),    # and of 128 rows
    (66000, 1, 1, 64, 2, 1),        # more heads than a grid's second axis
    (1100, 60, 2, 64, 3, 0),
])
def test_several_turns(B, Hkv, T, d, cap, start, dtype, cdt):
    g = torch.Generator().manual_seed(T + d)
    k, v = ((torch.randn((B, Hkv, T, d), generator=g) * 2.0 ** torch.randint(-20, 20, (B, Hkv, T, 1), generator=g)).to(dtype).to(DEV)
            for _ in range(2))
    cache = _stale(B, Hkv, cap, d, cdt)
    before = [None if t is None else t.clone() for t in cache]
    ra.cache_write(cache, k, v, torch.full((B,), start, dtype=torch.int32, device=DEV))
    for t, old in zip(cache, before):
        if t is not None:
            assert _same(t[:, :, :start], old[:, :, :start]) and _same(t[:, :, start + T:], old[:, :, start + T:])
    for x, values, exps in ((k, cache.k, cache.k_exp), (v, cache.v, cache.v_exp)):
        got = values[:, :, start:start + T]
        if cdt != E4M3:
            assert _same(got, x)
            continue
        ref, e = cu.quantised(x.cpu().double())
        assert torch.equal(exps[:, :, start:start + T].cpu().double() - 127, e)
        assert torch.equal(got.float().cpu().double(), ref)
    rk, rv = ra.cache_read(cache, T, row0=start, dtype=dtype)
    for got, values, exps in ((rk, cache.k, cache.k_exp), (rv, cache.v, cache.v_exp)):
        if cdt != E4M3:
            assert _same(got, values[:, :, start:start + T])
            continue
        ref = values[:, :, start:start + T].float().cpu().double() * 2.0 ** (exps[:, :, start:start + T].cpu().double() - 127).unsqueeze(-1)
        assert torch.equal(got.cpu().double(), ref.float().to(dtype).double())
