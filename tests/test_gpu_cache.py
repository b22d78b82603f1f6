"""The key/value cache: what is written is the definition's quantisation bit for bit, reading back is exact, and
nothing else in the cache changes."""
import pytest
import torch

import cache_util as cu
import sequence_sharded_exact_gb300 as ra
from sequence_sharded_exact_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E4M3 = torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def _clean_status():
    torch.cuda.set_device(0)
    ra.device_status()
    yield
    assert ra.device_status() == 0


def _rows(B, Hkv, T, d, dtype, seed, fused=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((B, T, 2 * Hkv + 3, d), generator=g) * 2.0 ** torch.randint(-20, 20, (B, T, 2 * Hkv + 3, 1), generator=g)
    x = x.to(dtype).to(DEV)
    k, v = x[:, :, :Hkv].transpose(1, 2), x[:, :, Hkv:2 * Hkv].transpose(1, 2)
    return (k, v) if fused else (k.contiguous(), v.contiguous())


def _stale(B, Hkv, cap, d, dtype, seed=99):
    """A cache whose every byte holds something."""
    c = ra.cache_alloc(B, Hkv, cap, d, dtype)
    g = torch.Generator().manual_seed(seed)
    for t in c:
        if t is not None:
            t.view(torch.uint8).copy_(torch.randint(0, 256, t.view(torch.uint8).shape, generator=g, dtype=torch.uint8))
    return c


def _same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


CASES = [
    # B, Hkv, T, d, cap, lens, ntok, dtype, cache dtype, fused
    (1, 1, 1, 64, 1, [0], None, torch.float32, E4M3, False),
    (3, 2, 5, 128, 77, [0, 72, 31], [5, 0, 3], torch.bfloat16, E4M3, True),
    (2, 8, 300, 128, 300, None, None, torch.bfloat16, E4M3, False),
    (2, 3, 33, 64, 100, [67, 1], [33, 32], torch.float32, E4M3, True),
    (3, 2, 5, 128, 77, [0, 72, 31], [5, 0, 3], torch.bfloat16, torch.bfloat16, True),
    (2, 3, 33, 64, 100, [67, 1], None, torch.float32, torch.float32, False),
]


@pytest.mark.parametrize("B,Hkv,T,d,cap,lens,ntok,dtype,cdt,fused", CASES)
def test_write_and_read_back(B, Hkv, T, d, cap, lens, ntok, dtype, cdt, fused):
    k, v = _rows(B, Hkv, T, d, dtype, seed=T + d, fused=fused)
    cache = _stale(B, Hkv, cap, d, cdt)
    before = [None if t is None else t.clone() for t in cache]
    i32 = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    assert ra.cache_write(cache, k, v, i32(lens), ntok=i32(ntok)) is cache
    torch.cuda.synchronize()
    written = torch.zeros((B, cap), dtype=torch.bool)
    for b in range(B):
        n0 = 0 if lens is None else lens[b]
        n = T if ntok is None else ntok[b]
        written[b, n0:n0 + n] = True
        for x, values, exps in ((k, cache.k, cache.k_exp), (v, cache.v, cache.v_exp)):
            got = values[b, :, n0:n0 + n]
            if cdt != E4M3:
                assert _same(got, x[b, :, :n])
                continue
            ref, e = cu.quantised(x[b, :, :n].cpu().double())
            assert torch.equal(exps[b, :, n0:n0 + n].cpu().double() - 127, e)
            assert torch.equal(got.float().cpu().double(), ref)
    keep = ~written.to(DEV)
    for t, old in zip(cache, before):
        if t is not None:
            assert _same(t.transpose(0, 1)[:, keep].view(torch.uint8), old.transpose(0, 1)[:, keep].view(torch.uint8))
    # reading back: the values it stands for, rounded once
    for n0, rows in ((0, cap), (cap // 3, cap - cap // 3), (cap - 1, 1), (0, 0)):
        rk, rv = ra.cache_read(cache, rows, row0=n0, dtype=dtype)
        for got, values, exps in ((rk, cache.k, cache.k_exp), (rv, cache.v, cache.v_exp)):
            if cdt != E4M3:
                assert _same(got, values[:, :, n0:n0 + rows])
                continue
            x = values[:, :, n0:n0 + rows].float().cpu().double()
            e = exps[:, :, n0:n0 + rows].cpu().double()
            ref = (x * 2.0 ** (e - 127).unsqueeze(-1)).float().to(dtype)
            ok = (e > 0) & (e < 248)  # bytes that a write leaves
            assert torch.equal(got.cpu().double().nan_to_num(7e77)[ok], ref.double().nan_to_num(7e77)[ok])


def test_values_at_the_edges_of_the_format():
    """Zero rows, 448 and its neighbours, ties, subnormals of e4m3 and of float32, infinities, NaN."""
    d = 64
    x = torch.zeros((1, 1, 10, d))
    x[0, 0, 1, :4] = torch.tensor([448.0, -448.0, 447.9, 2.0 ** -10])
    x[0, 0, 2, :3] = torch.tensor([448.0001, 224.0, 1.0])
    x[0, 0, 3, :5] = torch.tensor([256.0, 17.0, 19.0, 2.0 ** -9, 3 * 2.0 ** -10])  # 17 and 19 lie between e4m3 neighbours
    x[0, 0, 4, :2] = torch.tensor([1e-40, -1e-45])
    x[0, 0, 5, :2] = torch.tensor([3.0e38, 1.0])
    x[0, 0, 6, :3] = torch.tensor([float("inf"), -float("inf"), 1e30])
    x[0, 0, 7, :3] = torch.tensor([float("nan"), 2.0, -0.0])
    x[0, 0, 8, :2] = torch.tensor([2.0 ** -126, 2.0 ** -130])
    x[0, 0, 9, :2] = torch.tensor([torch.finfo(torch.float32).max, 1.0])
    x = x.to(DEV)
    cache = ra.cache_alloc(1, 1, 10, d)
    ra.cache_write(cache, x, x)
    k, v = ra.cache_read(cache, 10, dtype=torch.float32)
    assert _same(k, v)
    k, e = k[0, 0].cpu(), cache.k_exp[0, 0].cpu().int() - 127
    assert e.tolist() == [-126, 0, 1, 0, -126, 120, 120, -7, -126, 120]
    assert k[0].abs().max() == 0
    assert k[1, :4].tolist() == [448.0, -448.0, 448.0, 0.0]
    assert k[2, :3].tolist() == [448.0, 224.0, 1.0]
    assert k[3, :5].tolist() == [256.0, 16.0, 20.0, 2.0 ** -9, 2 * 2.0 ** -9]
    assert k[4, 0] == 2.0 ** -133 and k[4, 1:].abs().max() == 0  # subnormal float32 rows: steps of 2^-135
    assert k[6, 0] == float("inf") and k[6, 1] == -float("inf") and torch.isfinite(k[6, 2:]).all()
    assert abs(float(k[5, 0]) / 3e38 - 1) <= 2.0 ** -4
    assert torch.isnan(k[7, 0]) and k[7, 1] == 2.0 and torch.isfinite(k[7, 1:]).all()
    assert k[8, 0] == 2.0 ** -126 and k[9, 0] == float("inf")


def test_rows_outside_the_cache_are_left_out_and_reported():
    cache = _stale(2, 1, 20, 64, E4M3)
    before = [t.clone() for t in cache]
    k, v = _rows(2, 1, 4, 64, torch.bfloat16, seed=1)
    lens = torch.tensor([18, -2], dtype=torch.int32, device=DEV)
    ra.cache_write(cache, k, v, lens)
    assert ra.device_status() == binding.RA_DEVICE_RANGE
    ref, e = cu.quantised(k[0, :, :2].cpu().double())
    assert torch.equal(cache.k[0, :, 18:].float().cpu().double(), ref)
    assert _same(cache.k[0, :, :18], before[0][0, :, :18])
    assert _same(cache.k[1], before[0][1]) and _same(cache.v_exp[1], before[3][1])  # rows below zero: none of them, nor the others
    ra.cache_write(cache, k, v, torch.tensor([0, 0], dtype=torch.int32, device=DEV),
                   ntok=torch.tensor([5, -1], dtype=torch.int32, device=DEV))
    with pytest.raises(ra.RingAttnError) as err:
        ra.device_check()
    assert err.value.status == binding.RA_ERR_INVALID_ARG


def test_written_in_a_replayed_graph():
    cache = ra.cache_alloc(2, 2, 64, 128)
    k, v = _rows(2, 2, 3, 128, torch.bfloat16, seed=5)
    lens = torch.tensor([0, 10], dtype=torch.int32, device=DEV)
    ra.cache_write(cache, k, v, lens)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ra.cache_write(cache, k, v, lens)
        rk, rv = ra.cache_read(cache, 64)
    lens.copy_(torch.tensor([40, 61]))
    graph.replay()
    torch.cuda.synchronize()
    other = ra.cache_alloc(2, 2, 64, 128)
    for at in ([0, 10], [40, 61]):
        ra.cache_write(other, k, v, torch.tensor(at, dtype=torch.int32, device=DEV))
    assert all(_same(a, b) for a, b in zip(cache, other))
    assert all(_same(a, b) for a, b in zip((rk, rv), ra.cache_read(other, 64)))
