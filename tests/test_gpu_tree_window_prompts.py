"""Prompts that go in by chunks through a window with sinks: every row is what it is in the whole sequence, wherever the chunks
are cut, also where the first tokens lie in the step itself and the step is longer than the window."""
import math

import pytest
import torch

import cache_util as cu
import sequence_sharded_exact_gb300 as ra
import window_util as wu

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
TYPES = [(F32, F32), (F32, E4M3), (BF, BF), (BF, E4M3)]
WEIGHT_EPS = {BF: 2.0 ** -8, F32: 0.0}


@pytest.fixture(autouse=True)
def _clean_status():
    torch.cuda.set_device(0)
    ra.device_status()
    yield
    assert ra.device_status() == 0


def _i32(x):
    return torch.as_tensor(x, dtype=torch.int32).to(DEV)


def _randn(*shape, seed, dtype=F32):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


def _step_mask(lens, T, W, S):
    """[B, T, T]: token t, at lens[b] + t, sees the step's token j <= t within the window or among the first S tokens."""
    t, j = torch.arange(T)[:, None], torch.arange(T)[None, :]
    return torch.stack([(j <= t) & ((t - j < W) | (n + j < S)) for n in lens])


# (query heads of 2 kv heads, chunks): 1 to 16 query rows per kv head, up to 128 and beyond, so that every kernel takes some
CHUNKS = [(8, (1, 7, 64, 300)), (2, (3, 1, 5, 2, 8, 12, 16, 200)), (4, (300, 5, 1)), (8, (2, 2, 2, 9, 33, 150, 1))]


@pytest.mark.parametrize("dtype,cdt", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("W,S", [(16, 4), (3, 20), (1, 1), (130, 140), (40, 0)])
@pytest.mark.parametrize("H,chunks", CHUNKS)
def test_chunks_are_the_whole_sequence(H, chunks, W, S, d, dtype, cdt):
    Hkv, L = 2, sum(chunks)
    q, k, v = (_randn(1, h, L, d, seed=L + i, dtype=dtype) for i, h in enumerate((H, Hkv, Hkv)))
    cache = ra.cache_alloc(1, Hkv, L, d, cdt)
    got, at = [], 0
    for T in chunks:
        lens = _i32([at])
        ra.cache_write(cache, k[:, :, at:at + T], v[:, :, at:at + T], lens)
        got.append(ra.tree_fwd(q[:, :, at:at + T].contiguous(), cache, lens, window=W, sinks=S))
        at += T
    kc, vc = cu.cache_values(cache)
    ref = wu.fwd(q, kc, vc, 1, "contiguous", W, S, True)
    at = 0
    for T, x in zip(chunks, got):
        cu.check_tree(x, [r[:, :, at:at + T] for r in ref], WEIGHT_EPS[dtype], dtype, f"rows {at} to {at + T}")
        at += T


@pytest.mark.parametrize("dtype,cdt", TYPES)
@pytest.mark.parametrize("B,H,Hkv,T,d,cap,lens,ntok,W,S", [
    (5, 2, 2, 3, 64, 129, [126, 125, 0, 64, 1], None, 2, 1),
    (3, 8, 2, 4, 128, 300, [0, 1, 200], [4, 3, 2], 1, 3),
    (4, 16, 2, 5, 64, 300, [0, 2, 6, 100], [5, 5, 4, 0], 2, 6),
    (2, 8, 1, 40, 128, 400, [0, 5], [40, 33], 7, 30),
    (6, 2, 2, 9, 128, 200, [0, 1, 2, 3, 4, 90], None, 3, 4),
    (2, 4, 1, 200, 64, 500, [10, 130], [200, 199], 20, 160),   # sinks behind a tile's border in the step
    (2, 4, 1, 200, 64, 500, [10, 130], None, 20, 2 ** 31 - 1),
    (2, 4, 1, 200, 64, 500, [0, 130], None, 2 ** 31 - 1, 2 ** 31 - 1),
])
def test_first_tokens_inside_the_step(B, H, Hkv, T, d, cap, lens, ntok, W, S, dtype, cdt):
    """Batches whose sequences have none, some or all of the first tokens in the step; and the same step with its mask spelled out."""
    cache = ra.cache_alloc(B, Hkv, cap, d, cdt)
    ra.cache_write(cache, _randn(B, Hkv, cap, d, seed=1, dtype=dtype), _randn(B, Hkv, cap, d, seed=2, dtype=dtype))
    q = _randn(B, H, T, d, seed=3, dtype=dtype)
    nt = None if ntok is None else _i32(ntok)
    got = ra.tree_fwd(q, cache, _i32(lens), ntok=nt, window=W, sinks=S)
    mask = _step_mask(lens, T, W, S)
    k, v = cu.cache_values(cache)
    ref = wu.tree(q, k, v, lens, mask, ntok, W, S, None)
    cu.check_tree(got, ref, WEIGHT_EPS[dtype], dtype)
    masked = ra.tree_fwd(q, cache, _i32(lens), mask=mask.to(DEV), ntok=nt, window=W, sinks=S)
    cu.check_tree(masked, ref, WEIGHT_EPS[dtype], dtype, "with a mask")


@pytest.mark.parametrize("dtype,cdt", TYPES)
@pytest.mark.parametrize("R", [1, 2, 8])
@pytest.mark.parametrize("T", [7, 40])
def test_values_that_are_not_finite_inside_the_step(T, R, dtype, cdt):
    """A first token of the step reaches all later ones; another of its tokens those within the window, and nobody else."""
    Hkv, d, n, W, S = 2, 64, 2, 4, 5
    k, v = _randn(1, Hkv, n + T, d, seed=1, dtype=dtype), _randn(1, Hkv, n + T, d, seed=2, dtype=dtype)
    q = _randn(1, Hkv * R, T, d, seed=3, dtype=dtype)
    cache = ra.cache_alloc(1, Hkv, n + T, d, cdt)
    ra.cache_write(cache, k, v)
    out, lse = ra.tree_fwd(q, cache, _i32([n]), window=W, sinks=S)
    for row, seen in ((3, range(1, T)), (n + 3, range(3, min(T, 3 + W)))):
        k2, v2 = k.clone(), v.clone()
        k2[:, :, row, 7] = math.nan
        v2[:, :, row, 5] = math.inf
        ra.cache_write(cache, k2, v2)
        o2, l2 = ra.tree_fwd(q, cache, _i32([n]), window=W, sinks=S)
        sees = torch.tensor([t in seen for t in range(T)])
        assert not bool(torch.isfinite(o2[:, :, sees]).any()), row
        assert torch.equal(o2[:, :, ~sees], out[:, :, ~sees]) and torch.equal(l2[:, :, ~sees], lse[:, :, ~sees]), row
