"""Attention of new tokens over a cache through a window with sinks, against float64: windows and sinks around the tiles'
borders, trees with positions and chains, ragged batches, every cache type, both head dims."""
import math

import pytest
import torch

import cache_util as cu
import sequence_sharded_exact_gb300 as ra
import window_util as wu
from sequence_sharded_exact_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
TYPES = [(F32, F32), (F32, E4M3), (BF, BF), (BF, E4M3)]


@pytest.fixture(autouse=True)
def _clean_status():
    torch.cuda.set_device(0)
    ra.device_status()
    yield
    assert ra.device_status() == 0


def _i32(x):
    return None if x is None else torch.as_tensor(x, dtype=torch.int32).to(DEV)


def _randn(*shape, seed, dtype=F32):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


def _cache(B, Hkv, cap, d, dtype, cdt, seed):
    cache = ra.cache_alloc(B, Hkv, cap, d, cdt)
    k, v = _randn(B, Hkv, cap, d, seed=seed), _randn(B, Hkv, cap, d, seed=seed + 1)
    if cdt == E4M3:
        v *= 2.0 ** torch.randint(-6, 6, (B, Hkv, cap, 1), generator=torch.Generator().manual_seed(seed + 2)).to(DEV)
    ra.cache_write(cache, k.to(dtype), v.to(dtype))
    return cache


def _depths(mask):
    """The depth of each token of a tree of ancestors' masks."""
    return (mask.sum(-1) - 1).to(torch.int32)


def _check(q, cache, lens, window, sinks, mask=None, ntok=None, positions=None, out_dtype=None, what=""):
    got = ra.tree_fwd(q, cache, _i32(lens), mask=None if mask is None else mask.to(DEV), ntok=_i32(ntok), out_dtype=out_dtype,
                      window=window, sinks=sinks, positions=_i32(positions))
    k, v = cu.cache_values(cache)
    ref = wu.tree(q, k, v, lens, mask, ntok, window, sinks, positions)
    cu.check_tree(got, ref, 2.0 ** -8 if q.dtype == BF else 0.0, got[0].dtype, what)
    return got


CASES = [
    # B, H, Hkv, T, d, cap, lens, ntok, tree, window, sinks
    (1, 1, 1, 1, 64, 1, [0], None, False, 1, 0),
    (1, 4, 1, 1, 128, 400, [399], None, False, 1, 0),                # the token alone
    (1, 4, 2, 1, 128, 400, [399], None, False, 1, 3),
    (1, 8, 2, 1, 64, 900, [899], None, False, 128, 4),
    (1, 8, 2, 1, 128, 900, [896], None, False, 129, 128),            # sinks of a whole tile
    (2, 8, 2, 5, 64, 640, [500, 0], [5, 3], True, 60, 4),            # ragged, an empty prefix
    (3, 8, 8, 7, 128, 300, [1, 127, 250], [7, 1, 0], True, 9, 2),    # a sequence without tokens
    (1, 32, 8, 4, 128, 3000, [2900], None, True, 700, 130),          # 16 query rows
    (4, 8, 1, 9, 128, 1000, [0, 5, 640, 991], None, True, 300, 4),   # 72 rows, the last row of the cache
    (1, 16, 2, 33, 64, 700, [513], [31], True, 40, 1),               # 264 rows
    (2, 6, 3, 1, 128, 4500, [4321, 17], None, False, 1000, 50),
    (5, 2, 2, 3, 64, 129, [126, 125, 0, 64, 1], None, False, 2, 1),  # a window shorter than the step's tokens
    (1, 4, 2, 40, 128, 600, [512], None, False, 7, 0),
    (37, 4, 4, 2, 64, 340, [(37 * b) % 330 for b in range(37)], [b % 3 for b in range(37)], True, 100, 5),
    (2, 64, 8, 17, 128, 800, [700, 383], None, True, 200, 300),      # sinks that run into the window
    (1, 4, 1, 2, 128, 800, [700], None, False, 100000, 4),           # everything
    (1, 4, 1, 2, 64, 800, [700], None, False, 10, 100000),
    (64, 8, 2, 1, 128, 300, [4 * b for b in range(64)], None, False, 50, 4),  # many short items
]


@pytest.mark.parametrize("dtype,cdt", TYPES)
@pytest.mark.parametrize("B,H,Hkv,T,d,cap,lens,ntok,tree,window,sinks", CASES)
def test_against_float64(B, H, Hkv, T, d, cap, lens, ntok, tree, window, sinks, dtype, cdt):
    cache = _cache(B, Hkv, cap, d, dtype, cdt, seed=cap + T)
    q = _randn(B, H, T, d, seed=T, dtype=dtype)
    mask = cu.random_tree(B, T, cap) if tree else None
    pos = None if mask is None else torch.tensor(lens)[:, None] + _depths(mask)
    _check(q, cache, lens, window, sinks, mask, ntok, pos)


@pytest.mark.parametrize("dtype,cdt", TYPES)
@pytest.mark.parametrize("B,H,Hkv,T,d,cap,lens,window,sinks", [
    (1, 16, 4, 8, 128, 20000, [19000], 9000, 4),     # several tiles per CTA
    (1, 2, 1, 3, 64, 60000, [59001], 30000, 200),
    (1, 32, 1, 5, 128, 30000, [29995], 15000, 4),    # two query tiles
    (40, 4, 4, 2, 128, 900, [801 + b for b in range(40)], 600, 3),  # several items per CTA
])
def test_several_tiles_and_items_per_cta(B, H, Hkv, T, d, cap, lens, window, sinks, dtype, cdt):
    cache = _cache(B, Hkv, cap, d, dtype, cdt, seed=cap)
    q = _randn(B, H, T, d, seed=T, dtype=dtype)
    first = _check(q, cache, lens, window, sinks)
    for _ in range(10):
        again = ra.tree_fwd(q, cache, _i32(lens), window=window, sinks=sinks)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("dtype,cdt", TYPES)
def test_positions(dtype, cdt):
    """Masks without positions, positions outside their range, one mask for all sequences, float32 output."""
    B, H, Hkv, T, d, cap, lens = 2, 8, 2, 6, 128, 500, [300, 444]
    cache = _cache(B, Hkv, cap, d, dtype, cdt, seed=4)
    q = _randn(B, H, T, d, seed=1, dtype=dtype)
    mask = cu.random_tree(B, T, 9)
    _check(q, cache, lens, 20, 2, mask)
    wild = torch.tensor([[0, -5, 301, 400, 2 ** 31 - 1, 303], [-2 ** 31, 444, 449, 450, 445, 0]])
    _check(q, cache, lens, 20, 2, mask, positions=wild)
    _check(q, cache, lens, 3, 1, mask, positions=wild, out_dtype=F32)
    _check(q, cache, lens, 50, 0, mask[0], ntok=[4, 6])


@pytest.mark.parametrize("dtype,cdt", TYPES)
@pytest.mark.parametrize("R", [1, 3, 12, 40])
def test_what_is_hidden_has_no_part(R, dtype, cdt):
    """Rows between the sinks and the window, rows that some of the step's tokens see and others do not, and rows behind the
    sequence, with NaN and infinities in them."""
    B, Hkv, T, d, cap, n, W, S = 1, 2, 5, 64, 700, 600, 139, 130
    H = Hkv * R
    cache = _cache(B, Hkv, cap, d, dtype, cdt, seed=R)
    q = _randn(B, H, T, d, seed=2, dtype=dtype)
    out, lse = _check(q, cache, [n], W, S)
    lo = n - W + 1  # token t sees the prefix from lo + t on
    bad = torch.tensor([math.nan, math.inf, -math.inf], device=DEV)

    def spoil(rows):
        c = ra.KVCache(*(None if x is None else x.clone() for x in cache))
        for i, j in enumerate(rows):
            x = _randn(B, Hkv, 1, d, seed=j).to(dtype)
            x[..., i % d] = bad[i % 3]
            ra.cache_write(c, x, x, lens=_i32([j]))
        return c

    o2, l2 = ra.tree_fwd(q, spoil([S, S + 1, 200, 300, 383, 384, lo - 2, lo - 1, n + T, n + T + 1]), _i32([n]), window=W, sinks=S)
    assert torch.equal(o2, out) and torch.equal(l2, lse)
    for t in range(1, T):  # token t and later ones do not see row lo + t - 1, the ones before do
        o2, l2 = ra.tree_fwd(q, spoil([lo + t - 1]), _i32([n]), window=W, sinks=S)
        assert torch.equal(o2[:, :, t:], out[:, :, t:]) and torch.equal(l2[:, :, t:], lse[:, :, t:]), t
        assert not bool(torch.isfinite(o2[:, :, :t, 0]).any()), t
    for j in (0, S - 1):  # sinks reach every token
        o2, _ = ra.tree_fwd(q, spoil([j]), _i32([n]), window=W, sinks=S)
        assert not bool(torch.isfinite(o2[..., 0]).any()), j


@pytest.mark.parametrize("dtype,cdt", TYPES)
def test_values_alone_that_are_not_finite(dtype, cdt):
    """Only v is spoilt: who sees the row has the value, in its column alone."""
    B, H, Hkv, T, d, cap, n, W, S = 1, 8, 2, 6, 128, 400, 300, 100, 2
    cache = _cache(B, Hkv, cap, d, dtype, cdt, seed=8)
    q = _randn(B, H, T, d, seed=2, dtype=dtype)
    out, lse = ra.tree_fwd(q, cache, _i32([n]), window=W, sinks=S)
    t = 3
    c = ra.KVCache(*(None if x is None else x.clone() for x in cache))
    k, v = ra.cache_read(c, 1, row0=n - W + t, dtype=dtype)
    v[..., 9] = math.nan
    ra.cache_write(c, k, v, lens=_i32([n - W + t]))
    o2, l2 = ra.tree_fwd(q, c, _i32([n]), window=W, sinks=S)
    keep = [x for x in range(d) if x != 9]
    assert torch.equal(o2[:, :, t:], out[:, :, t:]) and bool(torch.isnan(o2[:, :, :t, 9]).all())
    if cdt != E4M3:  # (a quantised row's other elements do not change either, but its scale may)
        assert torch.allclose(o2[:, :, :t][..., keep].float(), out[:, :, :t][..., keep].float(), rtol=2.0 ** -7, atol=2.0 ** -9)


@pytest.mark.parametrize("dtype,cdt", TYPES)
@pytest.mark.parametrize("T", [1, 4, 40])
def test_a_window_of_everything_is_no_window(T, dtype, cdt):
    B, H, Hkv, d, cap, lens = 3, 8, 2, 128, 900, [850, 3, 400]
    cache = _cache(B, Hkv, cap, d, dtype, cdt, seed=T)
    q = _randn(B, H, T, d, seed=2, dtype=dtype)
    mask = cu.random_tree(B, T, 5).to(DEV)
    for kw in (dict(), dict(mask=mask)):
        a = ra.tree_fwd(q, cache, _i32(lens), **kw)
        b = ra.tree_fwd(q, cache, _i32(lens), window=2 ** 31 - 1, **kw)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("dtype,cdt", [(F32, F32), (BF, BF), (BF, E4M3)])
@pytest.mark.parametrize("T", [1, 16])
def test_a_replayed_graph_takes_new_lengths(T, dtype, cdt):
    B, H, Hkv, d, cap, W, S = 3, 8, 2, 64, 1200, 150, 4
    cache = _cache(B, Hkv, cap, d, dtype, cdt, seed=T)
    q = _randn(B, H, T, d, seed=2, dtype=dtype)
    lens = _i32([0, 0, 0])
    ra.tree_fwd(q, cache, lens, window=W, sinks=S)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = ra.tree_fwd(q, cache, lens, window=W, sinks=S)
    k, v = cu.cache_values(cache)
    for now in ([1100, 3, 500], [150, 149, 151], [0, 1184, 777]):
        lens.copy_(_i32(now))
        g.replay()
        torch.cuda.synchronize()
        cu.check_tree((out, lse), wu.tree(q, k, v, now, None, None, W, S, None), 2.0 ** -8 if dtype == BF else 0.0, dtype, str(now))


def test_lengths_outside_their_range():
    B, H, Hkv, T, d, cap = 3, 4, 2, 4, 64, 200
    cache = _cache(B, Hkv, cap, d, BF, BF, seed=1)
    q = _randn(B, H, T, d, seed=2, dtype=BF)
    got = ra.tree_fwd(q, cache, _i32([500, -3, 198]), window=30, sinks=2)
    assert ra.device_status() == binding.RA_DEVICE_RANGE
    ref = ra.tree_fwd(q, cache, _i32([200, 0, 198]), ntok=_i32([0, 4, 2]), window=30, sinks=2)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_refusals_and_the_python_form():
    B, H, Hkv, T, d, cap = 2, 8, 2, 4, 64, 200
    cache = _cache(B, Hkv, cap, d, BF, BF, seed=1)
    q, lens = _randn(B, H, T, d, seed=2, dtype=BF), _i32([100, 50])
    mask, pos = cu.random_tree(B, T, 1).to(DEV), _i32([[100] * T, [51] * T])
    s = torch.cuda.current_stream()
    for kw in (dict(window=9), dict(window=9, sinks=3), dict(window=9, sinks=3, mask=mask), dict(window=9, mask=mask, positions=pos)):
        assert all(torch.equal(a, b) for a, b in zip(ra.tree_fwd(q, cache, lens, **kw), ra.tree_fwd(q, cache, lens, stream=s, **kw)))
    for err, kw in [(ValueError, dict(sinks=3)), (ValueError, dict(positions=pos, mask=mask)), (binding.RingAttnError, dict(window=0)),
                    (binding.RingAttnError, dict(window=5, sinks=-1)), (binding.RingAttnError, dict(window=5, positions=pos)),
                    (ValueError, dict(window=5, mask=mask, positions=pos.long())), (TypeError, dict(window=5.0)), (ValueError, dict(window=2 ** 31))]:
        for stream in (None, s):
            with pytest.raises(err):
                ra.tree_fwd(q, cache, lens, stream=stream, **kw)


@pytest.mark.parametrize("cdt", [BF, E4M3])
def test_a_run_of_steps(cdt):
    """Serving through a window: a prompt through window_fwd, its keys and values written to the cache, then tokens one by
    one, and a step of several, over it.  Every step's rows against the same rows of the whole sequence's window_fwd."""
    B, H, Hkv, d, W, S, prompt, steps = 1, 8, 2, 128, 70, 4, 200, 9
    L = prompt + steps
    pos = torch.arange(L, dtype=torch.int32, device=DEV)
    grid = torch.stack((pos, pos // 3, pos % 7))[:, None].contiguous()
    qkv = _randn(B, L, H + 2 * Hkv, d, seed=3, dtype=BF)
    q, k, v = (t.transpose(1, 2) for t in qkv.split([H, Hkv, Hkv], dim=2))
    wq, wk = (1 + 0.1 * _randn(d, seed=i) for i in (5, 6))
    q, k = ra.qk_rope_axes(q, k, grid, (16, 24, 24), wq, wk)
    cache = ra.cache_alloc(B, Hkv, L, d, cdt)
    ra.cache_write(cache, k, v)
    kc, vc = ra.cache_read(cache, L, dtype=BF)  # what the cache stands for
    whole, wl = ra.window_fwd(q, kc, vc, 1, W, S, True, "contiguous")
    cache2 = ra.cache_alloc(B, Hkv, L, d, cdt)
    ra.cache_write(cache2, k[:, :, :prompt], v[:, :, :prompt])
    at = prompt
    for T in (1, 1, 4, 3):
        lens = _i32([at])
        ra.cache_write(cache2, k[:, :, at:at + T], v[:, :, at:at + T], lens)
        out, lse = ra.tree_fwd(q[:, :, at:at + T].contiguous(), cache2, lens, window=W, sinks=S)
        # both sides hold their weights in bfloat16 or better, and round outputs of up to about 4
        assert float((out.float() - whole[:, :, at:at + T].float()).abs().max()) <= 4 * 2.0 ** -7
        assert float((lse - wl[:, :, at:at + T]).abs().max()) <= 2.0 ** -7 if cdt == E4M3 else 2.0 ** -14
        at += T
    assert at == L
