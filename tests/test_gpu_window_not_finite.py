"""Attention of whole sequences through a window beside values that are not finite: who sees one has it in its column whatever its
weight, nobody else has a part of it, and looking at the rows again takes no wait's time and about as long as the products."""
import math

import pytest
import torch

import cache_util as cu
import sequence_sharded_exact_gb300 as ra
import window_util as wu

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
WEIGHT_EPS = {BF: 2.0 ** -8, F32: 0.0}


@pytest.fixture(autouse=True)
def _clean_status():
    torch.cuda.set_device(0)
    ra.device_status()
    yield
    assert ra.device_status() == 0


def _inputs(B, H, Hkv, L, d, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [torch.randn((B, h, L, d), generator=g, device=DEV).to(dtype) for h in (H, Hkv, Hkv)]


def _check(q, k, v, v2, n, layout, W, S, causal, out_dtype=None):
    """v2: v with elements that are not finite.  An element of the output that sees none of them is v's, within its bound; one
    that sees some is their sum: an infinity of one sign, or NaN."""
    L, d, G = q.shape[2], q.shape[3], q.shape[1] // k.shape[1]
    got, lse = ra.window_fwd(q, k, v2, n, W, S, causal, layout, out_dtype=out_dtype)
    out, rl, mag, big = wu.fwd(q, k, v, n, layout, W, S, causal)
    order = cu.natural(L, n, layout)
    sees = wu.sees(L, W, S, causal)[order][:, order].to(DEV).double()
    bad = v2.double()
    nan, inf, ninf = (x.double() for x in (torch.isnan(bad), bad == math.inf, bad == -math.inf))
    nan, inf, ninf = ((sees @ x > 0).repeat_interleave(G, 1) for x in (nan, inf, ninf))
    none, nan = ~(nan | inf | ninf), nan | (inf & ninf)
    assert bool(torch.isnan(got[nan]).all())
    assert bool((got[inf & ~nan] == math.inf).all()) and bool((got[ninf & ~nan] == -math.inf).all())
    cu.check_tree((torch.where(none.cpu(), got.cpu().double(), out), lse), (out, rl, mag, big), WEIGHT_EPS[q.dtype], got.dtype, "the rest")


SPOILS = {
    "one": lambda v, at: v[:, :, at[300], 5].fill_(math.nan),
    "signs": lambda v, at: [v[:, :, at[j], c].fill_(x) for j, c, x in
                            ((10, 0, math.inf), (127, 0, -math.inf), (128, 31, math.inf), (400, 32, -math.inf), (401, 63, math.nan), (639, 7, math.nan))],
    "rows": lambda v, at: [v[:, :, at[j]].fill_(x) for j, x in ((0, math.inf), (255, math.nan), (256, -math.inf), (511, math.inf))],
    "columns": lambda v, at: [v[..., c].fill_(x) for c, x in ((1, math.inf), (40, math.nan), (63, -math.inf))],
    "all": lambda v, at: v.fill_(-math.inf),
    "kv head": lambda v, at: v[:, 1].fill_(math.inf),
}


@pytest.mark.parametrize("what", SPOILS)
@pytest.mark.parametrize("H,Hkv,d,n,layout,W,S,causal", [
    (4, 2, 128, 1, "contiguous", 70, 3, True),
    (6, 2, 64, 4, "striped", 140, 0, True),
    (3, 3, 128, 5, "striped", 300, 130, True),
    (4, 2, 64, 2, "zigzag", 90, 5, False),
    (2, 2, 64, 1, "contiguous", 1000, 0, True),
])
@pytest.mark.parametrize("dtype,out_dtype", [(BF, BF), (BF, F32), (F32, F32)])
def test_where_values_go(dtype, out_dtype, H, Hkv, d, n, layout, W, S, causal, what):
    q, k, v = _inputs(1, H, Hkv, 640, d, dtype, seed=d + W)
    v2 = v.clone()
    SPOILS[what](v2, torch.argsort(cu.natural(640, n, layout)))
    _check(q, k, v, v2, n, layout, W, S, causal, out_dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("later", [False, True])
def test_a_weight_that_underflows(later, d, dtype):
    """A visible value that is not finite reaches the row although its weight, e^-400 and less, is 0 in float32: met before the
    row's largest score and behind it."""
    L, W, at, top = 400, 300, 150, 260
    if later:
        at, top = top, at
    q, k, v = _inputs(1, 2, 1, L, d, dtype, seed=d)
    q[:] = 1.0
    k *= 2.0 ** -6
    k[:, :, at] = -400 / math.sqrt(d)
    k[:, :, top] = 400 / math.sqrt(d)
    v2 = v.clone()
    v2[:, :, at, 3], v2[:, :, at, 9], v2[:, :, at, 20] = math.inf, -math.inf, math.nan
    _check(q, k, v, v2, 1, "contiguous", W, 0, True)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("what,times", [("sink", 12), ("all", 12), ("all NaN", 12), ("one hidden", 60)])
def test_how_long_it_takes(what, times, d):
    """A wide window.  A row beside such a value is looked at again: by tiles, a few times the products' time; the few rows that share a
    tile with one that they do not see, key by key, 16 thousand of them one after another."""
    L, W = 16384, 8192
    q, k, v = _inputs(1, 8, 2, L, d, BF, seed=d)
    v2 = v.clone()
    if what == "sink":
        v2[:, :, 1] = math.inf
    elif what == "all":
        v2[:] = math.inf
    elif what == "all NaN":
        v2[:] = math.nan
    else:
        v2[:, :, 127 + 128 * 100, 7] = math.nan

    def us(value):
        best = math.inf
        for _ in range(6):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            res = ra.window_fwd(q, k, value, 1, W, 2, True, "contiguous")
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b) * 1000)
        return best, res

    plain, (out, lse) = us(v)
    spoilt, (o2, l2) = us(v2)
    print(f"d {d} {what}: {spoilt:.0f} us, without {plain:.0f}")
    assert torch.equal(l2, lse)
    if what == "one hidden":
        j = 127 + 128 * 100
        assert bool(torch.isnan(o2[:, :, j:j + W, 7]).all())
        sees = torch.zeros(L, d, dtype=torch.bool, device=DEV)
        sees[j:j + W, 7] = True
        assert bool(torch.isfinite(o2[:, :, ~sees]).all())
        # another sum of the same values: both within a weight's rounding of the exact one
        assert float((o2.float() - out.float())[:, :, ~sees].abs().max()) <= 2.0 ** -7
    elif what == "sink":
        assert bool((o2[:, :, 1:] == math.inf).all())
    else:
        assert not bool(torch.isfinite(o2).any())
    assert spoilt <= times * plain, (spoilt, plain)
