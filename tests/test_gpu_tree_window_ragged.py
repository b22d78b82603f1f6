"""One long sequence among short ones, read through a wide window: the cached rows are shared out over the GPU whatever the batch, as
they are without a window."""
import pytest
import torch

import sequence_sharded_exact_gb300 as ra

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def _us(call, calls=10, turns=12):
    """The shortest mean of `calls` calls behind one another, in microseconds."""
    for _ in range(3):
        call()
    best = float("inf")
    for _ in range(turns):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(calls):
            call()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) * 1000 / calls)
    return best


@pytest.mark.parametrize("B,Hkv,G,T,dtype,cdt", [
    (152, 2, 4, 1, BF, BF),        # an item (sequence and kv head) for every CTA there is
    (152, 2, 4, 1, BF, E4M3),
    (19, 8, 4, 8, BF, E4M3),       # one CTA per SM
    (18, 8, 4, 8, BF, BF),
    (76, 8, 4, 1, F32, F32),       # four CTAs per SM
])
def test_one_long_sequence_among_short_ones(B, Hkv, G, T, dtype, cdt):
    """With a window of everything the call reads what it reads without one, and the split is the same: at most half as long again
    (and 15 us), where a CTA that walked the long sequence's rows of a kv head alone would take ten times as long.  Through 8192
    and 1024 rows the same bound holds."""
    d, cap, long = 64, 32800, 32700
    cache = ra.cache_alloc(B, Hkv, cap, d, cdt)
    for x in (cache.k, cache.v):
        x.view(torch.uint8).random_(0, 56)  # finite values of any of the types
    if cdt == E4M3:
        cache.k_exp.fill_(127)
        cache.v_exp.fill_(127)
    q = torch.randn((B, Hkv * G, T, d), device=DEV).to(dtype)
    lens = torch.full((B,), 60, dtype=torch.int32)
    lens[B // 2] = long
    lens = lens.to(DEV)
    none = _us(lambda: ra.tree_fwd(q, cache, lens))
    for W in (2 ** 31 - 1, 8192, 1024):
        got = _us(lambda: ra.tree_fwd(q, cache, lens, window=W, sinks=4))
        print(f"B {B} T {T} {dtype} {cdt} window {W}: {got:.1f} us, without one {none:.1f}")
        assert got <= 1.5 * none + 15, (W, got, none)
