"""Last tiles of every shape: warps of which some rows, all or none lie behind the sequence, in the forward's and the backward's
epilogues, several units per CTA; and steps over a cache whose query rows end inside a warp."""
import pytest
import torch

import cache_util as cu
import sequence_sharded_exact_gb300 as ra
import window_util as wu

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _clean_status():
    torch.cuda.set_device(0)
    ra.device_status()
    yield
    assert ra.device_status() == 0


def _randn(*shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(BF).to(DEV)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", [BF, F32])
@pytest.mark.parametrize("L", [1, 2, 31, 32, 33, 63, 65, 95, 97, 127, 129, 160, 161, 223, 255, 257])
def test_rows_behind_the_sequence(L, kind, d):
    q, k, v, dout = (_randn(40, h, L, d, seed=L + i) for i, h in enumerate((6, 2, 2, 6)))  # 240 heads: CTAs go through several units
    for causal in (True, False):
        out, lse = ra.window_fwd(q, k, v, 1, 50, 3, causal, "contiguous", out_dtype=kind)
        grads = ra.window_bwd(q, k, v, out, lse, dout, 1, 50, 3, causal, "contiguous", grad_dtype=kind)
        for b in (0, 39):
            one = [x[b:b + 1] for x in (q, k, v, out, lse, dout)]
            cu.check_tree([x[b:b + 1] for x in (out, lse)], wu.fwd(*one[:3], 1, "contiguous", 50, 3, causal), 2.0 ** -8, kind, f"{L} {b}")
            wu.check_bwd([x[b:b + 1] for x in grads], wu.bwd(*one, 1, "contiguous", 50, 3, causal, 2.0 ** -8), f"{L} {b}")


@pytest.mark.parametrize("window", [None, 60])
@pytest.mark.parametrize("kind", [BF, F32])
@pytest.mark.parametrize("T", [9, 17, 31, 33, 65, 129])
def test_query_rows_that_end_inside_a_warp(T, kind, window):
    B, H, Hkv, d, cap, lens = 3, 3, 1, 128, 700, [500, 0, 300]
    cache = ra.cache_alloc(B, Hkv, cap, d, BF)
    ra.cache_write(cache, _randn(B, Hkv, cap, d, seed=1), _randn(B, Hkv, cap, d, seed=2))
    q = _randn(B, H, T, d, seed=T)
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    k, v = cu.cache_values(cache)
    if window is None:
        ref, kw = cu.tree(q, k, v, lens, None, None), {}
    else:
        ref, kw = wu.tree(q, k, v, lens, torch.ones(T, T).tril().bool() & ~torch.ones(T, T).tril(-window).bool(), None, window, 0, None), dict(window=window)
    cu.check_tree(ra.tree_fwd(q, cache, n, out_dtype=kind, **kw), ref, 2.0 ** -8, kind)
