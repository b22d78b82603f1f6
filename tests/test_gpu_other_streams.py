"""Calls given another stream than the current one: what they allocate may be memory that the current stream still works with."""
import pytest
import torch

import sequence_sharded_exact_gb300 as ra

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, E4M3 = torch.bfloat16, torch.float8_e4m3fn


def _randn(*shape, seed, dtype=torch.float32):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


def _inputs():
    B, H, Hkv, T, d, cap = 1, 8, 2, 4, 128, 2000
    cache = ra.cache_alloc(B, Hkv, cap, d, E4M3)
    ra.cache_write(cache, _randn(B, Hkv, cap, d, seed=1, dtype=BF), _randn(B, Hkv, cap, d, seed=2, dtype=BF))
    q, k, w = _randn(B, H, T, d, seed=3, dtype=BF), _randn(B, Hkv, T, d, seed=4, dtype=BF), _randn(d, seed=5)
    lens = torch.tensor([1900], dtype=torch.int32, device=DEV)
    return {
        "cache_read": lambda **kw: ra.cache_read(cache, 300, row0=7, **kw),
        "qk_norm_rope": lambda **kw: ra.qk_norm_rope(q, k, w, w, **kw),
        "qk_norm_rope_bwd": lambda **kw: ra.qk_norm_rope_bwd(q, k, w, w, q, k, **kw),
        "tree_fwd": lambda **kw: ra.tree_fwd(q, cache, lens, **kw),
    }


@pytest.mark.parametrize("name", ["cache_read", "qk_norm_rope", "qk_norm_rope_bwd", "tree_fwd"])
def test_memory_that_the_current_stream_still_writes(name):
    call = _inputs()[name]
    ref = call()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        late = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in (1 << 12, 1 << 16, 1 << 20, 1 << 21) for _ in range(4)]
        torch.cuda._sleep(50_000_000)
        for t in late:
            t.fill_(255)
        del late, t  # free for the current stream, which has yet to write it
        got = call(stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_a_stream_that_is_part_of_a_capture():
    call = _inputs()["tree_fwd"]
    ref = call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call(stream=s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.wait_stream(torch.cuda.current_stream())
        got = call(stream=s)
        torch.cuda.current_stream().wait_stream(s)
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_nothing_waits_where_everything_is_given():
    """A call whose outputs and workspace are the caller's own runs beside the current stream's work."""
    call = _inputs()["tree_fwd"]
    out, lse = call()
    ws = torch.empty(ra.tree_workspace_size(1, 8, 2, 4, 128, 2000, BF, E4M3), dtype=torch.uint8, device=DEV)
    ref = out.clone(), lse.clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    torch.cuda._sleep(500_000_000)
    call(stream=s, out=out, lse=lse, workspace=ws)
    s.synchronize()
    assert not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
