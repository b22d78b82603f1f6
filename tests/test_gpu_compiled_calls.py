"""The compiled calls (csrc/calls.cpp) against the Python form of the same functions: the same bits, the same errors."""
import pytest
import torch

import sequence_sharded_exact_gb300 as ra
from sequence_sharded_exact_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def _randn(*shape, seed, dtype=F32):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _both(monkeypatch, call):
    """The call's results through the compiled form, and through the Python form."""
    ra.device_status()
    taken = []
    real = binding._calls
    assert real is not None

    class Watch:
        def __getattr__(self, name):
            def f(*a):
                r = getattr(real, name)(*a)
                taken.append(r is not None)
                return r
            return f

    monkeypatch.setattr(binding, "_calls", Watch())
    fast = call()
    assert taken == [True], "the compiled form did not take the call"
    monkeypatch.setattr(binding, "_calls", None)
    slow = call()
    monkeypatch.undo()
    return fast, slow


def _same(a, b):
    assert len(a) == len(b)
    for x, y in zip(a, b):
        assert x.dtype == y.dtype and x.shape == y.shape and x.is_contiguous() and not x.requires_grad
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("where", ["layout", "shard", "positions"])
def test_norms_with_rotation(monkeypatch, dtype, fused, where):
    B, H, Hkv, L, d = 2, 4, 2, 24, 64
    x = _randn(B, L, H + 2 * Hkv, d, seed=1, dtype=dtype)
    q, k, _ = (t.transpose(1, 2) for t in x.split([H, Hkv, Hkv], dim=2))
    if not fused:
        q, k = q.contiguous(), k.contiguous()
    wq, wk = torch.nn.Parameter(_randn(d, seed=2)), _randn(d, seed=3)
    kw = dict(layout=dict(n_shards=3, layout="zigzag"), shard=dict(n_shards=3, layout="striped", shard=2),
              positions=dict(positions=_i32(*range(B * L)).view(B, L)))[where]
    _same(*_both(monkeypatch, lambda: ra.qk_norm_rope(q, k, wq, wk, base=5000.0, eps=1e-5, **kw)))
    dq, dk = _randn(B, H, L, d, seed=4, dtype=dtype), _randn(B, Hkv, L, d, seed=5, dtype=dtype)
    _same(*_both(monkeypatch, lambda: ra.qk_norm_rope_bwd(q, k, wq, wk, dq, dk, base=5000.0, eps=1e-5, **kw)))
    qo, ko = torch.empty(B, H, L, d, dtype=dtype, device=DEV), torch.empty(B, Hkv, L, d, dtype=dtype, device=DEV)
    got = ra.qk_norm_rope(q, k, wq, wk, q_out=qo, k_out=ko, **kw)
    assert got[0].data_ptr() == qo.data_ptr() and got[1].data_ptr() == ko.data_ptr()


@pytest.mark.parametrize("dtype,cdt", [(BF, E4M3), (F32, E4M3), (BF, BF), (F32, F32)])
def test_cache_and_attention(monkeypatch, dtype, cdt):
    B, H, Hkv, T, d, cap = 2, 4, 2, 3, 64, 40
    k, v, q = _randn(B, Hkv, T, d, seed=1, dtype=dtype), _randn(B, Hkv, T, d, seed=2, dtype=dtype), _randn(B, H, T, d, seed=3, dtype=dtype)
    lens, ntok = _i32(20, 5), _i32(3, 1)

    def write():
        cache = ra.cache_alloc(B, Hkv, cap, d, cdt)
        assert ra.cache_write(cache, k, v, lens, ntok=ntok) is cache
        return [t for t in cache if t is not None]

    _same(*_both(monkeypatch, write))
    cache = ra.cache_alloc(B, Hkv, cap, d, cdt)
    ra.cache_write(cache, _randn(B, Hkv, cap, d, seed=4, dtype=dtype), _randn(B, Hkv, cap, d, seed=5, dtype=dtype))
    _same(*_both(monkeypatch, lambda: ra.cache_read(cache, 7, row0=4, dtype=dtype)))
    _same(*_both(monkeypatch, lambda: ra.tree_fwd(q, cache, lens)))
    mask = torch.eye(T, dtype=torch.bool, device=DEV)
    _same(*_both(monkeypatch, lambda: ra.tree_fwd(q, cache, lens, mask=mask, ntok=ntok, out_dtype=F32)))
    ws = torch.empty(ra.tree_workspace_size(B, H, Hkv, T, d, cap, dtype, cdt), dtype=torch.uint8, device=DEV)
    out, lse = torch.empty_like(q), torch.empty(B, H, T, device=DEV)
    _same(*_both(monkeypatch, lambda: ra.tree_fwd(q, cache, lens, mask=mask.expand(B, T, T).contiguous(), out=out, lse=lse, workspace=ws)))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):  # the current stream is another one
        fast, slow = _both(monkeypatch, lambda: ra.tree_fwd(q, cache, lens))
    s.synchronize()
    _same(fast, slow)
    assert ra.device_status() == 0


def test_errors_are_the_python_forms(monkeypatch):
    B, H, Hkv, T, d, cap = 1, 4, 2, 2, 64, 16
    cache, q = ra.cache_alloc(B, Hkv, cap, d, BF), torch.zeros(B, H, T, d, dtype=BF, device=DEV)
    lens, w = _i32(4), torch.ones(d, device=DEV)
    calls = [
        lambda: ra.tree_fwd(q, cache, lens.long()), lambda: ra.tree_fwd(q, cache, None), lambda: ra.tree_fwd(q.half(), cache, lens),
        lambda: ra.tree_fwd(q.transpose(1, 2), cache, lens), lambda: ra.tree_fwd(q, cache, lens, mask=torch.ones(3, 3, device=DEV)),
        lambda: ra.tree_fwd(q, cache, lens, out_dtype=torch.float16), lambda: ra.tree_fwd(q.cpu(), cache, lens),
        lambda: ra.tree_fwd(q, cache, lens, workspace=torch.empty(8, dtype=torch.uint8, device=DEV)),
        lambda: ra.cache_write(cache, q, q), lambda: ra.cache_read(cache, 17, dtype=BF), lambda: ra.cache_read(cache, 1),
        lambda: ra.cache_read(cache, 1, dtype=torch.float16), lambda: ra.qk_norm_rope(q, q, w.double(), w),
        lambda: ra.qk_norm_rope(q, q, w, w, n_shards=2, shard=5), lambda: ra.qk_norm_rope(q, q, w, w, layout="round"),
        lambda: ra.qk_norm_rope(q, q[..., ::2], w, w), lambda: ra.qk_norm_rope_bwd(q, q, w, w, q, q.float()),
    ]
    for i, call in enumerate(calls):
        said = []
        for compiled in (True, False):
            with monkeypatch.context() as m:
                if not compiled:
                    m.setattr(binding, "_calls", None)
                try:
                    call()
                    said.append(None)
                except Exception as e:
                    said.append((type(e), str(e)))
        assert said[0] == said[1], (i, said)
