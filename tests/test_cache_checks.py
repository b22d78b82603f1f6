"""Refusals of the norm-and-rotation, cache and tree attention calls: the binding's checks of tensors, and the
library's of its own arguments, before any CUDA call."""
import ctypes

import pytest
import torch

import sequence_sharded_exact_gb300 as ra
from sequence_sharded_exact_gb300 import binding

INV, UNS = binding.RA_ERR_INVALID_ARG, binding.RA_ERR_UNSUPPORTED
P = ctypes.c_void_p
B, H, Hkv, T, d, cap = 2, 4, 2, 3, 64, 10


@pytest.fixture(scope="module")
def lib():
    return binding.library()


def _strides(*s):
    return (ctypes.c_longlong * 3)(*s)


def _norm(lib, bwd=False, **kw):
    a = dict(q=16, qs=None, k=16, ks=None, wq=16, wk=16, yq=16, yk=16, dq=16, dk=16, dwq=16, dwk=16, ws=256, wsb=1 << 30,
             B=1, H=4, Hkv=2, L=32, d=64, n=2, shard=-1, layout=0, dtype=1, base=1e4, eps=1e-6, pos=None)
    a.update(kw)
    tail = (a["B"], a["H"], a["Hkv"], a["L"], a["d"], a["n"], a["shard"], a["layout"], a["dtype"], a["base"], a["eps"], a["pos"], None)
    if not bwd:
        return lib.ring_attn_qk_norm_rope(a["q"], a["qs"], a["k"], a["ks"], a["wq"], a["wk"], a["yq"], a["yk"], *tail)
    return lib.ring_attn_qk_norm_rope_bwd(a["q"], a["qs"], a["k"], a["ks"], a["wq"], a["wk"], a["yq"], a["yk"], a["dq"], a["dk"],
                                          a["dwq"], a["dwk"], a["ws"], a["wsb"], *tail)


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(q=0), INV), (dict(k=8), INV), (dict(wq=0), INV), (dict(yk=4), INV), (dict(B=0), INV), (dict(L=0), INV),
    (dict(H=3), INV), (dict(L=33), INV), (dict(layout=1, L=34), INV), (dict(layout=3), INV), (dict(dtype=2), INV),
    (dict(d=96), UNS), (dict(shard=2), INV), (dict(shard=-2), INV), (dict(base=0.0), INV), (dict(base=float("inf")), INV),
    (dict(base=float("nan")), INV), (dict(eps=-1e-6), INV), (dict(eps=float("nan")), INV), (dict(pos=2), INV),
    (dict(qs=_strides(1, 64, 4)), INV), (dict(ks=_strides(0, -64, 64)), INV), (dict(qs=_strides(0, 1 << 41, 64)), UNS),
])
def test_norm_rope_argument_errors(lib, bwd, kw, status):
    assert _norm(lib, bwd, **kw) == status
    assert lib.ring_attn_last_error().decode()


@pytest.mark.parametrize("kw", [dict(dwq=0), dict(dk=0), dict(ws=0), dict(ws=128), dict(wsb=1000)])
def test_norm_rope_backward_argument_errors(lib, kw):
    assert _norm(lib, True, **kw) == INV


def test_strides_of_axes_of_length_one_do_not_matter(lib):
    ok = (binding.RA_ERR_NO_DEVICE,) if not torch.cuda.is_available() else None
    if ok is None:
        pytest.skip("would launch")
    assert _norm(lib, B=1, H=1, Hkv=1, L=2, n=1, qs=_strides(3, 5, 64), ks=_strides(-1, 7, 64)) in ok


def _write(lib, **kw):
    a = dict(k=16, ks=None, v=16, vs=None, kc=16, vc=16, ke=1, ve=1, lens=4, ntok=None, B=2, Hkv=2, T=3, d=64, cap=10, dtype=1, cdt=2)
    a.update(kw)
    return lib.ring_attn_cache_write(a["k"], a["ks"], a["v"], a["vs"], a["kc"], a["vc"], a["ke"], a["ve"], a["lens"], a["ntok"],
                                     a["B"], a["Hkv"], a["T"], a["d"], a["cap"], a["dtype"], a["cdt"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(k=0), INV), (dict(vc=8), INV), (dict(ke=0), INV), (dict(lens=2), INV), (dict(ntok=1), INV), (dict(B=0), INV),
    (dict(T=0), INV), (dict(cap=0), INV), (dict(dtype=2), INV), (dict(cdt=0), INV), (dict(cdt=3), INV), (dict(d=32), UNS),
    (dict(lens=None, T=11), INV), (dict(ks=_strides(2, 64, 64)), INV), (dict(cap=1 << 30, B=1 << 10), UNS),
    (dict(B=1 << 16, Hkv=1 << 15), UNS),
])
def test_cache_write_argument_errors(lib, kw, status):
    assert _write(lib, **kw) == status


def _read(lib, **kw):
    a = dict(kc=16, vc=16, ke=1, ve=1, k=16, v=16, B=2, Hkv=2, row0=0, rows=10, d=64, cap=10, dtype=1, cdt=2)
    a.update(kw)
    return lib.ring_attn_cache_read(a["kc"], a["vc"], a["ke"], a["ve"], a["k"], a["v"], a["B"], a["Hkv"], a["row0"], a["rows"], a["d"],
                                    a["cap"], a["dtype"], a["cdt"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(row0=-1), INV), (dict(rows=-1), INV), (dict(rows=11), INV), (dict(row0=1), INV), (dict(row0=2 ** 31 - 1, rows=2 ** 31 - 1), INV),
    (dict(v=0), INV), (dict(ve=0), INV), (dict(cdt=1, dtype=0), INV), (dict(rows=0), binding.RA_OK),
])
def test_cache_read_argument_errors(lib, kw, status):
    assert _read(lib, **kw) == status


def _tree(lib, **kw):
    a = dict(q=16, kc=16, vc=16, ke=1, ve=1, lens=4, ntok=None, mask=1, mb=1, out=16, lse=16, ws=256, wsb=1 << 40, B=2, H=4, Hkv=2, T=3,
             d=64, cap=10, dtype=1, cdt=2, odt=1)
    a.update(kw)
    return lib.ring_attn_tree_fwd(a["q"], a["kc"], a["vc"], a["ke"], a["ve"], a["lens"], a["ntok"], a["mask"], a["mb"], a["out"], a["lse"],
                                  a["ws"], a["wsb"], a["B"], a["H"], a["Hkv"], a["T"], a["d"], a["cap"], a["dtype"], a["cdt"], a["odt"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=0), INV), (dict(out=8), INV), (dict(lens=None), INV), (dict(lens=2), INV), (dict(ntok=6), INV), (dict(H=3), INV),
    (dict(T=0), INV), (dict(H=0), INV), (dict(d=256), UNS), (dict(dtype=0, cdt=1), INV), (dict(odt=2), INV), (dict(dtype=0, odt=1), INV),
    (dict(ws=0), INV), (dict(ws=16), INV), (dict(wsb=64), INV), (dict(ke=None), INV), (dict(T=1 << 29), UNS), (dict(lse=0), INV),
])
def test_tree_argument_errors(lib, kw, status):
    assert _tree(lib, **kw) == status


def test_workspace_sizes(lib):
    f = lib.ring_attn_tree_fwd_workspace_size
    assert f(1, 4, 2, 1, 64, 1, 1, 1) >= 2 * 2 * 4 * 66  # two CTAs' slots of one row at least
    assert f(8, 32, 8, 64, 128, 1 << 20, 1, 2) <= 64 << 20  # bounded whatever the cache
    assert f(1, 3, 2, 1, 64, 10, 1, 1) == 0 and f(0, 4, 2, 1, 64, 10, 1, 1) == 0
    assert lib.ring_attn_qk_norm_rope_bwd_workspace_size(128) >= 2 * 128 * 4


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device answer")
def test_no_device_answer(lib):
    assert _norm(lib) == _norm(lib, True) == _write(lib) == _read(lib) == _tree(lib) == binding.RA_ERR_NO_DEVICE


def test_host_tensors_are_refused():
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
    q, k, w = z(B, H, T, d), z(B, Hkv, T, d), z(d, dt=torch.float32)
    cache = ra.KVCache(z(B, Hkv, cap, d), z(B, Hkv, cap, d))
    lens = torch.zeros(B, dtype=torch.int32)
    for call in (lambda: ra.qk_norm_rope(q, k, w, w), lambda: ra.qk_norm_rope_bwd(q, k, w, w, q, k),
                 lambda: ra.ring_qk_norm_rope(q, k, w, w), lambda: ra.cache_write(cache, k, k, lens),
                 lambda: ra.cache_read(cache, 4), lambda: ra.tree_fwd(q, cache, lens)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
    with pytest.raises(ValueError, match="dtype"):
        ra.cache_alloc(1, 1, 4, 64, dtype=torch.float16, device="cpu")


@pytest.mark.gpu
def test_device_tensors_that_do_not_fit_are_refused():
    dev = "cuda:0"
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device=dev)  # noqa: E731
    q, k, w = z(B, H, T, d), z(B, Hkv, T, d), z(d, dt=torch.float32)
    lens = torch.zeros(B, dtype=torch.int32, device=dev)
    cache = ra.cache_alloc(B, Hkv, cap, d)
    plain = ra.cache_alloc(B, Hkv, cap, d, torch.float32)
    ws = torch.zeros(64, dtype=torch.uint8, device=dev)
    bad = [
        lambda: ra.qk_norm_rope(q, k.float(), w, w),
        lambda: ra.qk_norm_rope(q.half(), k.half(), w, w),
        lambda: ra.qk_norm_rope(q, z(B, Hkv, T + 1, d), w, w),
        lambda: ra.qk_norm_rope(q, k, w.bfloat16(), w),
        lambda: ra.qk_norm_rope(q, k, w[:32], w),
        lambda: ra.qk_norm_rope(z(B, H, d, T).transpose(2, 3), k, w, w),           # rows not contiguous
        lambda: ra.qk_norm_rope(z(B, H, T, d + 4)[..., :d], k, w, w),              # rows off 16-byte boundaries
        lambda: ra.qk_norm_rope(q, k, w, w, q_out=z(B, T, H, d).transpose(1, 2)),  # outputs are contiguous
        lambda: ra.qk_norm_rope(q, k, w, w, positions=torch.zeros(B, T, device=dev)),
        lambda: ra.qk_norm_rope(q, k, w, w, 3, positions=torch.zeros(B, T, dtype=torch.int32, device=dev)),
        lambda: ra.qk_norm_rope(q, k, w, w, 2, shard=2),
        lambda: ra.qk_norm_rope_bwd(q, k, w, w, q.float(), k),
        lambda: ra.qk_norm_rope_bwd(q, k, w, w, z(B, T, H, d).transpose(1, 2), k),
        lambda: ra.qk_norm_rope_bwd(q, k, w, w, q, k, workspace=ws),
        lambda: ra.cache_write(cache, k, z(B, Hkv, T + 1, d), lens),
        lambda: ra.cache_write(cache, k, k, lens.long()),
        lambda: ra.cache_write(cache, k, k, lens[:1]),
        lambda: ra.cache_write(cache._replace(k_exp=None), k, k, lens),
        lambda: ra.cache_write(cache._replace(v=z(B, Hkv, cap - 1, d, dt=torch.float8_e4m3fn)), k, k, lens),
        lambda: ra.cache_write(plain, k, k, lens),                                 # float32 cache, bf16 rows
        lambda: ra.cache_read(cache, cap + 1),
        lambda: ra.cache_read(cache, 2, row0=cap - 1),
        lambda: ra.cache_read(cache, 2, dtype=torch.float16),
        lambda: ra.tree_fwd(q, plain, lens),
        lambda: ra.tree_fwd(q, cache, None),
        lambda: ra.tree_fwd(q, cache, lens, mask=torch.ones(B, T, T, device=dev)),
        lambda: ra.tree_fwd(q, cache, lens, mask=torch.ones(T, T + 1, dtype=torch.bool, device=dev)),
        lambda: ra.tree_fwd(q, cache, lens, out_dtype=torch.float16),
        lambda: ra.tree_fwd(q, cache, lens, workspace=ws),
        lambda: ra.tree_fwd(q, cache, lens, out=z(B, H, T, d, dt=torch.float32)),
        lambda: ra.tree_fwd(q[:1], cache, lens[:1]),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            call()
            pytest.fail(f"call {i} was taken")
    with pytest.raises(ra.RingAttnError, match="aligned"):  # a base off 16-byte boundaries
        x = z(B * H * T * d + 8)[2:2 + B * H * T * d].view(B, H, T, d)
        ra.qk_norm_rope(x, k, w, w)
    with pytest.raises(ra.RingAttnError, match="multiple of Hkv"):
        ra.tree_fwd(z(B, 3, T, d), cache, lens)
    torch.cuda.synchronize()
    assert ra.device_status() == 0


@pytest.mark.parametrize("call,kw", [
    ("write", dict(B=1, Hkv=1, T=1 << 30, cap=1 << 29)), ("write", dict(B=1, Hkv=1, cap=1 << 30)), ("read", dict(B=1, Hkv=1, cap=1 << 30)),
    ("read", dict(B=1 << 15, Hkv=1 << 15, cap=10)), ("tree", dict(B=1, Hkv=1, cap=1 << 30)),
])
def test_row_counts_that_an_int_could_not_step_over(lib, call, kw):
    assert {"write": _write, "read": _read, "tree": _tree}[call](lib, **kw) == UNS


def test_the_compiled_calls_are_there_and_leave_what_they_do_not_take(lib):
    """Built beside the library for this Python and torch; host tensors and odd arguments are left to the Python form."""
    calls = binding._calls
    assert calls is not None
    x = torch.zeros(1, 1, 1, 64)
    cache = binding.KVCache(x, x)
    assert calls.tree_fwd(x, cache, None, None, None, None, None, None, None) is None
    assert calls.cache_write(cache, x, x, None, None) is None
    assert calls.cache_read(cache, 1, 0, torch.float32, None, None) is None
    assert calls.cache_read(None, "1", 0, 3, None, None) is None
    assert calls.qk_norm_rope(x, x, x, x, 1, "zigzag", 1.0, 0.0, None, None, None, None) is None
    assert calls.qk_norm_rope_bwd(1, None, x, x, x, x, 1, 2, 1.0, 0.0, None, None, None, None, None) is None
    with pytest.raises(TypeError):
        calls.tree_fwd(x)
