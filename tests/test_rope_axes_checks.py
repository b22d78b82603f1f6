"""What the rotation by several axes refuses, without a GPU."""
import ctypes

import pytest
import torch

from sequence_sharded_exact_gb300 import binding

P = ctypes.c_void_p
BAD, UNSUP = binding.RA_ERR_INVALID_ARG, binding.RA_ERR_UNSUPPORTED
OK = binding.RA_OK if torch.cuda.is_available() else binding.RA_ERR_NO_DEVICE
BASE = dict(q=256, qs=None, k=256, ks=None, wq=256, wk=256, qo=256, ko=256, dyq=256, dyk=256, dwq=256, dwk=256, ws=256, bytes=1 << 30, B=1, H=4,
            Hkv=2, rows=10, d=128, axes=3, sections=(16, 24, 24), spectrum=0, dtype=1, base=10000.0, eps=1e-6, pos=256)


def _strides(x):
    return None if x is None else (ctypes.c_longlong * 3)(*x)


def _call(backward, **kw):
    a = {**BASE, **kw}
    lib = binding.library()
    sec = None if a["sections"] is None else (ctypes.c_int * len(a["sections"]))(*a["sections"])
    head = (P(a["q"]), _strides(a["qs"]), P(a["k"]), _strides(a["ks"]), P(a["wq"]), P(a["wk"]))
    tail = (a["B"], a["H"], a["Hkv"], a["rows"], a["d"], a["axes"], sec, a["spectrum"], a["dtype"], a["base"], a["eps"], P(a["pos"]), None)
    if backward:
        return lib.ring_attn_qk_rope_axes_bwd(*head, P(a["dyq"]), P(a["dyk"]), P(a["qo"]), P(a["ko"]), P(a["dwq"]), P(a["dwk"]), P(a["ws"]),
                                              a["bytes"], *tail)
    return lib.ring_attn_qk_rope_axes(*head, P(a["qo"]), P(a["ko"]), *tail)


@pytest.mark.parametrize("kw,status", [
    (dict(axes=0), BAD), (dict(axes=5, sections=(16, 16, 16, 8, 8)), BAD), (dict(sections=None), BAD), (dict(sections=(16, 24, 23)), BAD),
    (dict(sections=(80, -16, 0)), BAD), (dict(spectrum=2), BAD), (dict(pos=0), BAD), (dict(pos=258), BAD), (dict(d=96, sections=(16, 16, 16)), UNSUP),
    (dict(dtype=2), BAD), (dict(wq=0), BAD), (dict(wk=0), BAD), (dict(q=0), BAD), (dict(k=264), BAD), (dict(ko=0), BAD), (dict(base=0.0), BAD),
    (dict(eps=-1.0), BAD), (dict(H=3), BAD), (dict(rows=0), BAD), (dict(qs=(5120, 1280, 4)), BAD), (dict(ks=(-8, 1280, 128), B=2), BAD),
])
@pytest.mark.parametrize("backward", [False, True])
def test_refusals(backward, kw, status):
    assert _call(backward, **kw) == status
    assert binding.library().ring_attn_last_error()


@pytest.mark.parametrize("kw", [dict(dyq=0), dict(dyk=0), dict(dwq=0), dict(ws=0), dict(ws=128), dict(bytes=64)])
def test_refusals_of_the_backward(kw):
    assert _call(True, **kw) == BAD


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device answer")
def test_what_is_accepted():
    assert _call(False) == OK and _call(True) == OK
    assert _call(False, wq=0, wk=0, eps=0.0) == OK
    assert _call(True, wq=0, wk=0, q=0, k=0, dwq=0, dwk=0, ws=0, bytes=0) == OK
    assert _call(False, axes=1, sections=(64,)) == OK and _call(False, axes=4, sections=(64, 0, 0, 0), spectrum=1) == OK
