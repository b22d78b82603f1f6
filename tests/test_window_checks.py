"""What the attention through a window refuses, without a GPU."""
import ctypes

import pytest
import torch

import sequence_sharded_exact_gb300 as ra
from sequence_sharded_exact_gb300 import binding

P = ctypes.c_void_p
BAD, UNSUP = binding.RA_ERR_INVALID_ARG, binding.RA_ERR_UNSUPPORTED
OK = binding.RA_OK if torch.cuda.is_available() else binding.RA_ERR_NO_DEVICE
BASE = dict(q=256, k=256, v=256, out=256, lse=256, dout=256, dq=256, dk=256, dv=256, ws=256, bytes=1 << 40, B=1, H=4, Hkv=2, L=1024,
            d=128, n=4, window=100, sinks=4, causal=1, layout=1, dtype=1, out_dtype=1, grad=0)


def _fwd(**kw):
    a = {**BASE, **kw}
    return binding.library().ring_attn_window_fwd(
        P(a["q"]), P(a["k"]), P(a["v"]), P(a["out"]), P(a["lse"]), P(a["ws"]), a["bytes"], a["B"], a["H"], a["Hkv"], a["L"], a["d"],
        a["n"], a["window"], a["sinks"], a["causal"], a["layout"], a["dtype"], a["out_dtype"], None)


def _bwd(**kw):
    a = {**BASE, **kw}
    return binding.library().ring_attn_window_bwd(
        P(a["q"]), P(a["k"]), P(a["v"]), P(a["out"]), P(a["lse"]), P(a["dout"]), P(a["dq"]), P(a["dk"]), P(a["dv"]), P(a["ws"]),
        a["bytes"], a["B"], a["H"], a["Hkv"], a["L"], a["d"], a["n"], a["window"], a["sinks"], a["causal"], a["layout"], a["dtype"],
        a["out_dtype"], a["grad"], None)


REFUSED = [
    (dict(window=0), BAD), (dict(window=-5), BAD), (dict(sinks=-1), BAD), (dict(causal=2), BAD), (dict(layout=3), BAD),
    (dict(dtype=2), BAD), (dict(out_dtype=2), BAD), (dict(dtype=0, out_dtype=1), BAD), (dict(d=96), UNSUP), (dict(H=5), BAD),
    (dict(L=1020), BAD), (dict(L=0), BAD), (dict(B=0), BAD), (dict(q=0), BAD), (dict(k=8), BAD), (dict(lse=260), BAD),
    (dict(L=1 << 30, n=1, layout=0), UNSUP),
]


@pytest.mark.parametrize("kw,status", REFUSED)
def test_refusals(kw, status):
    for call in (_fwd, _bwd):
        assert call(**kw) == status
        assert binding.library().ring_attn_last_error()


@pytest.mark.parametrize("kw,status", [(dict(grad=2), BAD), (dict(dout=0), BAD), (dict(dv=24), BAD), (dict(ws=0), BAD), (dict(ws=128), BAD),
                                       (dict(bytes=16), BAD)])
def test_refusals_of_the_backward(kw, status):
    assert _bwd(**kw) == status


def test_workspaces():
    lib = binding.library()
    assert lib.ring_attn_window_bwd_workspace_size(1, 4, 2, 1024, 128, 4, 100, 4, 1, 1, 1) > 0
    for bad in ((0, 4, 2, 1024, 128, 4, 100, 4, 1, 1, 1), (1, 5, 2, 1024, 128, 4, 100, 4, 1, 1, 1), (1, 4, 2, 1024, 128, 4, 0, 4, 1, 1, 1)):
        assert lib.ring_attn_window_bwd_workspace_size(*bad) == 0


def test_sinks_need_a_window():
    q = torch.zeros(1, 2, 64, 64)
    with pytest.raises(ValueError, match="window"):
        ra.ring_attention(q, q, q, 1, sinks=4)


def test_tensors_are_checked_before_the_library_sees_them():
    q = torch.zeros(1, 2, 64, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ra.window_fwd(q, q, q, 1, 16)
