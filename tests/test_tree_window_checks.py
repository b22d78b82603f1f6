"""What the attention over a cache through a window refuses, without a GPU."""
import ctypes

import pytest
import torch

from sequence_sharded_exact_gb300 import binding

P = ctypes.c_void_p
BAD = binding.RA_ERR_INVALID_ARG
OK = binding.RA_OK if torch.cuda.is_available() else binding.RA_ERR_NO_DEVICE
BASE = dict(q=256, k=256, v=256, ke=256, ve=256, lens=256, ntok=0, mask=256, batched=1, pos=256, out=256, lse=256, ws=256, bytes=1 << 40, B=2, H=8,
            Hkv=2, T=4, d=128, cap=1000, window=100, sinks=4, dtype=1, cdt=2, odt=1)


def _call(**kw):
    a = {**BASE, **kw}
    return binding.library().ring_attn_tree_window_fwd(
        P(a["q"]), P(a["k"]), P(a["v"]), P(a["ke"]), P(a["ve"]), P(a["lens"]), P(a["ntok"]), P(a["mask"]), a["batched"], P(a["pos"]), P(a["out"]),
        P(a["lse"]), P(a["ws"]), a["bytes"], a["B"], a["H"], a["Hkv"], a["T"], a["d"], a["cap"], a["window"], a["sinks"], a["dtype"], a["cdt"],
        a["odt"], None)


@pytest.mark.parametrize("kw", [dict(window=0), dict(window=-1), dict(sinks=-1), dict(mask=0), dict(pos=258), dict(lens=0), dict(q=8), dict(T=0),
                                dict(H=7), dict(cap=0), dict(odt=2), dict(ws=0), dict(bytes=100), dict(ke=0), dict(cdt=0)])
def test_refusals(kw):
    assert _call(**kw) == BAD
    assert binding.library().ring_attn_last_error()


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device answer")
def test_what_is_accepted():
    for kw in (dict(), dict(pos=0), dict(pos=0, mask=0), dict(window=2 ** 31 - 1, sinks=2 ** 31 - 1), dict(window=1, sinks=0)):
        assert _call(**kw) == OK
