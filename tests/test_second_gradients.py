"""The attention's gradients come out of kernels and have no graph of their own: a second differentiation through them is refused
(it would otherwise leave these terms out without a word).  The calls below the operations are replaced, so no GPU is needed."""
import pytest
import torch

import sequence_sharded_exact_gb300 as ra
from sequence_sharded_exact_gb300 import binding, ring


def _fwd(q, k, v, *_, **__):
    return q * k * v, q.sum(-1)


def _bwd(q, k, v, out, lse, dout, *_, **__):
    return dout * k * v, dout * q * v, dout * q * k


def _attend(monkeypatch, how):
    if how == "distributed":
        monkeypatch.setattr(ring, "ring_fwd", _fwd)
        monkeypatch.setattr(ring, "ring_bwd", _bwd)
        return lambda q, k, v: ring.ring_attention_distributed(q, k, v, comm=None, ops=object())
    for name, f in (("fwd", _fwd), ("window_fwd", _fwd), ("bwd", _bwd), ("window_bwd", _bwd)):
        monkeypatch.setattr(binding, name, f)
    kw = dict(window=5, sinks=1) if how == "window" else {}
    return lambda q, k, v: ra.ring_attention(q, k, v, 1, **kw)


@pytest.mark.parametrize("how", ["whole", "window", "distributed"])
@pytest.mark.parametrize("loss", [lambda x: x.sum(), lambda x: x.square().sum()])  # the output's gradient: constant, or not
def test_a_second_differentiation_is_refused(monkeypatch, loss, how):
    attend = _attend(monkeypatch, how)
    q, k, v = (torch.randn(1, 2, 6, 64, requires_grad=True) for _ in range(3))
    out = attend(q, k, v)
    grads = torch.autograd.grad(loss(out), (q, k, v), create_graph=True)
    with torch.no_grad():
        ref = _bwd(q, k, v, None, None, torch.autograd.functional.vjp(loss, out)[1])
    assert all(torch.equal(a, b) for a, b in zip(grads, ref))
    penalty = out.square().sum() + sum(g.square().sum() for g in grads)
    with pytest.raises(RuntimeError, match="differentiated again"):
        penalty.backward()


@pytest.mark.parametrize("norm", [True, False])
def test_of_the_rotations_too(monkeypatch, norm):
    monkeypatch.setattr(binding, "as_rows", lambda t: t)
    monkeypatch.setattr(binding, "qk_norm_rope", lambda q, k, wq, wk, **_: (q * wq, k * wk))
    monkeypatch.setattr(binding, "qk_norm_rope_bwd", lambda q, k, wq, wk, dq, dk, **_: (dq * wq, dk * wk, (dq * q).sum((0, 1, 2)), (dk * k).sum((0, 1, 2))))
    monkeypatch.setattr(binding, "qk_rope_axes", lambda q, k, pos, sections, *w, **_: (2 * q, 2 * k))
    monkeypatch.setattr(binding, "qk_rope_axes_bwd", lambda dq, dk, pos, sections, **_: (2 * dq, 2 * dk, None, None))
    q, k = (torch.randn(1, 2, 6, 64, requires_grad=True) for _ in range(2))
    w = [torch.ones(64, requires_grad=True) for _ in range(2)]
    outs = ra.ring_qk_norm_rope(q, k, *w) if norm else ra.ring_qk_rope_axes(q, k, torch.zeros(1, 1, 6, dtype=torch.int32), (32,))
    grads = torch.autograd.grad(sum(x.sum() for x in outs), (q, k), create_graph=True)
    assert all(torch.equal(g, torch.full_like(g, 1.0 if norm else 2.0)) for g in grads)
    with pytest.raises(RuntimeError, match="differentiated again"):
        sum(g.square().sum() for g in grads).backward()


@pytest.mark.parametrize("how", ["whole", "window", "distributed"])
def test_first_gradients_are_as_they_were(monkeypatch, how):
    attend = _attend(monkeypatch, how)
    q, k, v = (torch.randn(1, 2, 6, 64, requires_grad=True) for _ in range(3))
    attend(q, k, v).sum().backward()
    with torch.no_grad():
        ref = _bwd(q, k, v, None, None, torch.ones_like(q))
    assert all(torch.equal(t.grad, r) for t, r in zip((q, k, v), ref))
