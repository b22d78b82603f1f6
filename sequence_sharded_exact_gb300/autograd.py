"""Ring attention as a differentiable PyTorch operation.

``ring_attention`` runs the library's forward and, when a gradient is needed, its backward: the
same ``ring_attn_fwd`` / ``ring_attn_bwd`` entry points as ``fwd`` and ``bwd`` in the binding.  The
forward saves its output and log-sum-exp; the backward recomputes the attention weights from them
(nothing quadratic is stored).  Gradients come back in the dtype of the inputs; they have no graph of their
own, and a second differentiation through them raises an error.

With ``f32_out=True`` (bf16 inputs) the forward keeps its output in float32 for the backward
(``ring_attn_fwd_f32out``, then ``ring_attn_f32_convert`` for the returned bf16 output) and the
backward takes D = rowsum(dout * out) from it (``ring_attn_bwd_f32out``) instead of from the rounded
output: twice the saved output's memory, and gradients closer to the exact ones where a gradient is
a short sum of large, cancelling terms (the first positions of a causal sequence).
"""
import functools

import torch

from . import binding


class _Refuse(torch.autograd.Function):
    @staticmethod
    def forward(ctx, *grads):
        return tuple(g.view_as(g) for g in grads)

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("the attention's and the rotations' gradients come out of kernels: they cannot be differentiated again")


def first_order(backward):
    """A Function's backward whose gradients have no graph of their own.  Where one is asked for (create_graph=True) they may
    still be used, but a differentiation through them raises an error in place of leaving those terms out.  (PyTorch's
    once_differentiable does so only where the output's gradient needs one: not for that of a plain sum.)"""
    @functools.wraps(backward)
    def run(ctx, *douts):
        with torch.no_grad():
            grads = backward(ctx, *douts)
        if not torch.is_grad_enabled():
            return grads
        marked = iter(_Refuse.apply(*(g.detach().requires_grad_() for g in grads if g is not None)))
        return tuple(None if g is None else next(marked) for g in grads)

    return run


class _RingAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, n_shards, causal, layout, f32_out, window, sinks):
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        f32_out = bool(f32_out) and q.dtype != torch.float32
        if window is not None:
            q, k, v = _dense(q), _dense(k), _dense(v)
            saved, lse = binding.window_fwd(q, k, v, n_shards, window, sinks, causal, layout,
                                            out_dtype=torch.float32 if f32_out else None)
            out = binding.f32_convert(saved, q.dtype) if f32_out else saved
        elif f32_out:
            saved, lse = binding.fwd_f32out(q, k, v, n_shards, causal, layout)
            out = binding.f32_convert(saved, q.dtype)
        else:
            out, lse = binding.fwd(q, k, v, n_shards, causal, layout)
            saved = out
        ctx.save_for_backward(q, k, v, saved, lse)
        ctx.cfg = (n_shards, causal, layout, f32_out, window, sinks)
        return out

    @staticmethod
    @first_order
    def backward(ctx, dout):
        q, k, v, saved, lse = ctx.saved_tensors
        n_shards, causal, layout, f32_out, window, sinks = ctx.cfg
        if window is not None:
            dq, dk, dv = binding.window_bwd(q, k, v, saved, lse, _dense(dout), n_shards, window, sinks, causal, layout,
                                            grad_dtype=q.dtype)
            return dq, dk, dv, None, None, None, None, None, None
        call = binding.bwd_f32out if f32_out else binding.bwd
        dq, dk, dv = call(q, k, v, saved, lse, dout.contiguous(), n_shards, causal, layout, grad_dtype=q.dtype)
        return dq, dk, dv, None, None, None, None, None, None


def ring_attention(q, k, v, n_shards, causal=True, layout="zigzag", f32_out=False, window=None, sinks=0):
    """Exact attention of q [B,H,L,d] over k, v [B,Hkv,L,d] (sequence axis in the layout's order),
    computed as the ring over n_shards shards; differentiable with respect to q, k and v.
    f32_out: keep the forward's output in float32 for the backward's D (see the module notes).
    window, sinks: every token sees the `window` last tokens (itself among them) and the first `sinks` ones alone
    (window_fwd); without a window all that `causal` allows, and `sinks` has to be 0."""
    if window is None and sinks:
        raise ValueError("sinks are the first tokens that a window leaves visible: they need a window")
    return _RingAttention.apply(q, k, v, n_shards, causal, layout, f32_out, window, sinks)


def _dense(t):
    """t, or a contiguous copy if it is not contiguous or off a 16-byte boundary (a view into a larger tensor)."""
    return t if t.is_contiguous() and t.data_ptr() % 16 == 0 else t.clone(memory_format=torch.contiguous_format)


class _QkNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, wq, wk, n_shards, layout, base, eps, shard, positions):
        q, k = binding.as_rows(q), binding.as_rows(k)
        cfg = dict(n_shards=n_shards, layout=layout, base=base, eps=eps, shard=shard)
        q_out, k_out = binding.qk_norm_rope(q, k, _dense(wq.float()), _dense(wk.float()), positions=positions, **cfg)
        ctx.save_for_backward(q, k, wq, wk, positions)
        ctx.cfg = cfg
        return q_out, k_out

    @staticmethod
    @first_order
    def backward(ctx, dq_out, dk_out):
        q, k, wq, wk, positions = ctx.saved_tensors
        dq, dk, dwq, dwk = binding.qk_norm_rope_bwd(q, k, _dense(wq.float()), _dense(wk.float()),
                                                    _dense(dq_out), _dense(dk_out), positions=positions, **ctx.cfg)
        return dq, dk, dwq.to(wq.dtype), dwk.to(wk.dtype), None, None, None, None, None, None


def ring_qk_norm_rope(q, k, wq, wk, n_shards=1, layout="contiguous", base=10000.0, eps=1e-6, shard=None, positions=None):
    """Norms of every query and key head and the rotation by natural position in one pass, in front of
    ring_attention (or, with `shard`, of one device's ring): differentiable with respect to q [B,H,rows,d],
    k [B,Hkv,rows,d] and the weights wq, wk [d] (any float dtype).  See qk_norm_rope for the arguments; q, k, the
    weights and the outputs' gradients are copied where the calls cannot read them as they lie."""
    return _QkNormRope.apply(q, k, wq, wk, n_shards, layout, base, eps, shard, positions)


class _QkRopeAxes(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, wq, wk, positions, sections, base, eps, spectrum):
        q, k, norm = binding.as_rows(q), binding.as_rows(k), wq is not None
        cfg = dict(base=base, eps=eps, spectrum=spectrum)
        w = (_dense(wq.float()), _dense(wk.float())) if norm else (None, None)
        q_out, k_out = binding.qk_rope_axes(q, k, positions, sections, *w, **cfg)
        ctx.save_for_backward(positions, *((q, k, wq, wk) if norm else ()))
        ctx.cfg, ctx.sections = cfg, sections
        return q_out, k_out

    @staticmethod
    @first_order
    def backward(ctx, dq_out, dk_out):
        positions, *saved = ctx.saved_tensors
        how = dict(ctx.cfg)
        if saved:
            q, k, wq, wk = saved
            how.update(q=q, k=k, wq=_dense(wq.float()), wk=_dense(wk.float()))
        dq, dk, dwq, dwk = binding.qk_rope_axes_bwd(_dense(dq_out), _dense(dk_out), positions, ctx.sections, **how)
        if saved:
            dwq, dwk = dwq.to(wq.dtype), dwk.to(wk.dtype)
        return dq, dk, dwq, dwk, None, None, None, None, None


def ring_qk_rope_axes(q, k, positions, sections, wq=None, wk=None, base=10000.0, eps=1e-6, spectrum="whole"):
    """The rotation of q [B,H,rows,d] and k [B,Hkv,rows,d] by positions with several axes [axes, B, rows] int32, after the
    norms of the heads where their weights wq, wk [d] (any float dtype) are given: differentiable with respect to q, k
    and the weights.  See qk_rope_axes for the arguments; q, k, the weights and the outputs' gradients are copied where the
    calls cannot read them as they lie."""
    if (wq is None) != (wk is None):
        raise ValueError("wq and wk must both be given, or neither")
    return _QkRopeAxes.apply(q, k, wq, wk, positions, tuple(sections), base, eps, spectrum)
