"""Ring attention as a differentiable PyTorch operation.

``ring_attention`` runs the library's forward and, when a gradient is needed, its backward: the
same ``ring_attn_fwd`` / ``ring_attn_bwd`` entry points as ``fwd`` and ``bwd`` in the binding.  The
forward saves its output and log-sum-exp; the backward recomputes the attention weights from them
(nothing quadratic is stored).  Gradients come back in the dtype of the inputs.

With ``f32_out=True`` (bf16 inputs) the forward keeps its output in float32 for the backward
(``ring_attn_fwd_f32out``, then ``ring_attn_f32_convert`` for the returned bf16 output) and the
backward takes D = rowsum(dout * out) from it (``ring_attn_bwd_f32out``) instead of from the rounded
output: twice the saved output's memory, and gradients closer to the exact ones where a gradient is
a short sum of large, cancelling terms (the first positions of a causal sequence).
"""
import torch

from . import binding


class _RingAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, n_shards, causal, layout, f32_out):
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        f32_out = bool(f32_out) and q.dtype != torch.float32
        if f32_out:
            saved, lse = binding.fwd_f32out(q, k, v, n_shards, causal, layout)
            out = binding.f32_convert(saved, q.dtype)
        else:
            out, lse = binding.fwd(q, k, v, n_shards, causal, layout)
            saved = out
        ctx.save_for_backward(q, k, v, saved, lse)
        ctx.cfg = (n_shards, causal, layout, f32_out)
        return out

    @staticmethod
    def backward(ctx, dout):
        q, k, v, saved, lse = ctx.saved_tensors
        n_shards, causal, layout, f32_out = ctx.cfg
        call = binding.bwd_f32out if f32_out else binding.bwd
        dq, dk, dv = call(q, k, v, saved, lse, dout.contiguous(), n_shards, causal, layout, grad_dtype=q.dtype)
        return dq, dk, dv, None, None, None, None


def ring_attention(q, k, v, n_shards, causal=True, layout="zigzag", f32_out=False):
    """Exact attention of q [B,H,L,d] over k, v [B,Hkv,L,d] (sequence axis in the layout's order),
    computed as the ring over n_shards shards; differentiable with respect to q, k and v.
    f32_out: keep the forward's output in float32 for the backward's D (see the module notes)."""
    return _RingAttention.apply(q, k, v, n_shards, causal, layout, f32_out)


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
    @torch.autograd.function.once_differentiable
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
