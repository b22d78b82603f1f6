"""The differentiable norm with rotation takes what a program hands it: gradients and weights that lie anywhere."""
import pytest
import torch

import sequence_sharded_exact_gb300 as ra

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _randn(*shape, seed, dtype=torch.float32):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradients_that_lie_off_16_byte_boundaries(dtype):
    """The outputs' gradients are views of a larger one's, one element in: autograd hands them on where they lie."""
    B, H, Hkv, L, d = 1, 4, 2, 6, 64
    w = [_randn(d, seed=s) for s in (1, 2)]
    g = _randn(1 + B * (H + Hkv) * L * d, seed=3, dtype=dtype)
    grads = []
    for odd in (False, True):
        q, k = (_randn(B, h, L, d, seed=4 + h, dtype=dtype).requires_grad_() for h in (H, Hkv))
        yq, yk = ra.ring_qk_norm_rope(q, k, *w)
        if odd:
            lead = torch.zeros(1, dtype=dtype, device=DEV, requires_grad=True)
            torch.cat([lead, yq.flatten(), yk.flatten()]).backward(g)
        else:
            n = yq.numel()
            torch.autograd.backward([yq, yk], [g[1:1 + n].clone().view_as(yq), g[1 + n:].clone().view_as(yk)])
        grads.append((q.grad, k.grad))
    assert all(torch.equal(a, b) for a, b in zip(*grads))


def test_weights_that_are_slices_of_a_flat_parameter():
    B, H, Hkv, L, d = 2, 4, 2, 6, 64
    flat = _randn(2 * d + 1, seed=1).requires_grad_()
    q, k = (_randn(B, h, L, d, seed=4 + h) for h in (H, Hkv))
    y = ra.ring_qk_norm_rope(q, k, flat[1:1 + d], flat[1 + d:])
    sum(t.square().sum() for t in y).backward()
    whole = [flat.detach()[1:1 + d].clone().requires_grad_(), flat.detach()[1 + d:].clone().requires_grad_()]
    ref = ra.ring_qk_norm_rope(q, k, *whole)
    sum(t.square().sum() for t in ref).backward()
    assert all(torch.equal(a, b) for a, b in zip(y, ref))
    assert torch.equal(flat.grad[1:], torch.cat([t.grad for t in whole])) and float(flat.grad[0]) == 0
