"""Small angles of the norm with rotation: the rotation of a small negative position is as exact as of a positive one."""
import math

import pytest
import torch

import sequence_sharded_exact_gb300 as ra

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("backward", [False, True])
def test_small_angles_of_either_sign(d, backward):
    """Pairs (1, 0) turned by p base^(-2i/d): the quotient of the turned pair is the angle's tangent whatever the norm.  The
    angle is held as a fraction of a turn in 32 bits (2^-32 turns), then as a float32 and through sinpi and cospi (a few 2^-24
    of itself)."""
    base, pos = 500000.0, [0, 1, -1, 2, -2, 5, -5, 100, -100, 999, -999]
    x = torch.zeros(1, 1, len(pos), d, device=DEV)
    x[..., 0::2] = 1.0
    w = torch.ones(d, device=DEV)
    p = torch.tensor([pos], dtype=torch.int32, device=DEV)
    if not backward:
        y, y2 = ra.qk_norm_rope(x, x, w, w, base=base, positions=p)
        assert torch.equal(y, y2)
    else:  # g = R(-p) dy; a row of zeros: dx = g / sqrt(eps) in float32
        y, y2, _, _ = ra.qk_norm_rope_bwd(torch.zeros_like(x), torch.zeros_like(x), w, w, x, x, base=base, eps=1.0, positions=p)
        assert torch.equal(y, y2)
    y = y[0, 0].cpu().double()
    sign = -1.0 if backward else 1.0
    angle = sign * torch.tensor(pos).double()[:, None] * torch.tensor([base ** (-2.0 * i / d) for i in range(d // 2)], dtype=torch.float64)
    small = angle.abs() < 0.5
    off = (torch.atan2(y[:, 1::2], y[:, 0::2]) - angle).abs() - (2 * math.pi * 2.0 ** -32 + 2.0 ** -21 * angle.abs())
    assert small.sum() > 5 * d // 2
    assert float(off[small].max()) <= 0, f"off by {float(off[small].max()):.3e} beyond its bound"
