"""Norms with rotation and their gradients where positions alone fill the GPU, so that a position's heads are not shared out."""
import pytest
import torch

import cache_util as cu
import sequence_sharded_exact_gb300 as ra
from test_gpu_norm_rope import _assert_rows

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _clean_status():
    torch.cuda.set_device(0)
    ra.device_status()
    yield
    assert ra.device_status() == 0


def _randn(*shape, seed, dtype=F32):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 128), (F32, 64)])
@pytest.mark.parametrize("H,Hkv,fused", [(2, 1, False), (6, 2, True)])
def test_positions_that_fill_the_gpu(dtype, d, H, Hkv, fused):
    lanes = d * (2 if dtype == BF else 4) // 16  # of a row: 1024 threads per SM take this many positions at a time
    L = torch.cuda.get_device_properties(0).multi_processor_count * 1024 // lanes + 77
    if fused:
        x = _randn(1, L, H + 2 * Hkv, d, seed=1, dtype=dtype)
        q, k, _ = (t.transpose(1, 2) for t in x.split([H, Hkv, Hkv], dim=2))
    else:
        q, k = _randn(1, H, L, d, seed=1, dtype=dtype), _randn(1, Hkv, L, d, seed=2, dtype=dtype)
    wq, wk = (1 + 0.2 * _randn(d, seed=s) for s in (3, 4))
    pos = torch.randperm(L, generator=torch.Generator().manual_seed(5)).to(torch.int32)[None].to(DEV)
    y = ra.qk_norm_rope(q, k, wq, wk, positions=pos)
    dy = [_randn(1, h, L, d, seed=6 + h, dtype=dtype) for h in (H, Hkv)]
    grads = ra.qk_norm_rope_bwd(q, k, wq, wk, *dy, positions=pos)
    again = ra.qk_norm_rope_bwd(q, k, wq, wk, *dy, positions=pos)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))
    for i, (x, w, what) in enumerate(((q, wq, "q"), (k, wk, "k"))):
        _assert_rows(y[i], cu.norm_rope(x, w, pos[:, None].cpu(), 1e4, 1e-6), dtype, what)
        r_dx, r_dw, mag = cu.norm_rope_bwd(x, w, dy[i], pos[:, None].cpu(), 1e4, 1e-6)
        row = r_dx.norm(dim=-1, keepdim=True) + (dy[i].cpu().double().norm(dim=-1, keepdim=True)
                                                 / x.cpu().double().norm(dim=-1, keepdim=True)) * d ** 0.5
        over = (grads[i].cpu().double() - r_dx).abs() - (cu.EPS2[dtype] * 1.01 * r_dx.abs() + 4e-6 * row)
        assert float(over.max()) <= 0, f"d{what}: off by {float(over.max()):.3e} beyond its bound"
        # dw: a lane adds the heads of at most a few positions in a row, a block 32 lanes' sums, then 320 blocks': below 2^-24 * 512
        assert bool(((grads[2 + i].cpu().double() - r_dw).abs() <= 2.0 ** -15 * mag + 1e-30).all()), f"dw{what}"
    # the same rows in a call of few positions, whose heads are shared out
    for at in (slice(0, 5), slice(L - 90, L)):
        few = ra.qk_norm_rope(q[:, :, at], k[:, :, at], wq, wk, positions=pos[:, at].contiguous())
        assert all(torch.equal(a, b[:, :, at]) for a, b in zip(few, y))
        few = ra.qk_norm_rope_bwd(q[:, :, at], k[:, :, at], wq, wk, *(t[:, :, at].contiguous() for t in dy), positions=pos[:, at].contiguous())
        assert all(torch.equal(a, b[:, :, at]) for a, b in zip(few[:2], grads[:2]))
