"""Norms of queries and keys with the rotation by natural position, and their gradients, against float64."""
import pytest
import torch

import cache_util as cu
import sequence_sharded_exact_gb300 as ra

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BASE, EPS = 500000.0, 1e-6


@pytest.fixture(autouse=True)
def _clean_status():
    torch.cuda.set_device(0)
    ra.device_status()
    yield
    assert ra.device_status() == 0


def _randn(*shape, seed=0, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype).to(DEV)


def _inputs(B, H, Hkv, L, d, dtype, fused, seed):
    if fused:
        x = _randn(B, L, H + 2 * Hkv, d, seed=seed, dtype=dtype)
        q, k, _ = (t.transpose(1, 2) for t in x.split([H, Hkv, Hkv], dim=2))
    else:
        q, k = _randn(B, H, L, d, seed=seed, dtype=dtype), _randn(B, Hkv, L, d, seed=seed + 1, dtype=dtype)
    w = [1 + 0.2 * _randn(d, seed=seed + i) for i in (2, 3)]
    return q, k, *w


def _assert_rows(got, ref, dtype, what):
    """One rounding to dtype, and float32 arithmetic: the angle is off by at most 2^-24 turns (4e-7), norms and
    products by a few 2^-24: 2e-6 of the pair's length."""
    got = got.detach().cpu().double()
    pair = ref.unflatten(-1, (-1, 2)).norm(dim=-1, keepdim=True).expand(*ref.shape[:-1], ref.shape[-1] // 2, 2).flatten(-2)
    over = (got - ref).abs() - (cu.EPS2[dtype] * 1.01 * ref.abs() + 2e-6 * pair + 1e-30)
    assert float(over.max()) <= 0, f"{what}: off by {float(over.max()):.3e} beyond its bound"


CASES = [
    # B, H, Hkv, L, d, n, layout, dtype, fused
    (1, 4, 2, 64, 128, 4, "zigzag", torch.bfloat16, False),
    (2, 6, 2, 1235, 64, 5, "striped", torch.float32, True),
    (1, 1, 1, 1, 64, 1, "contiguous", torch.float32, False),
    (3, 8, 1, 7, 128, 1, "contiguous", torch.bfloat16, True),
    (1, 40, 8, 33, 128, 1, "contiguous", torch.float32, False),
    (1, 5, 5, 4098, 64, 3, "zigzag", torch.bfloat16, True),
]


@pytest.mark.parametrize("B,H,Hkv,L,d,n,layout,dtype,fused", CASES)
def test_forward_and_backward_against_float64(B, H, Hkv, L, d, n, layout, dtype, fused):
    q, k, wq, wk = _inputs(B, H, Hkv, L, d, dtype, fused, seed=L)
    pos = cu.natural(L, n, layout)
    yq, yk = ra.qk_norm_rope(q, k, wq, wk, n, layout, base=BASE, eps=EPS)
    assert yq.is_contiguous() and yk.is_contiguous() and yq.dtype == dtype
    _assert_rows(yq, cu.norm_rope(q, wq, pos, BASE, EPS), dtype, "q")
    _assert_rows(yk, cu.norm_rope(k, wk, pos, BASE, EPS), dtype, "k")
    dyq, dyk = _randn(B, H, L, d, seed=5, dtype=dtype), _randn(B, Hkv, L, d, seed=6, dtype=dtype)
    dq, dk, dwq, dwk = ra.qk_norm_rope_bwd(q, k, wq, wk, dyq, dyk, n, layout, base=BASE, eps=EPS)
    for x, w, dy, dx, dw, what in ((q, wq, dyq, dq, dwq, "q"), (k, wk, dyk, dk, dwk, "k")):
        r_dx, r_dw, mag = cu.norm_rope_bwd(x, w, dy, pos, BASE, EPS)
        # dx: its rounding; its two terms are of the size of the gradient row / the norm, in float32 with sums of d
        row = r_dx.norm(dim=-1, keepdim=True) + (dy.cpu().double().norm(dim=-1, keepdim=True)
                                                 / x.cpu().double().norm(dim=-1, keepdim=True)) * d ** 0.5
        over = (dx.cpu().double() - r_dx).abs() - (cu.EPS2[dtype] * 1.01 * r_dx.abs() + 4e-6 * row)
        assert float(over.max()) <= 0, f"d{what}: off by {float(over.max()):.3e} beyond its bound"
        # dw: a lane adds at most rows / 64 + 40 terms in a row, then blocks of at most 32: below 2^-24 * 512 of the magnitudes
        assert bool(((dw.cpu().double() - r_dw).abs() <= 2.0 ** -15 * mag + 1e-30).all()), f"dw{what}"


def test_every_split_of_heads_gives_the_same_rows():
    """A batch too small to fill the SMs shares a position's heads out over groups; a large one does not."""
    H, Hkv, d = 32, 8, 128
    q, k, wq, wk = _inputs(1, H, Hkv, 2048, d, torch.bfloat16, False, seed=3)
    pos = torch.arange(2048, dtype=torch.int32, device=DEV)[None]
    big = ra.qk_norm_rope(q, k, wq, wk, positions=pos)
    for rows in (1, 3, 64):
        part = ra.qk_norm_rope(q[:, :, 7:7 + rows], k[:, :, 7:7 + rows], wq, wk, positions=pos[:, 7:7 + rows].contiguous())
        for a, b in zip(part, big):
            assert torch.equal(a, b[:, :, 7:7 + rows])


def test_positions_and_shards_name_the_same_rotation():
    B, H, Hkv, L, d, n = 2, 4, 2, 96, 64, 4
    q, k, wq, wk = _inputs(B, H, Hkv, L, d, torch.float32, False, seed=11)
    for layout in ("contiguous", "zigzag", "striped"):
        whole = ra.qk_norm_rope(q, k, wq, wk, n, layout)
        pos = cu.natural(L, n, layout).to(torch.int32).to(DEV).expand(B, L).contiguous()
        for a, b in zip(ra.qk_norm_rope(q, k, wq, wk, positions=pos), whole):
            assert torch.equal(a, b)
        S = L // n
        for i in range(n):
            s = slice(i * S, (i + 1) * S)
            for a, b in zip(ra.qk_norm_rope(q[:, :, s], k[:, :, s], wq, wk, n, layout, shard=i), whole):
                assert torch.equal(a, b[:, :, s])
    # after a weight of one and unit norms, the rotation is ring_attn_rope's
    u = (q / q.square().mean(-1, keepdim=True).sqrt()).contiguous()
    a, _ = ra.qk_norm_rope(u, k, torch.ones(d, device=DEV), wk, n, "zigzag", eps=0.0)
    assert torch.allclose(a, ra.rope(u.clone(), n, "zigzag"), atol=4e-6, rtol=0)


def test_far_and_negative_positions():
    q, k, wq, wk = _inputs(1, 2, 2, 6, 128, torch.float32, False, seed=13)
    pos = torch.tensor([[0, 1, -1, 2 ** 31 - 1, -2 ** 31, 1234567890]], dtype=torch.int32, device=DEV)
    y, _ = ra.qk_norm_rope(q, k, wq, wk, positions=pos, base=10000.0)
    _assert_rows(y, cu.norm_rope(q, wq, pos.cpu()[:, None, :], 10000.0, 1e-6), torch.float32, "far")


def test_zero_rows_in_place_and_repeated_rows():
    q, k, wq, wk = _inputs(1, 4, 2, 10, 128, torch.bfloat16, False, seed=17)
    q[0, 1, 3] = 0
    ref = ra.qk_norm_rope(q, k, wq, wk, eps=1e-5)
    assert bool((ref[0][0, 1, 3] == 0).all()) and bool(torch.isfinite(ref[0].float()).all())
    q2, k2 = q.clone(), k.clone()
    out = ra.qk_norm_rope(q2, k2, wq, wk, eps=1e-5, q_out=q2, k_out=k2)
    assert out[0] is q2 and torch.equal(q2, ref[0]) and torch.equal(k2, ref[1])
    wide = ra.qk_norm_rope(q[:, :1].expand(1, 4, 10, 128), k[:, :1], wq, wk)  # stride 0 along the heads
    for h in range(1, 4):
        assert torch.equal(wide[0][:, h], wide[0][:, 0])
    dy = _randn(1, 4, 10, 128, seed=1, dtype=torch.bfloat16)
    dk = _randn(1, 2, 10, 128, seed=2, dtype=torch.bfloat16)
    ref = ra.qk_norm_rope_bwd(q, k, wq, wk, dy, dk)
    got = ra.qk_norm_rope_bwd(q, k, wq, wk, dy, dk, dq=dy, dk=dk)  # over the gradients it reads
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    again = ra.qk_norm_rope_bwd(q, k, wq, wk, *(_randn(1, h, 10, 128, seed=s, dtype=torch.bfloat16) for h, s in ((4, 1), (2, 2))))
    assert all(torch.equal(a, b) for a, b in zip(again, ref))


@pytest.mark.parametrize("wdtype", [torch.float32, torch.bfloat16])
def test_autograd_against_differences_and_the_formula(wdtype):
    """The differentiable form in front of the ring: gradients of a scalar against central differences of the
    float64 statement along random directions, and against the backward call's."""
    B, H, Hkv, L, d, n = 1, 4, 2, 24, 64, 2
    x = _randn(B, L, H + 2 * Hkv, d, seed=23).requires_grad_()
    wq, wk = ((1 + 0.2 * _randn(d, seed=s)).to(wdtype).requires_grad_() for s in (24, 25))
    cq, ck = _randn(B, H, L, d, seed=26), _randn(B, Hkv, L, d, seed=27)

    def loss64(x64, wq64, wk64):
        pos = cu.natural(L, n, "zigzag")
        q, k, _ = (t.transpose(1, 2) for t in x64.split([H, Hkv, Hkv], dim=2))
        return float((cu.norm_rope(q, wq64, pos, 1e4, 1e-6) * cq.cpu().double()).sum()
                     + (cu.norm_rope(k, wk64, pos, 1e4, 1e-6) * ck.cpu().double()).sum())

    q, k, _ = (t.transpose(1, 2) for t in x.split([H, Hkv, Hkv], dim=2))
    yq, yk = ra.ring_qk_norm_rope(q, k, wq, wk, n, "zigzag")
    ((yq * cq).sum() + (yk * ck).sum()).backward()
    at = [t.detach().cpu().double() for t in (x, wq, wk)]
    for i, (leaf, seed) in enumerate(((x, 31), (wq, 32), (wk, 33))):
        u = torch.randn(at[i].shape, generator=torch.Generator().manual_seed(seed)).double()
        h = 1e-4
        up, down = [t.clone() for t in at], [t.clone() for t in at]
        up[i] += h * u
        down[i] -= h * u
        diff = (loss64(*up) - loss64(*down)) / (2 * h)
        got = float((leaf.grad.cpu().double() * u).sum())
        scale = float(leaf.grad.cpu().double().norm() * u.norm())
        # differences: h^2 times third derivatives (1e-6); gradients: float32 sums, bf16 weights' gradients rounded
        assert abs(got - diff) <= scale * (cu.EPS2[wdtype] + 1e-5), (i, got, diff)
    assert x.grad[:, :, H + Hkv:].abs().max() == 0 and wq.grad.dtype == wdtype


def test_one_output_unused_and_double_backward_refused():
    q, k, wq, wk = _inputs(1, 2, 1, 8, 64, torch.float32, False, seed=41)
    for t in (q, k, wq, wk):
        t.requires_grad_()
    yq, _ = ra.ring_qk_norm_rope(q, k, wq, wk)
    yq.sum().backward()
    assert bool((k.grad == 0).all()) and bool((wk.grad == 0).all()) and bool(q.grad.abs().sum() > 0)
    yq, _ = ra.ring_qk_norm_rope(q, k, wq, wk)
    g, = torch.autograd.grad(yq.sum(), q, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_captured_and_replayed_on_another_stream():
    q, k, wq, wk = _inputs(1, 4, 2, 32, 128, torch.bfloat16, False, seed=51)
    q2, k2, *_ = _inputs(1, 4, 2, 32, 128, torch.bfloat16, False, seed=52)
    dq, dk = torch.randn_like(q), torch.randn_like(k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ra.qk_norm_rope(q, k, wq, wk)
        ra.qk_norm_rope_bwd(q, k, wq, wk, dq, dk)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ra.qk_norm_rope(q, k, wq, wk)
        g = ra.qk_norm_rope_bwd(q, k, wq, wk, dq, dk)
    q.copy_(q2)
    k.copy_(k2)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip((*y, *g), (*ra.qk_norm_rope(q, k, wq, wk), *ra.qk_norm_rope_bwd(q, k, wq, wk, dq, dk))):
        assert torch.equal(a, b)
