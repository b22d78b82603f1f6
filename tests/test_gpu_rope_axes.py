"""The rotation by positions with several axes, after the norms of the heads or alone, and its gradients, against float64."""
import pytest
import torch

import cache_util as cu
import sequence_sharded_exact_gb300 as ra
from sequence_sharded_exact_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
BASE, EPS = 10000.0, 1e-6


@pytest.fixture(autouse=True)
def _clean_status():
    torch.cuda.set_device(0)
    ra.device_status()
    yield
    assert ra.device_status() == 0


def _randn(*shape, seed=0, dtype=F32):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


def _inputs(B, H, Hkv, rows, d, axes, dtype, fused, norm, seed, far=1 << 18):
    if fused:
        x = _randn(B, rows, H + 2 * Hkv, d, seed=seed, dtype=dtype)
        q, k, _ = (t.transpose(1, 2) for t in x.split([H, Hkv, Hkv], dim=2))
    else:
        q, k = _randn(B, H, rows, d, seed=seed, dtype=dtype), _randn(B, Hkv, rows, d, seed=seed + 1, dtype=dtype)
    w = [1 + 0.2 * _randn(d, seed=seed + i) for i in (2, 3)] if norm else [None, None]
    pos = torch.randint(-far, far, (axes, B, rows), generator=torch.Generator().manual_seed(seed + 4)).to(torch.int32).to(DEV)
    return q, k, *w, pos


def _angles(pos, sections, spectrum, d):
    """[B, 1, rows, d/2] in float64."""
    out, i = [], 0
    for a, m in enumerate(sections):
        for u in range(m):
            out.append(pos[a].cpu().double() * BASE ** (-(2.0 * i / d if spectrum == "whole" else u / m)))
            i += 1
    return torch.stack(out, -1)[:, None]


def _turn(x, angle):
    z = torch.view_as_complex(x.unflatten(-1, (-1, 2)).contiguous()) * torch.polar(torch.ones_like(angle), angle)
    return torch.view_as_real(z).flatten(-2)


def _ref(x, w, angle):
    x = x.detach().cpu().double()
    if w is not None:
        x = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * w.cpu().double()
    return _turn(x, angle)


def _assert_rows(got, ref, dtype, what):
    """As of qk_norm_rope: one rounding to dtype, the angle off by at most 2^-24 turns, norms and products by a few 2^-24."""
    got = got.detach().cpu().double()
    pair = ref.unflatten(-1, (-1, 2)).norm(dim=-1, keepdim=True).expand(*ref.shape[:-1], ref.shape[-1] // 2, 2).flatten(-2)
    over = (got - ref).abs() - (cu.EPS2[dtype] * 1.01 * ref.abs() + 2e-6 * pair + 1e-30)
    assert float(over.max()) <= 0, f"{what}: off by {float(over.max()):.3e} beyond its bound"


CASES = [
    # B, H, Hkv, rows, d, sections, spectrum, dtype, fused
    (1, 4, 2, 64, 128, (16, 24, 24), "whole", BF, False),
    (2, 6, 2, 1235, 64, (8, 12, 12), "axis", F32, True),
    (1, 1, 1, 1, 64, (32,), "whole", F32, False),
    (3, 8, 1, 7, 128, (1, 62, 1), "axis", BF, True),
    (1, 40, 8, 33, 128, (22, 21, 21), "whole", F32, False),     # axes that change inside a lane's pairs
    (1, 5, 5, 4098, 64, (9, 0, 13, 10), "axis", BF, True),      # an axis without pairs
    (2, 32, 8, 700, 128, (0, 64), "whole", BF, False),
]


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("B,H,Hkv,rows,d,sections,spectrum,dtype,fused", CASES)
def test_forward_and_backward_against_float64(B, H, Hkv, rows, d, sections, spectrum, dtype, fused, norm):
    q, k, wq, wk, pos = _inputs(B, H, Hkv, rows, d, len(sections), dtype, fused, norm, seed=rows)
    angle = _angles(pos, sections, spectrum, d)
    how = dict(base=BASE, eps=EPS, spectrum=spectrum)
    yq, yk = ra.qk_rope_axes(q, k, pos, sections, wq, wk, **how)
    assert yq.is_contiguous() and yk.is_contiguous() and yq.dtype == dtype
    _assert_rows(yq, _ref(q, wq, angle), dtype, "q")
    _assert_rows(yk, _ref(k, wk, angle), dtype, "k")
    dyq, dyk = _randn(B, H, rows, d, seed=5, dtype=dtype), _randn(B, Hkv, rows, d, seed=6, dtype=dtype)
    dq, dk, dwq, dwk = ra.qk_rope_axes_bwd(dyq, dyk, pos, sections, q=q if norm else None, k=k if norm else None, wq=wq, wk=wk, **how)
    if not norm:
        assert dwq is None and dwk is None
        _assert_rows(dq, _turn(dyq.cpu().double(), -angle), dtype, "dq")
        _assert_rows(dk, _turn(dyk.cpu().double(), -angle), dtype, "dk")
        return
    for x, w, dy, dx, dw, what in ((q, wq, dyq, dq, dwq, "q"), (k, wk, dyk, dk, dwk, "k")):
        x64, g = x.cpu().double(), _turn(dy.cpu().double(), -angle)
        r = (x64.square().mean(-1, keepdim=True) + EPS).rsqrt()
        u = g * w.cpu().double()
        r_dx = r * (u - x64 * r * r * (u * x64).mean(-1, keepdim=True))
        # dx and dw: the bounds of qk_norm_rope_bwd's test
        row = r_dx.norm(dim=-1, keepdim=True) + dy.cpu().double().norm(dim=-1, keepdim=True) / x64.norm(dim=-1, keepdim=True) * d ** 0.5
        over = (dx.cpu().double() - r_dx).abs() - (cu.EPS2[dtype] * 1.01 * r_dx.abs() + 4e-6 * row)
        assert float(over.max()) <= 0, f"d{what}: off by {float(over.max()):.3e} beyond its bound"
        mag = (g * x64 * r).abs().sum((0, 1, 2))
        assert bool(((dw.cpu().double() - (g * x64 * r).sum((0, 1, 2))).abs() <= 2.0 ** -15 * mag + 1e-30).all()), f"dw{what}"


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128])
def test_one_axis_is_the_rotation_by_positions(d, dtype):
    """One axis, or several with the same positions: bit for bit qk_norm_rope with these positions, and its gradients."""
    q, k, wq, wk, pos = _inputs(2, 4, 2, 50, d, 1, dtype, True, True, seed=3)
    ref = ra.qk_norm_rope(q, k, wq, wk, base=BASE, positions=pos[0])
    dyq, dyk = torch.randn_like(ref[0]), torch.randn_like(ref[1])
    gref = ra.qk_norm_rope_bwd(q, k, wq, wk, dyq, dyk, base=BASE, positions=pos[0])
    for axes, sections in ((1, (d // 2,)), (3, (d // 8, d // 4, d // 8)), (4, (1, d // 2 - 3, 1, 1))):
        p = pos.expand(axes, 2, 50).contiguous()
        assert all(torch.equal(a, b) for a, b in zip(ra.qk_rope_axes(q, k, p, sections, wq, wk, base=BASE), ref))
        got = ra.qk_rope_axes_bwd(dyq, dyk, p, sections, q=q, k=k, wq=wq, wk=wk, base=BASE)
        assert all(torch.equal(a, b) for a, b in zip(got, gref))


def test_far_positions():
    ends = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 1234567890], dtype=torch.int32)
    pos = torch.stack((ends, ends.flip(0), ends.roll(2)))[:, None].contiguous().to(DEV)
    q, k, _, _, _ = _inputs(1, 2, 2, 6, 128, 3, F32, False, False, seed=13)
    for spectrum in ("whole", "axis"):
        y, _ = ra.qk_rope_axes(q, k, pos, (16, 24, 24), base=BASE, spectrum=spectrum)
        _assert_rows(y, _ref(q, None, _angles(pos, (16, 24, 24), spectrum, 128)), F32, spectrum)


def test_tables_of_two_programs_in_turn():
    """Calls of different bases, sections and spectra after one another."""
    q, k, _, _, pos = _inputs(1, 2, 1, 9, 64, 2, F32, False, False, seed=2)
    hows = [((16, 16), "axis"), ((10, 22), "axis"), ((16, 16), "whole"), ((16, 16), "axis"), ((10, 22), "whole")]
    for sections, spectrum in hows * 2:
        y, _ = ra.qk_rope_axes(q, k, pos, sections, base=BASE, spectrum=spectrum)
        _assert_rows(y, _ref(q, None, _angles(pos, sections, spectrum, 64)), F32, f"{sections} {spectrum}")


@pytest.mark.parametrize("norm", [True, False])
def test_in_place_and_given_outputs(norm):
    q, k, wq, wk, pos = _inputs(2, 4, 2, 30, 128, 3, BF, False, norm, seed=6)
    sec = (16, 24, 24)
    ref = ra.qk_rope_axes(q, k, pos, sec, wq, wk)
    dyq, dyk = torch.randn_like(q), torch.randn_like(k)
    have = dict(q=q, k=k, wq=wq, wk=wk) if norm else {}
    gref = ra.qk_rope_axes_bwd(dyq, dyk, pos, sec, **have)
    g1, g2 = dyq.clone(), dyk.clone()
    got = ra.qk_rope_axes_bwd(g1, g2, pos, sec, dq=g1, dk=g2, **have)
    assert got[0] is g1 and torch.equal(g1, gref[0]) and torch.equal(g2, gref[1])
    q2, k2 = q.clone(), k.clone()
    got = ra.qk_rope_axes(q2, k2, pos, sec, wq, wk, q_out=q2, k_out=k2)
    assert got[0] is q2 and torch.equal(q2, ref[0]) and torch.equal(k2, ref[1])


@pytest.mark.parametrize("norm", [True, False])
def test_another_stream_and_a_replayed_graph(norm):
    q, k, wq, wk, pos = _inputs(1, 8, 2, 500, 64, 3, BF, True, norm, seed=6)
    sec = (8, 12, 12)
    ref = ra.qk_rope_axes(q, k, pos, sec, wq, wk)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = ra.qk_rope_axes(q, k, pos, sec, wq, wk, stream=s)
    back = ra.qk_rope_axes_bwd(*got, pos, sec, stream=s) if not norm else None
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    if not norm:
        assert all(torch.equal(a, b) for a, b in zip(back[:2], ra.qk_rope_axes_bwd(*ref, pos, sec)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = ra.qk_rope_axes(q, k, pos, sec, wq, wk)
    pos.add_(17)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, ra.qk_rope_axes(q, k, pos, sec, wq, wk)))


@pytest.mark.parametrize("wdtype", [F32, BF])
def test_autograd(wdtype):
    q, k, wq, wk, pos = _inputs(2, 4, 2, 20, 64, 2, F32, True, True, seed=8)
    wq, wk = wq.to(wdtype), wk.to(wdtype)
    leaves = [x.detach().clone().requires_grad_() for x in (q, k, wq, wk)]
    yq, yk = ra.ring_qk_rope_axes(leaves[0].transpose(1, 2).contiguous().transpose(1, 2), leaves[1], pos, [12, 20], leaves[2], leaves[3], spectrum="axis")
    gq, gk = _randn(*yq.shape, seed=1), _randn(*yk.shape, seed=2)
    (yq * gq).sum().backward(retain_graph=True)  # one output alone
    first = [None if x.grad is None else x.grad.clone() for x in leaves]
    (yk * gk).sum().backward()
    got = ra.qk_rope_axes_bwd(gq, gk, pos, (12, 20), q=q, k=k, wq=wq.float(), wk=wk.float(), spectrum="axis")
    for x, r in zip(leaves, got):
        assert x.grad.dtype == x.dtype
        assert torch.allclose(x.grad.float(), r, rtol=2.0 ** -7 if x.dtype == BF else 1e-6, atol=1e-6)
    assert float(first[1].abs().max()) == 0 and float(first[3].float().abs().max()) == 0
    yq, yk = ra.ring_qk_rope_axes(leaves[0], leaves[1], pos, (12, 20))
    dq, dk = torch.autograd.grad((yq * gq).sum() + (yk * gk).sum(), leaves[:2])
    assert all(torch.equal(a, b) for a, b in zip((dq, dk), ra.qk_rope_axes_bwd(gq, gk, pos, (12, 20))[:2]))


def test_gradients_against_differences():
    q, k, wq, wk, pos = _inputs(1, 2, 1, 5, 64, 3, F32, False, True, seed=18, far=1000)
    sec, h = (8, 12, 12), 1e-5
    angle = _angles(pos, sec, "whole", 64)
    dy = _randn(1, 2, 5, 64, seed=1)
    dq, _, dwq, _ = ra.qk_rope_axes_bwd(dy, _randn(1, 1, 5, 64, seed=2), pos, sec, q=q, k=k, wq=wq, wk=wk, base=BASE, eps=EPS)
    g = torch.Generator().manual_seed(3)
    for got, which in ((dq, 0), (dwq, 1)):
        step = torch.randn(got.shape, generator=g, dtype=torch.float64)
        val = []
        for sign in (h, -h):
            x, w = q.cpu().double() + sign * step * (which == 0), wq.cpu().double() + sign * step * (which == 1) if which else wq.cpu().double()
            val.append((_ref(x, w, angle) * dy.cpu().double()).sum())
        # the quotient is off by h^2 and by float64 roundings over h; the gradient by its float32 sums
        have = got.cpu().double() * step
        assert abs(float(val[0] - val[1]) / (2 * h) - float(have.sum())) <= 2e-5 * float(have.abs().sum())


def test_compiled_and_python_forms_refuse_and_answer_alike():
    q, k, wq, wk, pos = _inputs(1, 4, 2, 8, 64, 3, BF, False, True, seed=1)
    s = torch.cuda.current_stream()
    sec = (8, 12, 12)
    for kw in (dict(), dict(wq=wq, wk=wk), dict(spectrum="axis"), dict(base=500000, eps=0)):
        a, b = ra.qk_rope_axes(q, k, pos, sec, **kw), ra.qk_rope_axes(q, k, pos, list(sec), stream=s, **kw)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    for err, args, kw in [(ValueError, (q, k, pos[:2], sec), {}), (ValueError, (q, k, pos.long(), sec), {}), (ValueError, (q, k, pos, sec), dict(wq=wq)),
                          (ValueError, (q, k, pos, sec), dict(spectrum="each")), (binding.RingAttnError, (q, k, pos, (8, 12, 11)), {}),
                          (binding.RingAttnError, (q, k, pos, (33, -1, 0)), {}), (ValueError, (q, k, pos, (4,) * 5), {}),
                          (TypeError, (q, k, pos, (8, 12, 12.0)), {}), (ValueError, (q, k.float(), pos, sec), {}),
                          (ValueError, (q, k[:, :, :4], pos, sec), {}), (binding.RingAttnError, (q, k, pos, sec), dict(base=-1.0))]:
        for stream in (None, s):
            with pytest.raises(err):
                ra.qk_rope_axes(*args, stream=stream, **kw)
    with pytest.raises(ValueError):
        ra.qk_rope_axes_bwd(q, k, pos, sec, q=q, k=k)
    with pytest.raises(ValueError):
        ra.ring_qk_rope_axes(q, k, pos, sec, wq=wq)
