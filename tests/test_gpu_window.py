"""Attention through a window with sinks, forward and backward, against float64: every layout, lengths that no tile
divides, windows from one token to more than the sequence, sinks from none to all, both dtypes and head dims."""
import math

import pytest
import torch

import cache_util as cu
import sequence_sharded_exact_gb300 as ra
import window_util as wu

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
WEIGHT_EPS = {BF: 2.0 ** -8, F32: 0.0}  # weights and dS are held in bfloat16 for the tensor cores' products


@pytest.fixture(autouse=True)
def _clean_status():
    torch.cuda.set_device(0)
    ra.device_status()
    yield
    assert ra.device_status() == 0


def _inputs(B, H, Hkv, L, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn((B, h, L, d), generator=g).to(dtype).to(DEV) for h in (H, Hkv, Hkv, H)]


def _check(q, k, v, dout, n, layout, W, S, causal, out_dtype=None, grad_dtype=F32, what=""):
    out, lse = ra.window_fwd(q, k, v, n, W, S, causal, layout, out_dtype=out_dtype)
    assert out.dtype == (out_dtype or q.dtype) and lse.dtype == F32
    cu.check_tree((out, lse), wu.fwd(q, k, v, n, layout, W, S, causal), WEIGHT_EPS[q.dtype], out.dtype, what)
    got = ra.window_bwd(q, k, v, out, lse, dout, n, W, S, causal, layout, grad_dtype=grad_dtype)
    assert all(x.dtype == grad_dtype for x in got)
    wu.check_bwd(got, wu.bwd(q, k, v, out, lse, dout, n, layout, W, S, causal, WEIGHT_EPS[q.dtype]), what)
    return out, lse, got


CASES = [
    # B, H, Hkv, L, d, n, layout, window, sinks, causal
    (1, 1, 1, 1, 64, 1, "contiguous", 1, 0, True),
    (1, 2, 1, 2, 128, 1, "contiguous", 1, 1, True),
    (2, 4, 2, 63, 64, 1, "contiguous", 7, 0, True),
    (1, 4, 1, 64, 128, 2, "zigzag", 64, 4, True),
    (1, 2, 2, 129, 128, 1, "contiguous", 128, 0, True),
    (2, 3, 1, 257, 64, 1, "contiguous", 1, 3, True),             # the token itself and three sinks
    (1, 8, 2, 1000, 128, 5, "contiguous", 100, 4, True),
    (1, 8, 2, 1000, 64, 5, "striped", 130, 70, True),            # sinks of more than a tile, a stripe that 128 does not divide into
    (1, 4, 2, 1024, 128, 4, "zigzag", 200, 0, True),             # chunks of 128
    (1, 4, 4, 1024, 64, 8, "striped", 333, 5, True),
    (1, 6, 2, 924, 128, 2, "zigzag", 50, 9, True),               # chunks of 231
    (1, 2, 1, 896, 128, 128, "striped", 127, 1, True),
    (1, 5, 1, 770, 64, 7, "striped", 129, 300, True),            # more sinks than the window
    (1, 2, 1, 500, 128, 1, "contiguous", 500, 0, True),          # the whole sequence
    (1, 2, 1, 500, 64, 2, "zigzag", 100000, 9, True),
    (1, 2, 1, 400, 64, 1, "contiguous", 3, 1000, True),          # all tokens are sinks
    (1, 4, 2, 700, 128, 1, "contiguous", 60, 0, False),
    (2, 4, 2, 640, 64, 5, "striped", 1, 0, False),               # every token alone
    (1, 4, 1, 512, 128, 2, "zigzag", 129, 6, False),
    (1, 3, 3, 300, 64, 1, "contiguous", 2000, 5, False),
    (1, 2, 1, 1300, 128, 1, "contiguous", 640, 130, False),
    (1, 16, 2, 1536, 64, 2, "contiguous", 256, 128, True),       # everything on tile borders
    (1, 1, 1, 1537, 128, 1, "contiguous", 257, 129, True),
]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("B,H,Hkv,L,d,n,layout,W,S,causal", CASES)
def test_against_float64(B, H, Hkv, L, d, n, layout, W, S, causal, dtype):
    x = _inputs(B, H, Hkv, L, d, dtype, seed=L + W)
    _check(*x, n, layout, W, S, causal)


@pytest.mark.parametrize("dtype,out_dtype,grad_dtype", [(BF, BF, BF), (BF, F32, F32), (BF, F32, BF), (F32, F32, BF)])
@pytest.mark.parametrize("layout,n", [("contiguous", 1), ("striped", 4), ("zigzag", 3)])
def test_output_and_gradient_types(layout, n, dtype, out_dtype, grad_dtype):
    _check(*_inputs(1, 4, 2, 768, 128, dtype, seed=3), n, layout, 150, 5, True, out_dtype=out_dtype, grad_dtype=grad_dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("scale", [8.0, 2.0 ** -20])
def test_large_and_small_scores(scale, dtype):
    """Maxima that grow along the window, rows that one key dominates, and scores that are all alike."""
    q, k, v, dout = _inputs(1, 2, 1, 600, 128, dtype, seed=11)
    k = (k.float() * torch.linspace(0.1, 1.0, 600, device=DEV)[:, None]).to(dtype)
    _check((q.float() * scale).to(dtype), k, v, dout, 1, "contiguous", 260, 3, True)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_no_window_is_ring_attention(causal, d, dtype):
    """A window of the sequence's length against ring_attn_fwd and ring_attn_bwd."""
    q, k, v, dout = _inputs(1, 4, 2, 1024, d, dtype, seed=5)
    out, lse = ra.window_fwd(q, k, v, 4, 1024, 0, causal, "zigzag")
    ro, rl = ra.fwd(q, k, v, 4, causal, "zigzag")
    eps = 2.0 ** -7 if dtype == BF else 2.0 ** -17  # two roundings of the weights and two of the outputs of up to 4
    assert float((out.float() - ro.float()).abs().max()) <= 4 * eps
    assert float((lse - rl).abs().max()) <= 2.0 ** -16
    got = ra.window_bwd(q, k, v, ro, rl, dout, 4, 1024, 0, causal, "zigzag")
    for a, b in zip(got, ra.bwd(q, k, v, ro, rl, dout, 4, causal, "zigzag")):
        assert float((a - b).norm() / b.norm()) <= (2.0 ** -7 if dtype == BF else 2.0 ** -17)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("layout,n", [("contiguous", 1), ("striped", 4), ("zigzag", 2)])
def test_what_is_hidden_has_no_part(layout, n, dtype):
    """NaN and infinities in keys and values that most rows do not see.  In float32 those rows keep every bit.  With bf16
    inputs the rows that share a tile with such a value are computed once more, with unrounded weights: to the bounds of any
    row, and lse, which has no value in it, to the last bit."""
    B, H, Hkv, L, d, W, S = 1, 4, 2, 640, 128, 70, 3
    q, k, v, _ = _inputs(B, H, Hkv, L, d, dtype, seed=9)
    order = cu.natural(L, n, layout)
    at = torch.argsort(order)
    out, lse = ra.window_fwd(q, k, v, n, W, S, True, layout)
    ref = wu.fwd(q, k, v, n, layout, W, S, True)
    for j, (kx, vx) in {200: (math.nan, 1.0), 301: (1.0, math.nan), 383: (1.0, math.inf), 384: (1.0, -math.inf), 511: (math.inf, math.nan)}.items():
        k2, v2 = k.clone(), v.clone()
        k2[:, :, at[j], 5] *= kx
        v2[:, :, at[j], 7] *= vx
        o2, l2 = ra.window_fwd(q, k2, v2, n, W, S, True, layout)
        hidden = torch.ones(L, dtype=torch.bool)
        hidden[j:j + W] = False
        rows = hidden[order].to(DEV)
        assert torch.equal(l2[:, :, rows], lse[:, :, rows]), j
        if dtype == F32 or math.isfinite(vx):
            assert torch.equal(o2[:, :, rows], out[:, :, rows]), j
        cu.check_tree((o2[:, :, rows], l2[:, :, rows]), [x[:, :, rows.cpu()] for x in ref], WEIGHT_EPS[dtype], dtype, str(j))
        if not math.isfinite(vx):  # who sees it has it
            assert not bool(torch.isfinite(o2[:, :, ~rows][..., 7]).any())
            if math.isfinite(kx):
                keep = [c for c in range(d) if c != 7]
                assert bool(torch.isfinite(o2[..., keep]).all())


def test_memory_around_the_outputs_is_left_alone():
    B, H, Hkv, L, d, n = 1, 4, 2, 777, 64, 1
    q, k, v, dout = _inputs(B, H, Hkv, L, d, BF, seed=2)
    room = [torch.full((t.numel() + 4096,), 7.0, dtype=t.dtype, device=DEV) for t in (q, q, k, v)]
    out, dq, dk, dv = (r[2048:2048 + t.numel()].view(t.shape) for r, t in zip(room, (q, q, k, v)))
    lroom = torch.full((B * H * L + 2048,), 7.0, device=DEV)
    lse = lroom[1024:1024 + B * H * L].view(B, H, L)
    ra.window_fwd(q, k, v, n, 100, 4, True, "contiguous", out=out, lse=lse)
    ra.window_bwd(q, k, v, out, lse, dout, n, 100, 4, True, "contiguous", grad_dtype=BF, dq=dq, dk=dk, dv=dv)
    for r in (*room, lroom):
        m = 2048 if r is not lroom else 1024
        assert bool((r[:m] == 7).all()) and bool((r[-m:] == 7).all())


@pytest.mark.parametrize("dtype", [F32, BF])
def test_captured_and_replayed_on_new_inputs(dtype):
    B, H, Hkv, L, d, n = 1, 4, 2, 512, 128, 4
    q, k, v, dout = _inputs(B, H, Hkv, L, d, dtype, seed=21)

    def step():
        out, lse = ra.window_fwd(q, k, v, n, 90, 4, True, "striped")
        return (out, lse, *ra.window_bwd(q, k, v, out, lse, dout, n, 90, 4, True, "striped"))

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for seed in (31, 32):
        for t, x in zip((q, k, v, dout), _inputs(B, H, Hkv, L, d, dtype, seed)):
            t.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        cu.check_tree(got[:2], wu.fwd(q, k, v, n, "striped", 90, 4, True), WEIGHT_EPS[dtype], dtype)
        wu.check_bwd(got[2:], wu.bwd(q, k, v, got[0], got[1], dout, n, "striped", 90, 4, True, WEIGHT_EPS[dtype]))


@pytest.mark.parametrize("dtype", [F32, BF])
def test_another_stream(dtype):
    q, k, v, dout = _inputs(1, 4, 2, 1024, 64, dtype, seed=8)
    ref = _check(q, k, v, dout, 2, "zigzag", 200, 4, True)
    s = torch.cuda.Stream()
    big = torch.randn(4096, 4096, device=DEV)
    for _ in range(20):
        big = big @ big * 1e-3  # the current stream is busy when the other one is given
    s.wait_stream(torch.cuda.current_stream())
    out, lse = ra.window_fwd(q, k, v, 2, 200, 4, True, "zigzag", stream=s)
    got = ra.window_bwd(q, k, v, out, lse, dout, 2, 200, 4, True, "zigzag", stream=s)
    s.synchronize()
    assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
    assert torch.equal(got[1], ref[2][1]) and torch.equal(got[2], ref[2][2])


@pytest.mark.parametrize("f32_out", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_autograd(dtype, f32_out):
    q, k, v, dout = _inputs(2, 4, 2, 320, 64, dtype, seed=4)
    q, k, v = (x.requires_grad_() for x in (q, k, v))
    out = ra.ring_attention(q, k, v, 2, True, "striped", f32_out=f32_out, window=77, sinks=3)
    out.backward(dout.transpose(1, 2).contiguous().transpose(1, 2))  # a gradient that does not lie as the output does
    o2, lse = ra.window_fwd(q, k, v, 2, 77, 3, True, "striped", out_dtype=F32 if f32_out and dtype == BF else None)
    assert torch.equal(out, o2.to(dtype))
    ref = wu.bwd(q, k, v, o2, lse, dout, 2, "striped", 77, 3, True, WEIGHT_EPS[dtype])
    wu.check_bwd((q.grad, k.grad, v.grad), ref)


def test_gradients_against_differences():
    """The gradient along a random direction against the difference quotient of the float64 definition's value."""
    q, k, v, dout = _inputs(1, 2, 1, 200, 64, F32, seed=6)
    out, lse = ra.window_fwd(q, k, v, 1, 30, 2, True, "contiguous")
    got = ra.window_bwd(q, k, v, out, lse, dout, 1, 30, 2, True, "contiguous")
    g = torch.Generator().manual_seed(1)
    h, dd = 1e-4, dout.cpu().double()
    for i in range(3):
        x = [q, k, v]
        step = torch.randn(x[i].shape, generator=g, dtype=torch.float64)
        val = []
        for sign in (1, -1):
            y = [t.cpu().double() for t in x]
            y[i] = y[i] + sign * h * step
            val.append((wu.fwd(*y, 1, "contiguous", 30, 2, True)[0] * dd).sum())
        quotient = float(val[0] - val[1]) / (2 * h)
        have = float((got[i].cpu().double() * step).sum())
        # the quotient's own error is of h^2 and of the float64 roundings over h; the gradient's that of float32 sums
        assert abs(quotient - have) <= 1e-5 * float((got[i].cpu().double() * step).abs().sum()), i


@pytest.mark.parametrize("dtype", [F32, BF])
def test_results_that_do_not_vary(dtype):
    x = _inputs(1, 8, 2, 1500, 128, dtype, seed=14)
    q, k, v, dout = x
    out, lse = ra.window_fwd(q, k, v, 1, 300, 140, True, "contiguous")
    first = ra.window_bwd(q, k, v, out, lse, dout, 1, 300, 140, True, "contiguous")
    for _ in range(5):
        o2, l2 = ra.window_fwd(q, k, v, 1, 300, 140, True, "contiguous")
        again = ra.window_bwd(q, k, v, out, lse, dout, 1, 300, 140, True, "contiguous")
        assert torch.equal(out, o2) and torch.equal(lse, l2)
        assert all(torch.equal(a, b) for a, b in zip(first[0 if dtype == F32 else 1:], again[0 if dtype == F32 else 1:]))
