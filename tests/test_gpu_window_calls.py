"""Calls of the attention through a window that the arguments allow beyond the plain one: both forms of a call, given outputs
and workspaces with anything in them, addresses that only 16 bytes divide, two streams at once, replayed graphs, sizes on both
sides of the rules that choose a launch."""
import math

import pytest
import torch

import cache_util as cu
import sequence_sharded_exact_gb300 as ra
import window_util as wu
from sequence_sharded_exact_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
WEIGHT_EPS = {BF: 2.0 ** -8, F32: 0.0}
LAYOUTS = [("contiguous", 1), ("zigzag", 2), ("striped", 4), ("striped", 5)]


@pytest.fixture(autouse=True)
def _clean_status():
    torch.cuda.set_device(0)
    ra.device_status()
    yield
    assert ra.device_status() == 0


def _inputs(B, H, Hkv, L, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn((B, h, L, d), generator=g).to(dtype).to(DEV) for h in (H, Hkv, Hkv, H)]


def _same(got, ref, dtype):
    """Bit for bit, but for dq (the first) of bf16 inputs, whose sums' order varies: both within a few float32 roundings of
    sums of at most 32 tiles' terms, whose magnitudes are a few times the sum's norm."""
    assert all(torch.equal(a, b) for a, b in zip(got[1:], ref[1:]))
    if dtype == F32:
        assert torch.equal(got[0], ref[0])
    else:
        assert float((got[0] - ref[0]).norm() / ref[0].norm()) <= 2.0 ** -17


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("layout,n", LAYOUTS)
def test_both_forms_and_given_buffers(layout, n, dtype):
    B, H, Hkv, L, d, W, S = 2, 4, 2, 1280, 64, 150, 140
    q, k, v, dout = _inputs(B, H, Hkv, L, d, dtype, seed=1)
    s = torch.cuda.current_stream()
    out, lse = ra.window_fwd(q, k, v, n, W, S, True, layout)
    ref = ra.window_bwd(q, k, v, out, lse, dout, n, W, S, True, layout)
    code, lay = binding._dtype_code(dtype), binding._layout(layout)
    sizes = (binding.library().ring_attn_window_fwd_workspace_size(B, H, Hkv, L, d, n, lay, code),
             binding.library().ring_attn_window_bwd_workspace_size(B, H, Hkv, L, d, n, W, S, 1, lay, code))
    # (chunks of 320 positions, or 5 stripes, are no whole boxes of 128: bf16 inputs are copied)
    assert (sizes[0] > 0) == (dtype == BF and (layout == "zigzag" or n == 5)) and sizes[1] > 0
    for stream in (None, s):
        o, l = ra.window_fwd(q, k, v, n, W, S, True, layout, stream=stream)
        assert torch.equal(o, out) and torch.equal(l, lse)
        _same(ra.window_bwd(q, k, v, out, lse, dout, n, W, S, True, layout, stream=stream), ref, dtype)
        # what the buffers hold does not matter, and every element of the outputs is written
        ws = [torch.full((x,), 0xff, dtype=torch.uint8, device=DEV) for x in sizes]
        o, l = torch.full_like(out, math.nan), torch.full_like(lse, math.nan)
        got = ra.window_fwd(q, k, v, n, W, S, True, layout, out=o, lse=l, workspace=ws[0], stream=stream)
        assert got[0].data_ptr() == o.data_ptr() and torch.equal(o, out) and torch.equal(l, lse)
        grads = [torch.full_like(x, math.nan) for x in ref]
        ra.window_bwd(q, k, v, out, lse, dout, n, W, S, True, layout, dq=grads[0], dk=grads[1], dv=grads[2], workspace=ws[1], stream=stream)
        _same(grads, ref, dtype)


def test_both_forms_refuse_alike():
    q, k, v, dout = _inputs(1, 4, 2, 256, 64, BF, seed=1)
    out, lse = ra.window_fwd(q, k, v, 2, 9, 0, True, "zigzag")
    small = torch.empty(64, dtype=torch.uint8, device=DEV)
    refused = [(binding.RingAttnError, dict(window=0)), (binding.RingAttnError, dict(sinks=-1)), (ValueError, dict(window=2 ** 31)),
               (TypeError, dict(window=4.0)), (KeyError, dict(layout="other")), (binding.RingAttnError, dict(n_shards=3))]
    for stream in (None, torch.cuda.current_stream()):
        for err, kw in refused + [(ValueError, dict(out_dtype=torch.float16)), (ValueError, dict(out=out.float()))]:
            with pytest.raises(err):
                ra.window_fwd(q, k, v, **{**dict(n_shards=2, window=9), **kw}, stream=stream)
        for err, kw in refused + [(ValueError, dict(workspace=small)), (ValueError, dict(dq=torch.empty_like(k, dtype=F32)))]:
            with pytest.raises(err):
                ra.window_bwd(q, k, v, out, lse, dout, **{**dict(n_shards=2, window=9), **kw}, stream=stream)
        for bad in (k.float(), k.transpose(1, 2).contiguous().transpose(1, 2), k[:, :, :-1], k.cpu()):
            with pytest.raises(ValueError):
                ra.window_fwd(q, bad, v, 2, 9, stream=stream)
            with pytest.raises(ValueError):
                ra.window_bwd(q, bad, v, out, lse, dout, 2, 9, stream=stream)


@pytest.mark.parametrize("grad_dtype", [F32, BF])
@pytest.mark.parametrize("dtype,out_dtype", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("d", [64, 128])
def test_addresses_that_16_bytes_divide(d, dtype, out_dtype, grad_dtype):
    """Inputs and outputs 16 bytes behind a border of 32, 128 and 256."""
    B, H, Hkv, L = 1, 4, 2, 321

    def moved(x):
        room = torch.empty(x.numel() + 256, dtype=x.dtype, device=DEV)
        assert room.data_ptr() % 256 == 0
        y = room[16 // x.element_size():][:x.numel()].view(x.shape)
        y.copy_(x)
        return y

    x = _inputs(B, H, Hkv, L, d, dtype, seed=d)
    out, lse = ra.window_fwd(*x[:3], 1, 100, 3, True, "contiguous", out_dtype=out_dtype)
    ref = ra.window_bwd(*x[:3], out, lse, x[3], 1, 100, 3, True, "contiguous", grad_dtype=grad_dtype)
    q, k, v, dout = (moved(t) for t in x)
    o, l = moved(torch.zeros_like(out)), moved(torch.zeros_like(lse))
    ra.window_fwd(q, k, v, 1, 100, 3, True, "contiguous", out_dtype=out_dtype, out=o, lse=l)
    assert torch.equal(o, out) and torch.equal(l, lse)
    g = [moved(torch.zeros_like(t)) for t in ref]
    ra.window_bwd(q, k, v, o, l, dout, 1, 100, 3, True, "contiguous", grad_dtype=grad_dtype, dq=g[0], dk=g[1], dv=g[2])
    if grad_dtype == F32:
        _same(g, ref, dtype)
    else:  # (dq's order may move a value over a border between two roundings)
        assert torch.equal(g[1], ref[1]) and torch.equal(g[2], ref[2])
        assert float((g[0].float() - ref[0].float()).norm() / ref[0].float().norm()) <= 2.0 ** -7


@pytest.mark.parametrize("layout,n", LAYOUTS)
def test_two_streams_at_once(layout, n):
    """Short calls, whose launches follow one another early, in turns on two streams."""
    cases = []
    for seed in (3, 4):
        x = _inputs(1, 8, 2, 640, 64, BF, seed)
        out, lse = ra.window_fwd(*x[:3], n, 70, 4, True, layout)
        cases.append((x, out, lse, ra.window_bwd(*x[:3], out, lse, x[3], n, 70, 4, True, layout)))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = ([], [])
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                x, out, lse, _ = cases[i]
                got[i].append((*ra.window_fwd(*x[:3], n, 70, 4, True, layout), ra.window_bwd(*x[:3], out, lse, x[3], n, 70, 4, True, layout)))
    torch.cuda.synchronize()
    for (x, out, lse, ref), have in zip(cases, got):
        for o, l, g in have:
            assert torch.equal(o, out) and torch.equal(l, lse)
            _same(g, ref, BF)


def test_a_graph_of_several_backward_calls():
    """Backward calls behind one another in one graph, on one workspace: each one's launches wait for those before."""
    n, W, S, layout = 4, 90, 130, "striped"
    x = [_inputs(1, 4, 2, 768, 128, BF, seed) for seed in (5, 6, 7)]
    need = binding.library().ring_attn_window_bwd_workspace_size(1, 4, 2, 768, 128, n, W, S, 1, binding._layout(layout), 1)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    fwd = [ra.window_fwd(*t[:3], n, W, S, True, layout) for t in x]

    def step():
        return [ra.window_bwd(*t[:3], o, l, t[3], n, W, S, True, layout, workspace=ws) for t, (o, l) in zip(x, fwd)]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ref = step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for _ in range(5):
        for grads in got:
            for t in grads:
                t.fill_(math.nan)
        ws.fill_(0xff)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, ref):
            _same(a, b, BF)


@pytest.mark.parametrize("W,S", [(300, 0), (4096, 0)])
def test_a_batch_is_its_sequences(W, S):
    """Four sequences at once, dQ's accumulator beyond 128 MB (launches one after another), and each alone (below)."""
    x = _inputs(4, 32, 8, 4096, 128, BF, seed=8)
    out, lse = ra.window_fwd(*x[:3], 4, W, S, True, "zigzag")
    got = ra.window_bwd(*x[:3], out, lse, x[3], 4, W, S, True, "zigzag")
    for b in range(4):
        y = [t[b:b + 1] for t in x]
        o, l = ra.window_fwd(*y[:3], 4, W, S, True, "zigzag")
        assert torch.equal(o, out[b:b + 1]) and torch.equal(l, lse[b:b + 1])
        _same([t[b:b + 1] for t in got], ra.window_bwd(*y[:3], o, l, y[3], 4, W, S, True, "zigzag"), BF)


@pytest.mark.parametrize("B,H,Hkv,L,d,n,layout,W,S,causal", [
    (1, 8, 2, 640, 64, 1, "contiguous", 600, 3, True),     # one round: every tile but the sinks' in several units
    (1, 8, 2, 640, 128, 1, "contiguous", 600, 0, True),
    (2, 6, 2, 700, 128, 7, "striped", 300, 200, True),     # of the last tile only a part is in the sequence
    (1, 14, 14, 1410, 64, 5, "zigzag", 1400, 0, True),     # 168 units: a whole round, and 16 in pieces
    (1, 14, 14, 1410, 128, 1, "contiguous", 700, 100, False),
])
def test_backward_units_in_pieces(B, H, Hkv, L, d, n, layout, W, S, causal):
    """Batches whose last round of units is cut."""
    x = _inputs(B, H, Hkv, L, d, BF, seed=L + d)
    out, lse = ra.window_fwd(*x[:3], n, W, S, causal, layout)
    got = ra.window_bwd(*x[:3], out, lse, x[3], n, W, S, causal, layout)
    wu.check_bwd(got, wu.bwd(*x[:3], out, lse, x[3], n, layout, W, S, causal, 2.0 ** -8))
    again = ra.window_bwd(*x[:3], out, lse, x[3], n, W, S, causal, layout)
    _same(again, got, BF)


@pytest.mark.parametrize("layout,n", [("contiguous", 1), ("striped", 5)])
@pytest.mark.parametrize("out_dtype", [BF, F32])
def test_rows_beside_values_that_are_not_finite(out_dtype, layout, n):
    """bf16 values with infinities and NaN in several rows and columns: who sees one has it in its column, and every other
    element is within its bound."""
    B, H, Hkv, L, d, W, S = 1, 6, 2, 640, 64, 140, 2
    q, k, v, _ = _inputs(B, H, Hkv, L, d, BF, seed=12)
    order = cu.natural(L, n, layout)
    at = torch.argsort(order)
    bad = {10: (0, math.inf), 250: (5, math.nan), 251: (5, -math.inf), 252: (63, math.inf), 639: (7, math.nan)}
    v2 = v.clone()
    for j, (c, x) in bad.items():
        v2[:, :, at[j], c] = x
    got = ra.window_fwd(q, k, v2, n, W, S, True, layout, out_dtype=out_dtype)
    out, lse, mag, big = wu.fwd(q, k, v, n, layout, W, S, True)
    seen = torch.zeros(L, d, dtype=torch.bool)
    sees = wu.sees(L, W, S, True)
    for j, (c, _) in bad.items():
        seen[sees[:, j], c] = True
    seen = seen[order].expand(B, H, L, d)
    o = got[0].cpu()
    assert not bool(torch.isfinite(o[seen]).any())
    assert bool(torch.isinf(o[..., 63][seen[..., 63]]).all()) and bool(torch.isinf(o[..., 0][seen[..., 0]]).all())
    # the others: their float64 value does not have the bad elements in it
    o = torch.where(seen, out.to(o.dtype), o)
    cu.check_tree((o, got[1].cpu()), (out, lse, mag, big), 2.0 ** -8, out_dtype, "the rest")


@pytest.mark.parametrize("d", [64, 128])
def test_a_sink_of_infinities(d):
    """A value that every row sees, infinite in all columns: every output is, lse is what it was, and the call ends without a wait
    that ran out (the fixture's status) although every row is looked at again."""
    q, k, v, _ = _inputs(1, 4, 2, 4096, d, BF, seed=d)
    out, lse = ra.window_fwd(q, k, v, 1, 1024, 2, True, "contiguous")
    v2 = v.clone()
    v2[:, :, 1] = math.inf
    v2[:, :, 1, 5] = -math.inf
    o2, l2 = ra.window_fwd(q, k, v2, 1, 1024, 2, True, "contiguous")
    assert torch.equal(l2, lse) and torch.equal(o2[:, :, :1], out[:, :, :1])
    sign = torch.ones(d, device=DEV)
    sign[5] = -1
    assert bool((o2[:, :, 1:] == sign * math.inf).all())


def test_the_smallest_and_odd_stripes():
    """A row per shard, shards of a row each in a tile of 128, and heads that pair up or do not."""
    for L, n, layout in ((2, 2, "striped"), (64, 64, "striped"), (256, 64, "striped"), (384, 128, "striped"), (6, 3, "zigzag"), (128, 1, "zigzag")):
        for H, Hkv in ((2, 1), (3, 1), (3, 3)):
            q, k, v, dout = _inputs(1, H, Hkv, L, 128, BF, seed=L)
            out, lse = ra.window_fwd(q, k, v, n, 33, 1, True, layout)
            cu.check_tree((out, lse), wu.fwd(q, k, v, n, layout, 33, 1, True), 2.0 ** -8, BF, f"{L} {n} {layout}")
            got = ra.window_bwd(q, k, v, out, lse, dout, n, 33, 1, True, layout)
            wu.check_bwd(got, wu.bwd(q, k, v, out, lse, dout, n, layout, 33, 1, True, 2.0 ** -8), f"{L} {n} {layout}")


def test_one_tensor_for_several_inputs():
    """q, k and v in one tensor, and the gradients' sum through autograd."""
    x = _inputs(1, 2, 2, 300, 64, F32, seed=3)[0]
    dout = torch.randn_like(x)
    out, lse = ra.window_fwd(x, x, x, 1, 40, 2, True, "contiguous")
    cu.check_tree((out, lse), wu.fwd(x, x, x, 1, "contiguous", 40, 2, True), 0.0, F32)
    parts = ra.window_bwd(x, x, x, out, lse, dout, 1, 40, 2, True, "contiguous")
    y = x.transpose(1, 2).contiguous().transpose(1, 2).requires_grad_()  # does not lie as the call wants it
    o = ra.ring_attention(y, y, y, 1, True, "contiguous", window=40, sinks=2)
    assert torch.equal(o, out)
    o.backward(dout)
    total = sum(p.double() for p in parts)
    # three float32 gradients added in float32
    assert float((y.grad.double() - total).abs().max()) <= 2.0 ** -22 * float(sum(p.abs().double() for p in parts).max())


@pytest.mark.parametrize("dtype,cdt", [(F32, F32), (F32, E4M3), (BF, BF), (BF, E4M3)])
@pytest.mark.parametrize("B", [8, 20, 37, 64, 200, 700])
def test_batches_on_both_sides_of_an_item_per_cta(B, dtype, cdt):
    """Batches whose items are fewer than the CTAs, about as many, and more, with sequences of no tokens among them: every
    sequence as it is alone, to the roundings of another split."""
    H, Hkv, T, d, cap, W, S = 8, 2, 2, 64, 520, 200, 3
    g = torch.Generator().manual_seed(B)
    cache = ra.cache_alloc(B, Hkv, cap, d, cdt)
    k, v = (torch.randn((B, Hkv, cap, d), generator=g).to(dtype).to(DEV) for _ in range(2))
    ra.cache_write(cache, k, v)
    q = torch.randn((B, H, T, d), generator=g).to(dtype).to(DEV)
    lens = torch.randint(0, cap - T + 1, (B,), generator=g).to(torch.int32)
    ntok = torch.randint(0, T + 1, (B,), generator=g).to(torch.int32)
    lens[0], ntok[0] = cap - T, T
    got = ra.tree_fwd(q, cache, lens.to(DEV), ntok=ntok.to(DEV), window=W, sinks=S,
                      out=torch.full_like(q, math.nan), lse=torch.full((B, H, T), math.nan, device=DEV))
    for b in range(0, B, max(1, B // 20)):
        one = ra.KVCache(*(None if x is None else x[b:b + 1] for x in cache))
        ref = ra.tree_fwd(q[b:b + 1], one, lens[b:b + 1].to(DEV), ntok=ntok[b:b + 1].to(DEV), window=W, sinks=S)
        kv, vv = cu.cache_values(one)
        exact = wu.tree(q[b:b + 1], kv, vv, lens[b:b + 1], None, ntok[b:b + 1], W, S, None)
        cu.check_tree([x[b:b + 1] for x in got], exact, WEIGHT_EPS[dtype], dtype, f"{B} {b}")
        cu.check_tree(ref, exact, WEIGHT_EPS[dtype], dtype, f"alone {b}")
        none = slice(int(ntok[b]), T)
        assert bool((got[0][b, :, none] == 0).all()) and bool((got[1][b, :, none] == -math.inf).all())


def test_windowed_steps_on_two_streams():
    B, H, Hkv, T, d, cap = 24, 8, 2, 4, 128, 900
    cases = []
    for seed in (1, 2):
        g = torch.Generator().manual_seed(seed)
        cache = ra.cache_alloc(B, Hkv, cap, d, BF)
        ra.cache_write(cache, *(torch.randn((B, Hkv, cap, d), generator=g).to(BF).to(DEV) for _ in range(2)))
        q = torch.randn((B, H, T, d), generator=g).to(BF).to(DEV)
        lens = torch.randint(0, cap - T + 1, (B,), generator=g).to(torch.int32).to(DEV)
        cases.append((q, cache, lens, ra.tree_fwd(q, cache, lens, window=300, sinks=4)))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = ([], [])
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(ra.tree_fwd(*cases[i][:3], window=300, sinks=4))
    torch.cuda.synchronize()
    for c, have in zip(cases, got):
        assert all(torch.equal(a, b) for x in have for a, b in zip(x, c[3]))
