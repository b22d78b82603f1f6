"""Attention through a window at the lengths that it is for, 64K tokens, against float64: sampled rows of the output, lse and dq,
sampled keys of dk and dv, among them the first tokens, which all later ones see, and the borders of tiles and windows."""
import math

import pytest
import torch

import cache_util as cu
import sequence_sharded_exact_gb300 as ra

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
WEIGHT_EPS = {BF: 2.0 ** -8, F32: 0.0}
L = 65536


@pytest.fixture(autouse=True)
def _clean_status():
    torch.cuda.set_device(0)
    ra.device_status()
    yield
    assert ra.device_status() == 0


def _sees(p, j, W, S, causal):
    near = (p[:, None] - j).abs() < W
    return ((near | (j < S)) & (j <= p[:, None])) if causal else (near | (j < S))


def _scores(q, k):
    return q @ k.transpose(-1, -2) / math.sqrt(q.shape[-1])


def _row_ref(q, k, v, rows, W, S, causal):
    """wu.fwd's four results at the given positions of one head, all in float64 and natural order."""
    hide = ~_sees(rows, torch.arange(L, device=DEV), W, S, causal)
    s = _scores(q[rows], k).masked_fill(hide, -math.inf)
    lse = torch.logsumexp(s, -1)
    w = torch.exp(s - lse[:, None])
    return w @ v, lse, w @ v.abs(), s.masked_fill(hide, 0.0).abs().amax(-1)


def _pair_ref(q, k, v, out, lse, dout, hide, eps):
    """P, dS and how far a kernel's may be off, as in wu.bwd, for some queries and some keys of one head."""
    scale = 1.0 / math.sqrt(q.shape[-1])
    p = torch.exp(_scores(q, k).masked_fill(hide, -math.inf) - lse[:, None])
    t = dout @ v.T - (dout * out).sum(-1, keepdim=True)
    ds = p * t * scale
    mag = dout.abs() @ v.abs().T + (dout * out).abs().sum(-1, keepdim=True)
    p_err = 2.0 ** -18 * (1 + q.abs() @ k.abs().T * scale) + (2.0 ** -23 * lse.abs())[:, None] + 2.0 ** -20
    return p, ds, p * (p_err + eps + 2.0 ** -18), p * scale * (p_err * t.abs() + 2.0 ** -18 * mag) + (eps + 2.0 ** -18) * ds.abs()


@pytest.mark.parametrize("dtype,H,Hkv,d,n,layout,W,S,causal", [
    (BF, 4, 1, 128, 16, "zigzag", 4096, 4, True),
    (BF, 4, 1, 64, 16, "striped", 1024, 130, True),
    (BF, 3, 1, 128, 1, "contiguous", 128, 0, True),
    (BF, 2, 2, 64, 2, "zigzag", 512, 2, False),
    (F32, 2, 1, 128, 16, "zigzag", 1000, 4, True),
    (F32, 2, 1, 64, 16, "striped", 300, 3, False),
])
def test_64k_tokens_sampled(dtype, H, Hkv, d, n, layout, W, S, causal):
    g = torch.Generator(device=DEV).manual_seed(W + d)
    q, k, v, dout = (torch.randn((1, h, L, d), generator=g, device=DEV).to(dtype) for h in (H, Hkv, Hkv, H))
    order = cu.natural(L, n, layout).to(DEV)
    nat = lambda x: x.index_select(2, torch.argsort(order))  # noqa: E731
    out, lse = ra.window_fwd(q, k, v, n, W, S, causal, layout)
    grads = ra.window_bwd(q, k, v, out, lse, dout, n, W, S, causal, layout)
    q, k, v, dout, out, lse = (nat(x)[0].double() for x in (q, k, v, dout, out, lse))
    dq, dk, dv = (nat(x)[0] for x in grads)
    pick = torch.randint(0, L, (40,), generator=torch.Generator().manual_seed(1)).tolist()
    at = torch.tensor(sorted({0, 1, S, W - 1, W, W + 1, 127, 128, L // 2 - 1, L // 2, L - W, L - 129, L - 128, L - 1, *pick}), device=DEV)
    every, G, eps = torch.arange(L, device=DEV), H // Hkv, WEIGHT_EPS[dtype]
    for h in range(H):
        z = h // G
        ref = _row_ref(q[h], k[z], v[z], at, W, S, causal)
        cu.check_tree((out[h][at], lse[h][at]), [x.cpu() for x in ref], eps, dtype, f"head {h}")
        _, ds, _, err = _pair_ref(q[h][at], k[z], v[z], out[h][at], lse[h][at], dout[h][at], ~_sees(at, every, W, S, causal), eps)
        # (the other two are looked at below)
        have, want, off = dq[h][at].double(), ds @ k[z], err @ k[z].abs()
        assert float(((have - want).abs() - off - 2.0 ** -23 * want.abs()).max()) <= 1e-30, f"dq of head {h}"
    for z in range(Hkv):
        want = [torch.zeros((len(at), d), dtype=torch.float64, device=DEV) for _ in range(4)]
        for h in range(z * G, (z + 1) * G):
            p, ds, p_err, ds_err = _pair_ref(q[h], k[z][at], v[z][at], out[h], lse[h], dout[h], ~_sees(every, at, W, S, causal), eps)
            for x, y in zip(want, (ds.T @ q[h], p.T @ dout[h], ds_err.T @ q[h].abs(), p_err.T @ dout[h].abs())):
                x += y
        for name, have, x, off in (("dk", dk, want[0], want[2]), ("dv", dv, want[1], want[3])):
            assert float(((have[z][at].double() - x).abs() - off - 2.0 ** -23 * x.abs()).max()) <= 1e-30, f"{name} of kv head {z}"
