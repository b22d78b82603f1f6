"""The attention through a window in float64 on the CPU, for the tests: the definition over the whole score matrix,
nothing of the package; and how far a kernel may be off, from the roundings that it makes."""
import math

import torch

import cache_util as cu

EPS2 = cu.EPS2  # half a step, relative


def sees(L, W, S, causal):
    """[L, L] by natural positions: does query p see key j."""
    p, j = torch.arange(L)[:, None], torch.arange(L)[None, :]
    near = (p - j).abs() < W
    return ((near | (j < S)) & (j <= p)) if causal else (near | (j < S))


def _natural(x, order):
    """Rows (third dimension) of x, in the layout's order, as float64 in natural order."""
    return x.detach().cpu().double()[:, :, torch.argsort(order)]


def _layout(x, order):
    return x[:, :, order]


def fwd(q, k, v, n, layout, W, S, causal):
    """out, lse, sum_j w_j |v_j| and the largest visible |score| per row, in the layout's order (as cache_util.tree's)."""
    order = cu.natural(q.shape[2], n, layout)
    q, k, v = (_natural(x, order) for x in (q, k, v))
    G = q.shape[1] // k.shape[1]
    hide = ~sees(q.shape[2], W, S, causal)
    k, v = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    s = torch.where(hide, -math.inf, q @ k.transpose(-1, -2) / math.sqrt(q.shape[-1]))
    lse = torch.logsumexp(s, -1)
    w = torch.exp(s - lse.unsqueeze(-1))
    big = s.masked_fill(hide, 0.0).abs().amax(-1)
    return tuple(_layout(x, order) for x in (w @ v, lse, w @ v.abs(), big))


def bwd(q, k, v, out, lse, dout, n, layout, W, S, causal, weight_eps):
    """(dq, dk, dv) of the formulas for the given out and lse, and for each how far a kernel may be off before its
    output's rounding.  A sum of float32 products is off by at most 2^-18 of its terms' magnitudes (d = 128 terms of 2^-24
    each, their sums' roundings); a weight by the score's error, lse's half step, exp2's 2^-20, and weight_eps for the type in
    which it goes into the products with positions; dS likewise."""
    order = cu.natural(q.shape[2], n, layout)
    q, k, v, out, dout = (_natural(x, order) for x in (q, k, v, out, dout))
    lse = _natural(lse.unsqueeze(-1), order)
    G, scale = q.shape[1] // k.shape[1], 1.0 / math.sqrt(q.shape[-1])
    hide = ~sees(q.shape[2], W, S, causal)
    kk, vv = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    s = (q @ kk.transpose(-1, -2) * scale).masked_fill(hide, -math.inf)
    p = torch.exp(s - lse)
    t = dout @ vv.transpose(-1, -2) - (dout * out).sum(-1, keepdim=True)
    ds = p * t * scale
    mag = dout.abs() @ vv.abs().transpose(-1, -2) + (dout * out).abs().sum(-1, keepdim=True)
    p_err = 2.0 ** -18 * (1 + q.abs() @ kk.abs().transpose(-1, -2) * scale) + 2.0 ** -23 * lse.abs() + 2.0 ** -20
    ds_err = p * scale * (p_err * t.abs() + 2.0 ** -18 * mag) + (weight_eps + 2.0 ** -18) * ds.abs()
    dv_err = p * (p_err + weight_eps + 2.0 ** -18)
    heads = lambda x: x.unflatten(1, (-1, G)).sum(2)  # noqa: E731
    tr = lambda x: x.transpose(-1, -2)  # noqa: E731
    got = ds @ kk, heads(tr(ds) @ q), heads(tr(p) @ dout)
    err = ds_err @ kk.abs(), heads(tr(ds_err) @ q.abs()), heads(tr(dv_err) @ dout.abs())
    return tuple(_layout(x, order) for x in got), tuple(_layout(x, order) for x in err)


def check_bwd(got, ref, what=""):
    for name, g, r, e in zip(("dq", "dk", "dv"), got, *ref):
        tol = e + EPS2[g.dtype] * 1.01 * (r.abs() + e) + 1e-30
        d = (g.detach().cpu().double() - r).abs() - tol
        assert float(d.max()) <= 0, f"{what}: {name} off by {float(d.max()):.3e} beyond its bound"


def tree(q, k, v, lens, mask, ntok, window, sinks, positions):
    """cache_util.tree through a window: the same four results."""
    q = q.float().cpu().double()
    B, H, T, d = q.shape
    Hkv = k.shape[1]
    out = torch.zeros((B, H, T, d), dtype=torch.float64)
    mag = torch.zeros_like(out)
    lse = torch.full((B, H, T), -math.inf, dtype=torch.float64)
    big = torch.zeros_like(lse)
    for b in range(B):
        n = int(lens[b])
        cnt = T if ntok is None else int(ntok[b])
        for t in range(cnt):
            p = n + t if positions is None else min(max(int(positions[b, t]), n), n + T - 1)
            prefix = [j for j in range(n) if j < sinks or p - j < window]
            if mask is None:
                step = [n + j for j in range(t + 1) if t - j < window]
            else:
                row = (mask[b, t] if mask.dim() == 3 else mask[t]).cpu()
                step = [n + j for j in range(cnt) if row[j]]
            rows = torch.tensor(prefix + step, dtype=torch.long)
            if rows.numel() == 0:
                continue
            for g in range(Hkv):
                kk, vv = k[b, g, rows], v[b, g, rows]
                h = slice(g * (H // Hkv), (g + 1) * (H // Hkv))
                s = q[b, h, t] @ kk.T / math.sqrt(d)
                big[b, h, t] = s.abs().amax(-1)
                lse[b, h, t] = torch.logsumexp(s, -1)
                w = torch.exp(s - lse[b, h, t].unsqueeze(-1))
                out[b, h, t] = w @ vv
                mag[b, h, t] = w @ vv.abs()
    return out, lse, mag, big
