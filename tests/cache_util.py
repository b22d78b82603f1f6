"""Plain float64 statements of the norm with rotation, the quantised cache and the attention over it, on the
CPU, for the tests: loops and elementary operations, nothing of the package."""
import math

import numpy as np
import torch

EPS2 = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, relative


def natural(L, n, layout):
    S = L // n
    rows = []
    for i in range(n):
        if layout == "contiguous":
            rows += range(i * S, (i + 1) * S)
        elif layout == "striped":
            rows += range(i, L, n)
        else:
            C = S // 2
            rows += list(range(i * C, (i + 1) * C)) + list(range((2 * n - 1 - i) * C, (2 * n - i) * C))
    return torch.tensor(rows)


def turn(x, pos, base, sign=1.0):
    """x [.., rows, d] float64 rotated by sign * pos * base^(-2i/d); pos broadcasts to [.., rows]."""
    d = x.shape[-1]
    f = torch.tensor([base ** (-2.0 * i / d) for i in range(d // 2)], dtype=torch.float64)
    a = sign * pos.double().unsqueeze(-1) * f
    z = torch.view_as_complex(x.unflatten(-1, (d // 2, 2)).contiguous()) * torch.polar(torch.ones_like(a), a)
    return torch.view_as_real(z).flatten(-2)


def norm_rope(x, w, pos, base, eps):
    x = x.detach().cpu().double()
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    return turn(x * r * w.detach().cpu().double(), pos, base)


def norm_rope_bwd(x, w, dy, pos, base, eps):
    """dx, dw and the sum of the magnitudes behind each dw."""
    x, w = x.detach().cpu().double(), w.detach().cpu().double()
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    g = turn(dy.detach().cpu().double(), pos, base, -1.0)
    u = g * w
    return r * (u - x * r * r * (u * x).mean(-1, keepdim=True)), (g * x * r).sum((0, 1, 2)), (g * x * r).abs().sum((0, 1, 2))


def e4m3_nearest(y):
    """Nearest e4m3 value (ties to even) of float64 |y| <= 448."""
    step = 2.0 ** (torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3.0)
    return torch.round(y / step) * step


def quantised(x):
    """(values, exponents) of float64 rows by the definition: the smallest e >= -126 with amax <= 448 * 2^e."""
    amax = x.abs().amax(-1)
    e = torch.full(amax.shape, -126, dtype=torch.float64)
    for _ in range(2):
        e = torch.where(amax > 0, torch.ceil(torch.log2(amax / 448.0)), e)
    e = torch.where(amax > 448.0 * 2.0 ** e, e + 1, e)
    e = torch.where((amax <= 448.0 * 2.0 ** (e - 1)) & (amax > 0), e - 1, e).clamp_min(-126.0)
    return e4m3_nearest(x * 2.0 ** -e.unsqueeze(-1)), e


def cache_values(cache):
    """k, v of a KVCache as float64 on the CPU."""
    out = []
    for x, e in ((cache.k, cache.k_exp), (cache.v, cache.v_exp)):
        f = x.float().cpu().double()
        out.append(f if e is None else f * 2.0 ** (e.cpu().double() - 127.0).unsqueeze(-1))
    return out


def tree(q, k, v, lens, mask, ntok):
    """out, lse, sum_j w_j |v_j| (w the weights) and the largest |score| per row, float64.  k, v float64 [B,Hkv,cap,d];
    only rows that a query sees are touched."""
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
            own = torch.arange(T) <= t if mask is None else (mask[b, t] if mask.dim() == 3 else mask[t]).cpu()
            rows = torch.cat([torch.arange(n), n + torch.nonzero(own[:cnt]).flatten()])
            if rows.numel() == 0:
                continue
            for h in range(H):
                g = h // (H // Hkv)
                kk, vv = k[b, g, rows], v[b, g, rows]
                s = kk @ q[b, h, t] / math.sqrt(d)
                big[b, h, t] = s.abs().max()
                lse[b, h, t] = torch.logsumexp(s, 0)
                w = torch.exp(s - lse[b, h, t])
                out[b, h, t] = w @ vv
                mag[b, h, t] = w @ vv.abs()
    return out, lse, mag, big


def random_tree(B, T, seed, p_root=0.1):
    r = np.random.default_rng(seed)
    m = np.zeros((B, T, T), dtype=bool)
    for b in range(B):
        for t in range(T):
            if t and r.random() > p_root:
                m[b, t] = m[b, r.integers(0, t)]
            m[b, t, t] = True
    return torch.from_numpy(m)


def check_tree(got, ref, weight_eps, out_dtype, what=""):
    """out and lse against tree()'s.  A score is a sum of d products in float32: off by at most 2^-24 * (a few) of
    the sum of magnitudes, taken as 2^-18 (1 + |s|max) here; a weight is off by that, by exp2 (2^-21) and by its rounding
    for the product (weight_eps: half a step of the type it is held in, 0 if float32); the output is off by twice
    the weights' relative error times sum w |v|, and by its own rounding."""
    out, lse = got
    r_out, r_lse, mag, big = ref
    out, lse = out.detach().cpu().double(), lse.detach().cpu().double()
    empty = torch.isinf(r_lse)
    assert torch.equal(torch.isinf(lse) & (lse < 0), empty), f"{what}: rows that see nothing"
    assert bool((out[empty] == 0).all()), f"{what}: output of rows that see nothing"
    s_err = 2.0 ** -18 * (1 + big)
    d = (lse - r_lse).abs()[~empty] - (s_err + 2.0 ** -22 * r_lse.abs())[~empty]
    assert d.numel() == 0 or float(d.max()) <= 0, f"{what}: lse off by {float(d.max()):.3e} beyond its bound"
    tol = mag * (weight_eps + 2 * (s_err + 2.0 ** -20)).unsqueeze(-1) + EPS2[out_dtype] * 1.01 * r_out.abs() + 1e-30
    d = (out - r_out).abs() - tol
    assert float(d.max()) <= 0, f"{what}: out off by {float(d.max()):.3e} beyond its bound"
