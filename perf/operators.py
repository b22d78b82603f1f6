"""What is measured of the operators around the attention of a sequence: the norms of queries and keys with
the rotation by natural position (forward and backward), the key/value cache that is quantised as it is
written and read back, and the attention of a tree of drafted tokens over that cache.

listed() holds the cases, draw() more of the same ranges, prepare() makes what a program has in hand before
the call, run() makes one pass (own: through the package's calls; otherwise in elementary torch operations in
float32), exact() computes the same in float64, work() counts what a pass cannot do without.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "f32": 4, "e4m3": 1}


# --------------------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------------------
def listed():
    return [
        # the long-context training step (64K tokens in 16 zigzag shards, 32 query and 8 kv heads of 128):
        # norms and rotation of q and k before the attention, and their gradients after its backward
        dict(name="norm_rope_train_64k", op="norm_rope", B=1, H=32, Hkv=8, L=65536, d=128, n=16, layout="zigzag",
             dtype="bf16", backward=False, fused=False, tokens=False),
        dict(name="norm_rope_train_64k_bwd", op="norm_rope", B=1, H=32, Hkv=8, L=65536, d=128, n=16, layout="zigzag",
             dtype="bf16", backward=True, fused=False, tokens=False),
        # one serving step: 16 sequences of 8 drafted tokens straight out of the fused projection
        # ([B, T, H + 2 Hkv, d]), each at its own far position
        dict(name="norm_rope_drafted", op="norm_rope", B=16, H=32, Hkv=8, L=8, d=128, n=1, layout="contiguous",
             dtype="bf16", backward=False, fused=True, tokens=True),
        # a float32 check run of odd sizes, backward, inputs as slices of the fused projection
        dict(name="norm_rope_f32_odd_bwd", op="norm_rope", B=2, H=6, Hkv=2, L=1235, d=64, n=5, layout="striped",
             dtype="f32", backward=True, fused=True, tokens=False),
        # a prompt of 128K tokens quantised into the cache, and read back for the next chunk's attention
        dict(name="cache_write_prompt_128k", op="cache_write", B=1, Hkv=8, T=131072, cap=131200, length=0, d=128,
             dtype="bf16", fused=False, ragged=False),
        dict(name="cache_read_128k", op="cache_read", B=1, Hkv=8, T=131072, cap=131200, row0=0, d=128, dtype="bf16"),
        # the drafted tokens of a ragged batch written behind each sequence's prefix
        dict(name="cache_write_drafted", op="cache_write", B=16, Hkv=8, T=8, cap=4100, length=4000, d=128,
             dtype="bf16", fused=True, ragged=True),
        # one token after a 128K-token prompt, the cache kept in bfloat16
        dict(name="tree_decode_128k", op="tree", B=1, H=32, Hkv=8, T=1, cap=131200, length=131072, d=128,
             dtype="bf16", cache="bf16", tree=False, ragged=False, blank=False),
        # a ragged batch of eight sequences, 32 drafted tokens each, over the quantised cache
        dict(name="tree_e4m3_ragged", op="tree", B=8, H=32, Hkv=8, T=32, cap=33001, length=32768, d=128,
             dtype="bf16", cache="e4m3", tree=True, ragged=True, blank=False),
        # the smallest calls: a few drafted tokens over short prefixes, one of them empty
        dict(name="tree_small_blank", op="tree", B=2, H=8, Hkv=2, T=5, cap=640, length=500, d=64,
             dtype="bf16", cache="bf16", tree=True, ragged=True, blank=True),
        # a wide tree (64 tokens under 4 query heads per kv head): the products count
        dict(name="tree_wide", op="tree", B=2, H=32, Hkv=8, T=64, cap=32900, length=32768, d=128,
             dtype="bf16", cache="bf16", tree=True, ragged=False, blank=False),
        # float32 end to end
        dict(name="tree_f32", op="tree", B=1, H=8, Hkv=2, T=5, cap=9100, length=9000, d=64,
             dtype="f32", cache="f32", tree=True, ragged=False, blank=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope", "cache_write", "cache_read", "tree", "tree", "tree"])
    d = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 4, 8])
    if op == "norm_rope":
        tokens = rng.random() < 0.4
        dtype = rng.choice(["bf16", "bf16", "f32"])
        n, layout = 1, "contiguous"
        if tokens:
            B, L = rng.randint(1, 48), rng.randint(1, 64)
        else:
            B, L = rng.randint(1, 2), _log(rng, 64, 16384)
            n, layout = rng.choice([1, 2, 4, 5, 8, 16]), rng.choice(["contiguous", "zigzag", "striped"])
            step = 2 * n if layout == "zigzag" else n
            L = max(1, L // step) * step
        return dict(op=op, B=B, H=Hkv * G, Hkv=Hkv, L=L, d=d, n=n, layout=layout, dtype=dtype,
                    backward=rng.random() < 0.5, fused=rng.random() < 0.5, tokens=tokens)
    if op == "cache_write":
        T = _log(rng, 1, 65536)
        B = rng.randint(1, 32) if T <= 512 else 1
        length = 0 if T > 512 else _log(rng, 1, 4000)
        return dict(op=op, B=B, Hkv=Hkv, T=T, cap=length + T + rng.randint(0, 100), length=length, d=d,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), fused=rng.random() < 0.5, ragged=rng.random() < 0.5)
    if op == "cache_read":
        T, row0 = _log(rng, 1, 65536), rng.randint(0, 300)
        return dict(op=op, B=rng.randint(1, 4) if T <= 8192 else 1, Hkv=Hkv, T=T, cap=row0 + T + rng.randint(0, 100),
                    row0=row0, d=d, dtype=rng.choice(["bf16", "bf16", "f32"]))
    T = rng.choice([1, 1, _log(rng, 2, 64), _log(rng, 2, 64)])
    dtype, cache = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("bf16", "e4m3"), ("bf16", "e4m3"), ("f32", "f32"),
                               ("f32", "e4m3")])
    B = _log(rng, 1, 16)
    length = _log(rng, 1, 32768) if dtype == "bf16" else _log(rng, 1, 8192)
    length = max(1, min(length, 262144 // (B * Hkv)))
    return dict(op=op, B=B, H=Hkv * G, Hkv=Hkv, T=T, cap=length + T + rng.randint(0, 200), length=length, d=d,
                dtype=dtype, cache=cache, tree=rng.random() < 0.7, ragged=rng.random() < 0.5, blank=rng.random() < 0.2)


def _lengths(c):
    """Prefix lengths of the batch: all `length`, or (ragged) spread below it."""
    B = c["B"]
    lens = [c["length"] - (c["length"] * b) // (B + 1) if c["ragged"] else c["length"] for b in range(B)]
    if c.get("blank"):
        lens[-1] = 0
    return lens


def _counts(c):
    """Tokens of each sequence in this step: all T, or (ragged) 1 to T of them."""
    return [1 + (5 * b + c["T"] - 1) % c["T"] if c["ragged"] else c["T"] for b in range(c["B"])]


def work(case):
    c = case
    if c["op"] == "norm_rope":
        elems = c["B"] * (c["H"] + c["Hkv"]) * c["L"] * c["d"]
        passes = 3 if c["backward"] else 2  # x (and dy) read, y or dx written
        return {"bytes": passes * elems * SIZE[c["dtype"]] + 16 * c["d"], "flops": (18 if c["backward"] else 8) * elems}
    if c["op"] == "cache_write":
        rows = 2 * c["Hkv"] * sum(_counts(c))
        return {"bytes": rows * (c["d"] * (SIZE[c["dtype"]] + 1) + 1), "flops": 2 * rows * c["d"]}
    if c["op"] == "cache_read":
        rows = 2 * c["B"] * c["Hkv"] * c["T"]
        return {"bytes": rows * (c["d"] * (SIZE[c["dtype"]] + 1) + 1), "flops": rows * c["d"]}
    keys = sum(_lengths(c)) + sum(_counts(c))
    kv = 2 * c["Hkv"] * keys * (c["d"] * SIZE[c["cache"]] + (1 if c["cache"] == "e4m3" else 0))
    q = c["B"] * c["H"] * c["T"]
    return {"bytes": kv + q * (2 * c["d"] * SIZE[c["dtype"]] + 4), "flops": 4 * c["H"] * c["T"] * keys * c["d"]}


# --------------------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------------------
def _randn(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _heads(c, rows, g, dtype):
    """q [B, H, rows, d], k and v [B, Hkv, rows, d]: tensors of their own, or slices of one fused projection."""
    B, Hkv, d = c["B"], c["Hkv"], c["d"]
    H = c.get("H", Hkv)
    if c["fused"]:
        x = _randn((B, rows, H + 2 * Hkv, d), g).to(dtype)
        return tuple(t.transpose(1, 2) for t in x.split([H, Hkv, Hkv], dim=2))
    return tuple(_randn((B, h, rows, d), g).to(dtype) for h in (H, Hkv, Hkv))


def _quantised(x):
    """(e4m3 values, uint8 exponent + 127) of float32 rows: the smallest power of two 2^e, e >= -126, that brings
    the row's largest magnitude to at most 448."""
    mant, ex = torch.frexp(x.abs().amax(-1))
    e = torch.where(mant > 0.875, ex - 8, ex - 9)
    e = torch.where(mant == 0, torch.full_like(e, -126), e).clamp(-126, 120)
    return torch.ldexp(x, -e.unsqueeze(-1)).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _cache(c, rows_in_use, g):
    """k, v [B, Hkv, cap, d] in the cache's type and their exponents, every row filled (rows behind a sequence
    hold what an earlier one left there); the first key of each sequence draws much of the attention."""
    shape = (c["B"], c["Hkv"], c["cap"], c["d"])
    k, v = _randn(shape, g), _randn(shape, g)
    k[:, :, 0] *= 2.0
    if c["cache"] != "e4m3":
        return k.to(DTYPES[c["cache"]]), v.to(DTYPES[c["cache"]]), None, None
    (kq, ke), (vq, ve) = _quantised(k), _quantised(v)
    return kq, vq, ke, ve


def _tree_mask(c, seed):
    """[B, T, T]: drafted token t sees itself and its ancestors in a random tree."""
    r = np.random.default_rng(seed)
    B, T = c["B"], c["T"]
    m = np.zeros((B, T, T), dtype=bool)
    for b in range(B):
        for t in range(T):
            if t and r.random() < 0.9:
                m[b, t] = m[b, r.integers(0, t)]
            m[b, t, t] = True
    if c["blank"]:
        m[-1, 0] = False  # with an empty prefix: a row that sees no key at all
    return torch.from_numpy(m).cuda()


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 17)
    i32 = dict(dtype=torch.int32, device="cuda")
    st = {"c": c}
    if c["op"] == "norm_rope":
        dt = DTYPES[c["dtype"]]
        st["q"], st["k"], _ = _heads(c, c["L"], g, dt)
        st["wq"], st["wk"] = (1.0 + 0.1 * _randn((c["d"],), g) for _ in range(2))
        st["pos"] = None
        if c["tokens"]:  # each sequence's tokens stand behind a prefix of its own length
            start = torch.randint(0, 131072, (c["B"], 1), generator=g, device="cuda")
            st["pos"] = (start + torch.arange(c["L"], device="cuda")).to(torch.int32)
        if c["backward"]:
            st["dyq"] = _randn((c["B"], c["H"], c["L"], c["d"]), g).to(dt)
            st["dyk"] = _randn((c["B"], c["Hkv"], c["L"], c["d"]), g).to(dt)
    elif c["op"] == "cache_write":
        _, st["k"], st["v"] = _heads(c, c["T"], g, DTYPES[c["dtype"]])
        shape = (c["B"], c["Hkv"], c["cap"])
        st["cache"] = tuple(torch.zeros((*shape, c["d"]), dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)) + \
            tuple(torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2))
        st["lens"] = torch.tensor(_lengths(c), **i32)
        st["ntok"] = torch.tensor(_counts(c), **i32) if c["ragged"] else None
    elif c["op"] == "cache_read":
        st["cache"] = _cache({**c, "cache": "e4m3"}, c["cap"], g)
    else:
        st["q"] = _randn((c["B"], c["H"], c["T"], c["d"]), g).to(DTYPES[c["dtype"]])
        st["cache"] = _cache(c, c["cap"], g)
        st["lens"] = torch.tensor(_lengths(c), **i32)
        st["ntok"] = torch.tensor(_counts(c), **i32) if c["ragged"] else None
        st["mask"] = _tree_mask(c, seed) if c["tree"] else None
    return st


# --------------------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------------------
BASE, EPS = 500000.0, 1e-6


def run(state):
    c = state["c"]
    if own:
        return _run_own(c, state)
    if c["op"] == "norm_rope":
        return _plain_norm_rope(c, state)
    if c["op"] == "cache_write":
        return _plain_cache_write(c, state)
    if c["op"] == "cache_read":
        return _plain_cache_read(c, state)
    return _plain_tree(c, state)


def _run_own(c, st):
    import sequence_sharded_exact_gb300 as ra

    if c["op"] == "norm_rope":
        if c["backward"]:
            return ra.qk_norm_rope_bwd(st["q"], st["k"], st["wq"], st["wk"], st["dyq"], st["dyk"], c["n"], c["layout"],
                                       base=BASE, eps=EPS, positions=st["pos"])
        return ra.qk_norm_rope(st["q"], st["k"], st["wq"], st["wk"], c["n"], c["layout"], base=BASE, eps=EPS,
                               positions=st["pos"])
    cache = ra.KVCache(*st["cache"])
    if c["op"] == "cache_write":
        ra.cache_write(cache, st["k"], st["v"], st["lens"], ntok=st["ntok"])
        return st["cache"]
    if c["op"] == "cache_read":
        return ra.cache_read(cache, c["T"], row0=c["row0"], dtype=DTYPES[c["dtype"]])
    return ra.tree_fwd(st["q"], cache, st["lens"], mask=st["mask"], ntok=st["ntok"])


def _positions(c, st):
    """The natural position of every buffer row, [B or 1, 1, L]."""
    if st["pos"] is not None:
        return st["pos"][:, None, :]
    L, n = c["L"], c["n"]
    r = torch.arange(L, device="cuda")
    if c["layout"] == "striped":
        r = (r % (L // n)) * n + r // (L // n)
    elif c["layout"] == "zigzag":
        C = L // (2 * n)
        half, shard, off = (r // C) % 2, r // (2 * C), r % C
        r = torch.where(half == 0, shard, 2 * n - 1 - shard) * C + off
    return r[None, None, :]


def _angles(c, st):
    """cos and sin [.., L, d/2]; the angle itself in float64, where far positions keep their fraction of a turn."""
    freq = BASE ** (-2.0 * torch.arange(c["d"] // 2, device="cuda", dtype=torch.float64) / c["d"])
    a = _positions(c, st).double().unsqueeze(-1) * freq
    return a.cos().float(), a.sin().float()


def _turn(x, cos, sin):
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)


def _plain_norm_rope(c, st):
    cos, sin = _angles(c, st)
    if not c["backward"]:
        return tuple(_norm_turn(st[x], st[w], cos, sin) for x, w in (("q", "wq"), ("k", "wk")))
    (dq, dwq), (dk, dwk) = (_norm_turn_bwd(st[x], st[w], st[dy], cos, sin)
                            for x, w, dy in (("q", "wq", "dyq"), ("k", "wk", "dyk")))
    return dq, dk, dwq, dwk


def _norm_turn(x, w, cos, sin):
    f = x.float()
    return _turn(f * torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS) * w, cos, sin).to(x.dtype)


def _norm_turn_bwd(x, w, dy, cos, sin):
    f = x.float()
    r = torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS)
    g = _turn(dy.float(), cos, -sin)
    xh = f * r
    dw = (g * xh).sum((0, 1, 2))
    gw = g * w
    return (r * (gw - xh * (gw * xh).mean(-1, keepdim=True))).to(x.dtype), dw


def _plain_cache_write(c, st):
    kc, vc, ke, ve = st["cache"]
    t = torch.arange(c["T"], device="cuda")
    count = st["ntok"] if st["ntok"] is not None else torch.full_like(st["lens"], c["T"])
    written = (t[None, :] < count[:, None])[:, None, :]
    row = (st["lens"].long()[:, None] + t)[:, None, :].expand(-1, c["Hkv"], -1)
    for x, values, exps in ((st["k"], kc, ke), (st["v"], vc, ve)):
        q, e = _quantised(x.float())
        wide, values = row.unsqueeze(-1).expand(-1, -1, -1, c["d"]), values.view(torch.uint8)
        values.scatter_(2, wide, torch.where(written.unsqueeze(-1), q.view(torch.uint8), values.gather(2, wide)))
        exps.scatter_(2, row, torch.where(written, e, exps.gather(2, row)))
    return st["cache"]


def _values(x, e):
    return x.float() if e is None else torch.ldexp(x.float(), e.unsqueeze(-1).int() - 127)


def _plain_cache_read(c, st):
    kc, vc, ke, ve = st["cache"]
    s = slice(c["row0"], c["row0"] + c["T"])
    return tuple(_values(x[:, :, s], e[:, :, s]).to(DTYPES[c["dtype"]]) for x, e in ((kc, ke), (vc, ve)))


def _visible(c, st):
    """[B, T, cap]: which cache rows a drafted token sees -- the prefix, and of the step's own rows its mask's."""
    T, cap = c["T"], c["cap"]
    lens = st["lens"].long()[:, None]
    count = st["ntok"].long()[:, None] if st["ntok"] is not None else torch.full_like(lens, T)
    j = torch.arange(cap, device="cuda")[None, :]
    mask = st["mask"]
    if mask is None:
        mask = torch.ones((T, T), dtype=torch.bool, device="cuda").tril().expand(c["B"], T, T)
    at = (j - lens).clamp(0, T - 1)[:, None, :].expand(-1, T, -1)
    drafted = (j >= lens) & (j < lens + count)
    seen = (j < lens)[:, None, :] | (drafted[:, None, :] & mask.gather(2, at))
    return seen & (torch.arange(T, device="cuda")[None, :, None] < count[:, :, None])


def _plain_tree(c, st):
    B, H, Hkv, T, d = (c[x] for x in ("B", "H", "Hkv", "T", "d"))
    kc, vc, ke, ve = st["cache"]
    k, v = _values(kc, ke), _values(vc, ve)
    q = st["q"].float().view(B, Hkv, (H // Hkv) * T, d)
    seen = _visible(c, st)[:, None, None].expand(B, Hkv, H // Hkv, T, -1).reshape(B, Hkv, (H // Hkv) * T, -1)
    s = (torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(d)).masked_fill_(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(m.clamp_min(torch.finfo(torch.float32).min)).exp_()
    l = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / l.clamp_min(torch.finfo(torch.float32).tiny)
    lse = (m + l.log()).masked_fill(l == 0, -math.inf)
    return out.view(B, H, T, d).to(st["q"].dtype), lse.view(B, H, T)


# --------------------------------------------------------------------------------------------------
# the definitions in float64
# --------------------------------------------------------------------------------------------------
def exact(case, seed):
    c, st = case, prepare(case, seed)
    if c["op"] == "norm_rope":
        return _exact_norm_rope(c, st)
    if c["op"] == "cache_write":
        return _exact_cache_write(c, st)
    if c["op"] == "cache_read":
        s = slice(c["row0"], c["row0"] + c["T"])
        return tuple(x[:, :, s].double() * torch.exp2(e[:, :, s].double() - 127.0).unsqueeze(-1)
                     for x, e in zip(st["cache"][:2], st["cache"][2:]))
    return _exact_tree(c, st)


def _exact_norm_rope(c, st):
    L, n, d = c["L"], c["n"], c["d"]
    if st["pos"] is not None:
        pos = st["pos"].double().view(c["B"], 1, L, 1)
    else:  # the shards' natural positions, one shard after another
        rows, S = [], L // n
        for i in range(n):
            if c["layout"] == "contiguous":
                rows += range(i * S, (i + 1) * S)
            elif c["layout"] == "striped":
                rows += range(i, L, n)
            else:
                C = S // 2
                rows += list(range(i * C, (i + 1) * C)) + list(range((2 * n - 1 - i) * C, (2 * n - i) * C))
        pos = torch.tensor(rows, dtype=torch.float64, device="cuda").view(1, 1, L, 1)
    i = torch.arange(d // 2, dtype=torch.float64, device="cuda")
    z = torch.exp(1j * pos * torch.exp(-2.0 * i / d * math.log(BASE)))  # the rotation as a complex factor
    outs, grads = [], []
    for x, w, dy in (("q", "wq", "dyq"), ("k", "wk", "dyk")):
        ys, gx, gw = [], [], torch.zeros(d, dtype=torch.float64, device="cuda")
        for h in range(st[x].shape[1]):  # one head at a time keeps the float64 copies small
            v = st[x][:, h:h + 1].double()
            r = (v.pow(2).sum(-1, keepdim=True) / d + EPS).pow(-0.5)
            if not c["backward"]:
                ys.append(torch.view_as_real(torch.view_as_complex((v * r * st[w].double()).unflatten(-1, (d // 2, 2)).contiguous())
                                             * z).flatten(-2))
                continue
            g = torch.view_as_real(torch.view_as_complex(st[dy][:, h:h + 1].double().unflatten(-1, (d // 2, 2)).contiguous())
                                   * z.conj()).flatten(-2)
            gw += (g * v * r).sum((0, 1, 2))
            u = g * st[w].double()
            gx.append(u * r - v * r.pow(3) / d * (u * v).sum(-1, keepdim=True))
        if c["backward"]:
            outs.append(torch.cat(gx, 1))
            grads.append(gw)
        else:
            outs.append(torch.cat(ys, 1))
    return tuple(outs + grads)


def _exact_cache_write(c, st):
    """The exponents from logarithms in float64, the values as the nearest multiples of e4m3's steps, one sequence
    after another."""
    out_v = [torch.zeros(x.shape, dtype=torch.float64, device="cuda") for x in st["cache"][:2]]
    out_e = [torch.zeros(x.shape, dtype=torch.uint8, device="cuda") for x in st["cache"][2:]]
    lens, counts = _lengths(c), _counts(c)
    for x, ov, oe in zip((st["k"], st["v"]), out_v, out_e):
        for b in range(c["B"]):
            a = x[b, :, :counts[b]].double()
            big = a.abs().amax(-1)
            e = torch.ceil(torch.log2(big / 448.0))
            e = torch.where(big > 448.0 * torch.exp2(e), e + 1, torch.where(big <= 448.0 * torch.exp2(e - 1), e - 1, e)).clamp(-126, 120)
            y = a * torch.exp2(-e).unsqueeze(-1)
            step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3.0)
            ov[b, :, lens[b]:lens[b] + counts[b]] = torch.round(y / step) * step  # ties to even
            oe[b, :, lens[b]:lens[b] + counts[b]] = (e + 127).to(torch.uint8)
    return (*out_v, *out_e)


def _exact_tree(c, st):
    B, H, Hkv, T, d = (c[x] for x in ("B", "H", "Hkv", "T", "d"))
    lens, counts = _lengths(c), _counts(c)
    out = torch.zeros((B, H, T, d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, T), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        n, t = lens[b] + counts[b], counts[b]
        hide = torch.zeros((t, n), dtype=torch.float64, device="cuda")
        own_rows = torch.ones((t, t), device="cuda").tril().bool() if st["mask"] is None else st["mask"][b, :t, :t]
        hide[:, lens[b]:][~own_rows] = -math.inf
        for g in range(Hkv):
            k, v = (x[b, g, :n].double() for x in st["cache"][:2])
            if st["cache"][2] is not None:
                k, v = (x * torch.exp2(e[b, g, :n].double() - 127.0)[:, None] for x, e in ((k, st["cache"][2]), (v, st["cache"][3])))
            for h in range(g * (H // Hkv), (g + 1) * (H // Hkv)):
                s = st["q"][b, h, :t].double() @ k.T * d ** -0.5 + hide
                z = torch.logsumexp(s, -1)
                lse[b, h, :t] = z
                out[b, h, :t] = torch.where(z[:, None] == -math.inf, 0.0, torch.exp(s - z[:, None]).nan_to_num(0.0) @ v)
    return out, lse
