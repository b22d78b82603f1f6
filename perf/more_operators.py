"""What is measured of the operators for long sequences that are seen through a window, and for images and video:
attention with a sliding window and a few first tokens that stay visible (whole sequences, forward and backward, and
new tokens over a key/value cache), and the rotation by positions with several axes (forward and backward).

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
BASE, EPS = 500000.0, 1e-6
# frequency pairs of each axis of the positions (time, height, width), per head dim
SECTIONS = {64: (8, 12, 12), 128: (16, 24, 24)}


# --------------------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------------------
def listed():
    return [
        # a windowed layer of the long-context training step (64K tokens in 16 zigzag shards, 32 query and 8 kv heads)
        dict(name="window_train_64k", op="window", B=1, H=32, Hkv=8, L=65536, d=128, n=16, layout="zigzag", window=4096,
             sinks=4, causal=True, dtype="bf16", backward=False),
        # the backward pass of such a layer over 32K tokens
        dict(name="window_train_32k_bwd", op="window", B=1, H=32, Hkv=8, L=32768, d=128, n=16, layout="zigzag",
             window=4096, sinks=4, causal=True, dtype="bf16", backward=True),
        # a short prompt through a narrow window: latency
        dict(name="window_prompt_1k", op="window", B=2, H=8, Hkv=2, L=1000, d=64, n=1, layout="contiguous", window=128,
             sinks=4, causal=True, dtype="bf16", backward=False),
        # a sequence that no tile divides, dealt out round-robin to 7 shards, gradients
        dict(name="window_odd_striped_bwd", op="window", B=2, H=12, Hkv=4, L=5005, d=128, n=7, layout="striped", window=640,
             sinks=20, causal=True, dtype="bf16", backward=True),
        # an encoder's layer: every token sees the 511 tokens on both sides of it
        dict(name="window_both_sides_16k", op="window", B=2, H=16, Hkv=16, L=16384, d=64, n=8, layout="striped", window=512,
             sinks=0, causal=False, dtype="bf16", backward=False),
        # a float32 check run of odd sizes, gradients
        dict(name="window_f32_odd_bwd", op="window", B=1, H=6, Hkv=2, L=1235, d=64, n=5, layout="striped", window=200,
             sinks=7, causal=True, dtype="f32", backward=True),
        # one token each of 64 ragged sequences, a window of 4096 rows over a bfloat16 cache
        dict(name="cache_window_batch", op="tree", B=64, H=32, Hkv=8, T=1, cap=16500, length=16384, d=128, window=4096,
             sinks=4, dtype="bf16", cache="bf16", tree=False, ragged=True, blank=False),
        # 8 drafted tokens each of 16 ragged sequences over the quantised cache, a narrower window
        dict(name="cache_window_drafted_e4m3", op="tree", B=16, H=32, Hkv=8, T=8, cap=33001, length=32768, d=128,
             window=1024, sinks=4, dtype="bf16", cache="e4m3", tree=True, ragged=True, blank=False),
        # a single sequence's next token: the smallest serving step
        dict(name="cache_window_one", op="tree", B=1, H=32, Hkv=8, T=1, cap=33001, length=32768, d=128, window=4096,
             sinks=4, dtype="bf16", cache="bf16", tree=False, ragged=False, blank=False),
        # video tokens in training: norms of the heads and the rotation by (time, height, width), and their gradients
        dict(name="axes_video_48k", op="axes", B=1, H=32, Hkv=8, L=49152, d=128, dtype="bf16", norm=True, spectrum="whole",
             backward=False, fused=True, grid=True),
        dict(name="axes_video_48k_bwd", op="axes", B=1, H=32, Hkv=8, L=49152, d=128, dtype="bf16", norm=True,
             spectrum="whole", backward=True, fused=True, grid=True),
        # a serving step of 16 sequences with 8 tokens each: the rotation alone, each axis with frequencies of its own
        dict(name="axes_step", op="axes", B=16, H=32, Hkv=8, L=8, d=64, dtype="f32", norm=False, spectrum="axis",
             backward=False, fused=False, grid=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["window", "window", "window", "tree", "tree", "axes"])
    d = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 4, 8])
    if op == "axes":
        grid = rng.random() < 0.6
        B, L = (rng.randint(1, 2), _log(rng, 64, 16384)) if grid else (rng.randint(1, 48), rng.randint(1, 64))
        return dict(op=op, B=B, H=Hkv * G, Hkv=Hkv, L=L, d=d, dtype=rng.choice(["bf16", "bf16", "f32"]), norm=rng.random() < 0.6,
                    spectrum=rng.choice(["whole", "axis"]), backward=rng.random() < 0.5, fused=rng.random() < 0.5, grid=grid)
    sinks = rng.choice([0, 0, 4, 4, rng.randint(1, 200)])
    if op == "window":
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        window = _log(rng, 16, 8192 if dtype == "bf16" else 1024)
        L = _log(rng, 64, 16384 if dtype == "bf16" else 4096)
        n, layout = rng.choice([1, 2, 4, 5, 8, 16]), rng.choice(["contiguous", "zigzag", "striped"])
        step = 2 * n if layout == "zigzag" else n
        L = max(1, L // step) * step
        return dict(op=op, B=rng.randint(1, 2), H=Hkv * G, Hkv=Hkv, L=L, d=d, n=n, layout=layout, window=window, sinks=sinks,
                    causal=rng.random() < 0.85, dtype=dtype, backward=rng.random() < 0.5)
    T = rng.choice([1, 1, _log(rng, 2, 64)])
    dtype, cache = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("bf16", "e4m3"), ("bf16", "e4m3"), ("f32", "f32"), ("f32", "e4m3")])
    B = _log(rng, 1, 32)
    length = max(1, min(_log(rng, 1, 32768), 1048576 // (B * Hkv)))
    return dict(op=op, B=B, H=Hkv * G, Hkv=Hkv, T=T, cap=length + T + rng.randint(0, 200), length=length, d=d,
                window=max(T, _log(rng, 16, 8192 if dtype == "bf16" else 2048)), sinks=sinks, dtype=dtype, cache=cache,
                tree=rng.random() < 0.5, ragged=rng.random() < 0.5, blank=rng.random() < 0.2)


def _lengths(c):
    """Prefix lengths of the batch: all `length`, or (ragged) spread below it."""
    B = c["B"]
    lens = [c["length"] - (c["length"] * b) // (B + 1) if c["ragged"] else c["length"] for b in range(B)]
    if c["blank"]:
        lens[-1] = 0
    return lens


def _counts(c):
    """Tokens of each sequence in this step: all T, or (ragged) 1 to T of them."""
    return [1 + (5 * b + c["T"] - 1) % c["T"] if c["ragged"] else c["T"] for b in range(c["B"])]


def _pairs(c):
    """(query, key) pairs that one head of one sequence of a window case sees."""
    L, W, S = c["L"], c["window"], c["sinks"]
    p = np.arange(L, dtype=np.int64)
    lo = np.maximum(p - W + 1, 0)
    hi = p if c["causal"] else np.minimum(p + W - 1, L - 1)
    pairs = (hi - lo + 1) + np.minimum(lo, S)
    if not c["causal"]:
        pairs = pairs + np.maximum(S - 1 - hi, 0)
    return int(pairs.sum())


def work(case):
    c = case
    d, size = c["d"], SIZE[c["dtype"]]
    if c["op"] == "axes":
        elems = c["B"] * (c["H"] + c["Hkv"]) * c["L"] * d
        passes = 3 if c["backward"] and c["norm"] else 2  # x or dy (both with a norm's gradient) read, y or dx written
        flops = (18 if c["backward"] else 8) if c["norm"] else 3
        return {"bytes": passes * elems * size + 12 * c["B"] * c["L"], "flops": flops * elems}
    if c["op"] == "window":
        q, kv = c["B"] * c["H"] * c["L"], c["B"] * c["Hkv"] * c["L"]
        pairs = c["B"] * c["H"] * _pairs(c)
        if c["backward"]:  # q, out, dout, dq; k, v, dk, dv; lse
            return {"bytes": 4 * (q + kv) * d * size + 4 * q, "flops": 10 * pairs * d}
        return {"bytes": 2 * (q + kv) * d * size + 4 * q, "flops": 4 * pairs * d}
    keys = sum(min(l, c["window"] - 1 + min(c["sinks"], max(0, l - c["window"] + 1))) + n for l, n in zip(_lengths(c), _counts(c)))
    kv = 2 * c["Hkv"] * keys * (d * SIZE[c["cache"]] + (1 if c["cache"] == "e4m3" else 0))
    q = c["B"] * c["H"] * c["T"]
    return {"bytes": kv + q * (2 * d * size + 4), "flops": 4 * c["H"] * c["T"] * keys * d}


# --------------------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------------------
def _randn(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _quantised(x):
    """(e4m3 values, uint8 exponent + 127) of float32 rows: the smallest power of two 2^e, e >= -126, that brings
    the row's largest magnitude to at most 448."""
    mant, ex = torch.frexp(x.abs().amax(-1))
    e = torch.where(mant > 0.875, ex - 8, ex - 9)
    e = torch.where(mant == 0, torch.full_like(e, -126), e).clamp(-126, 120)
    return torch.ldexp(x, -e.unsqueeze(-1)).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _cache(c, g):
    """k, v [B, Hkv, cap, d] in the cache's type and their exponents, every row filled (rows behind a sequence
    hold what an earlier one left there); the first keys of each sequence draw much of the attention."""
    shape = (c["B"], c["Hkv"], c["cap"], c["d"])
    k, v = _randn(shape, g), _randn(shape, g)
    k[:, :, :4] *= 2.0
    if c["cache"] != "e4m3":
        return k.to(DTYPES[c["cache"]]), v.to(DTYPES[c["cache"]]), None, None
    (kq, ke), (vq, ve) = _quantised(k), _quantised(v)
    return kq, vq, ke, ve


def _tree(c, seed):
    """A random tree of drafted tokens: [B, T, T] truth values, token t sees itself and its ancestors; and how deep
    each lies, [B, T]."""
    r = np.random.default_rng(seed)
    B, T = c["B"], c["T"]
    m, depth = np.zeros((B, T, T), dtype=bool), np.zeros((B, T), dtype=np.int32)
    for b in range(B):
        for t in range(T):
            if t and r.random() < 0.9:
                parent = r.integers(0, t)
                m[b, t], depth[b, t] = m[b, parent], depth[b, parent] + 1
            m[b, t, t] = True
    if c["blank"]:
        m[-1, 0] = False  # with an empty prefix: a row that sees no key at all
    return torch.from_numpy(m).cuda(), torch.from_numpy(depth).cuda()


def _grid(c, g):
    """Positions [3, B, L] of a few text tokens (all three axes alike) in front of a video's patches (time, height,
    width, each counted from the text's end), or (no grid) of tokens far into a sequence."""
    B, L = c["B"], c["L"]
    t = torch.arange(L, device="cuda")
    if not c["grid"]:
        start = torch.randint(0, 131072, (3, B, 1), generator=g, device="cuda")
        return (start + t).to(torch.int32).contiguous()
    text = torch.randint(0, 1 + L // 16, (B, 1), generator=g, device="cuda")
    width = max(1, math.isqrt(L // 16))
    at = (t - text).clamp_min(0)
    axes = torch.stack((at // (width * width), at // width % width, at % width)) + text
    return torch.where(t < text, t.expand_as(axes), axes).to(torch.int32).contiguous()


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 29)
    i32 = dict(dtype=torch.int32, device="cuda")
    dt, st = DTYPES[c["dtype"]], {"c": c}
    B, H, Hkv, d = c["B"], c["H"], c["Hkv"], c["d"]
    if c["op"] == "window":
        L = c["L"]
        q, k, v = (_randn((B, h, L, d), g) for h in (H, Hkv, Hkv))
        k[:, :, _rows(c)[:4]] *= 1.5  # the first tokens draw attention from everywhere
        st["q"], st["k"], st["v"] = q.to(dt), k.to(dt), v.to(dt)
        if c["backward"]:  # the forward's results, which the training step has kept, and the gradient of its output
            st["out"], st["lse"] = _plain_window(c, st)
            st["dout"] = _randn((B, H, L, d), g).to(dt)
    elif c["op"] == "tree":
        st["q"] = _randn((B, H, c["T"], d), g).to(dt)
        st["cache"] = _cache(c, g)
        st["lens"] = torch.tensor(_lengths(c), **i32)
        st["ntok"] = torch.tensor(_counts(c), **i32) if c["ragged"] else None
        st["mask"], st["pos"] = None, None
        if c["tree"]:
            st["mask"], depth = _tree(c, seed)
            st["pos"] = st["lens"][:, None] + depth
    else:
        rows = c["L"]
        if c["fused"]:  # slices of one projection [B, rows, H + 2 Hkv, d]
            x = _randn((B, rows, H + 2 * Hkv, d), g).to(dt)
            st["q"], st["k"], _ = (t.transpose(1, 2) for t in x.split([H, Hkv, Hkv], dim=2))
        else:
            st["q"], st["k"] = (_randn((B, h, rows, d), g).to(dt) for h in (H, Hkv))
        st["wq"], st["wk"] = (1.0 + 0.1 * _randn((d,), g) for _ in range(2)) if c["norm"] else (None, None)
        st["pos"] = _grid(c, g)
        if c["backward"]:
            st["dyq"], st["dyk"] = (_randn((B, h, rows, d), g).to(dt) for h in (H, Hkv))
    return st


# --------------------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------------------
def run(state):
    c = state["c"]
    if own:
        return _run_own(c, state)
    if c["op"] == "window":
        return _plain_window_bwd(c, state) if c["backward"] else _plain_window(c, state)
    if c["op"] == "tree":
        return _plain_tree(c, state)
    return _plain_axes_bwd(c, state) if c["backward"] else _plain_axes(c, state)


def _run_own(c, st):
    import sequence_sharded_exact_gb300 as ra

    if c["op"] == "window":
        how = dict(sinks=c["sinks"], causal=c["causal"], layout=c["layout"])
        if c["backward"]:
            return ra.window_bwd(st["q"], st["k"], st["v"], st["out"], st["lse"], st["dout"], c["n"], c["window"],
                                 grad_dtype=st["q"].dtype, **how)
        return ra.window_fwd(st["q"], st["k"], st["v"], c["n"], c["window"], **how)
    if c["op"] == "tree":
        return ra.tree_fwd(st["q"], ra.KVCache(*st["cache"]), st["lens"], mask=st["mask"], ntok=st["ntok"],
                           window=c["window"], sinks=c["sinks"], positions=st["pos"])
    how = dict(base=BASE, eps=EPS, spectrum=c["spectrum"])
    if c["backward"]:
        return ra.qk_rope_axes_bwd(st["dyq"], st["dyk"], st["pos"], SECTIONS[c["d"]], q=st["q"] if c["norm"] else None,
                                   k=st["k"] if c["norm"] else None, wq=st["wq"], wk=st["wk"], **how)
    return ra.qk_rope_axes(st["q"], st["k"], st["pos"], SECTIONS[c["d"]], wq=st["wq"], wk=st["wk"], **how)


# ---- whole sequences through a window --------------------------------------------------------------
def _rows(c):
    """The buffer row of every natural position."""
    L, n = c["L"], c["n"]
    p = torch.arange(L, device="cuda")
    if c["layout"] == "striped":
        return p % n * (L // n) + p // n
    if c["layout"] == "zigzag":
        C = L // (2 * n)
        chunk, off = p // C, p % C
        return torch.where(chunk < n, 2 * chunk, 2 * (2 * n - 1 - chunk) + 1) * C + off
    return p


class _Band:
    """The natural order of a case's tensors, cut into blocks of queries and the keys that their windows reach, and the
    first keys, which every query reaches."""

    def __init__(self, c):
        self.c, self.rows = c, _rows(c)
        L, W, self.S = c["L"], min(c["window"], c["L"]), min(c["sinks"], c["L"])
        self.block = min(1024, L)
        self.nb = -(-L // self.block)
        self.front, self.back = W - 1, 0 if c["causal"] else W - 1
        self.keys = self.block + self.front + self.back
        p = torch.arange(self.nb * self.block, device="cuda").view(self.nb, 1, self.block, 1)
        j = (torch.arange(self.nb, device="cuda") * self.block - self.front).view(-1, 1, 1, 1) + torch.arange(self.keys, device="cuda")
        self.hidden = (j < 0) | (j >= L) | (p - j >= W) | (j > p if c["causal"] else j - p >= W)
        j = torch.arange(self.S, device="cuda")
        self.hidden_first = (j > p) | (p - j < W) if c["causal"] else (p - j).abs() < W

    def queries(self, x):  # [B, H, L, d] -> [B, Hkv, nb, G * block, d]
        c, d = self.c, x.shape[-1]
        x = torch.nn.functional.pad(x[:, :, self.rows].float(), (0, 0, 0, self.nb * self.block - c["L"]))
        return x.view(c["B"], c["Hkv"], -1, self.nb, self.block, d).transpose(2, 3).reshape(c["B"], c["Hkv"], self.nb, -1, d)

    def back_to(self, x, like):  # and back, to the layout's order
        c, d = self.c, x.shape[-1]
        x = x.view(c["B"], c["Hkv"], self.nb, -1, self.block, d).transpose(2, 3).reshape(c["B"], c["H"], -1, d)
        out = torch.empty((c["B"], c["H"], c["L"], d), dtype=like, device="cuda")
        out[:, :, self.rows] = x[:, :, :c["L"]].to(like)
        return out

    def windows(self, x):  # [B, Hkv, L, d] -> [B, Hkv, nb, d, keys] and the first keys [B, Hkv, 1, d, S]
        x = x[:, :, self.rows].float()
        pad = self.nb * self.block - self.c["L"] + self.back
        return torch.nn.functional.pad(x, (0, 0, self.front, pad)).unfold(2, self.keys, self.block), x[:, :, None, :self.S].transpose(-1, -2)

    def gather(self, near, first, like):  # gradients of windows [B, Hkv, nb, keys, d] and of first keys [B, Hkv, nb, S, d]
        c = self.c
        B, Hkv, d = c["B"], c["Hkv"], c["d"]
        at = (torch.arange(self.nb, device="cuda") * self.block)[:, None] + torch.arange(self.keys, device="cuda")
        x = torch.zeros((B, Hkv, self.front + self.nb * self.block + self.back, d), device="cuda")
        x.index_add_(2, at.view(-1), near.reshape(B, Hkv, -1, d))
        x = x[:, :, self.front:self.front + c["L"]]
        x[:, :, :self.S] += first.sum(2)
        out = torch.empty((B, Hkv, c["L"], d), dtype=like, device="cuda")
        out[:, :, self.rows] = x.to(like)
        return out

    def scores(self, q, k):
        """Both kinds of keys' scores, hidden ones -infinity."""
        c = self.c
        s = []
        for keys, hidden in zip(k, (self.hidden, self.hidden_first)):
            x = torch.matmul(q, keys).mul_(1.0 / math.sqrt(c["d"]))
            x.view(c["B"], c["Hkv"], self.nb, c["H"] // c["Hkv"], self.block, x.shape[-1]).masked_fill_(hidden, -math.inf)
            s.append(x)
        return s


def _plain_window(c, st):
    b = _Band(c)
    near, first = b.scores(b.queries(st["q"]), b.windows(st["k"]))
    m = near.amax(-1, keepdim=True)
    if b.S:
        m = torch.maximum(m, first.amax(-1, keepdim=True))
    m = m.clamp_min(torch.finfo(torch.float32).min)  # (rows behind the sequence see nothing)
    near, first = near.sub_(m).exp_(), first.sub_(m).exp_()
    v, v_first = b.windows(st["v"])
    l = (near.sum(-1, keepdim=True) + first.sum(-1, keepdim=True)).clamp_min(torch.finfo(torch.float32).tiny)
    out = (torch.matmul(near, v.transpose(-1, -2)) + torch.matmul(first, v_first.transpose(-1, -2))) / l
    return b.back_to(out, st["q"].dtype), b.back_to(m + l.log(), torch.float32).squeeze(-1)


def _plain_window_bwd(c, st):
    b, scale = _Band(c), 1.0 / math.sqrt(c["d"])
    q, dout, dt = b.queries(st["q"]), b.queries(st["dout"]), st["q"].dtype
    lse = b.queries(st["lse"].unsqueeze(-1))
    D = (dout * b.queries(st["out"])).sum(-1, keepdim=True)
    k, v = b.windows(st["k"]), b.windows(st["v"])
    dq, dk, dv = 0.0, [], []
    for s, keys, values in zip(b.scores(q, k), k, v):  # the window's keys, then the first ones
        p = s.sub_(lse).exp_()
        dv.append(torch.matmul(p.transpose(-1, -2), dout))
        ds = torch.matmul(dout, values).sub_(D).mul_(p).mul_(scale)
        dq = dq + torch.matmul(ds, keys.transpose(-1, -2))
        dk.append(torch.matmul(ds.transpose(-1, -2), q))
    return b.back_to(dq, dt), b.gather(*dk, dt), b.gather(*dv, dt)


# ---- new tokens over a cache -----------------------------------------------------------------------
def _plain_tree(c, st):
    B, H, Hkv, T, d, W, S = (c[x] for x in ("B", "H", "Hkv", "T", "d", "window", "sinks"))
    kc, vc, ke, ve = st["cache"]
    lens = st["lens"].long()[:, None]
    count = st["ntok"].long()[:, None] if st["ntok"] is not None else torch.full_like(lens, T)
    # the rows that any of the tokens may see: the first ones, then from the window's far end to the last token
    reach = min(W - 1, c["cap"])
    first = torch.arange(min(S, c["cap"]), device="cuda").expand(B, -1)
    rows = torch.cat((first, lens - reach + torch.arange(reach + T, device="cuda")), 1)
    twice = torch.zeros_like(rows, dtype=torch.bool)
    twice[:, :first.shape[1]] = first >= lens - reach
    at = rows.clamp(0, c["cap"] - 1)
    b, h = torch.arange(B, device="cuda")[:, None, None], torch.arange(Hkv, device="cuda")[None, :, None]
    k, v = (x[b, h, at[:, None]].float() if e is None else torch.ldexp(x[b, h, at[:, None]].float(), e[b, h, at[:, None]].unsqueeze(-1).int() - 127)
            for x, e in ((kc, ke), (vc, ve)))
    # what each token sees of them
    pos = (st["pos"].long() if st["pos"] is not None else lens + torch.arange(T, device="cuda")).clamp_min(0)
    j = rows[:, None, :]
    prefix = (j >= 0) & (j < lens[:, :, None]) & ((j < S) | (pos[:, :, None] - j < W))
    mask = st["mask"] if st["mask"] is not None else torch.ones((T, T), dtype=torch.bool, device="cuda").tril().expand(B, T, T)
    drafted = (j >= lens[:, :, None]) & (j < (lens + count)[:, :, None])
    seen = (prefix | (drafted & mask.gather(2, (j - lens[:, :, None]).clamp(0, T - 1).expand(-1, T, -1)))) & ~twice[:, None, :]
    seen = seen & (torch.arange(T, device="cuda") < count)[:, :, None]
    q = st["q"].float().view(B, Hkv, (H // Hkv) * T, d)
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d))
    s.view(B, Hkv, H // Hkv, T, -1).masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(m.clamp_min(torch.finfo(torch.float32).min)).exp_()
    l = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / l.clamp_min(torch.finfo(torch.float32).tiny)
    lse = (m + l.log()).masked_fill(l == 0, -math.inf)
    return out.view(B, H, T, d).to(st["q"].dtype), lse.view(B, H, T)


# ---- rotation by several axes ------------------------------------------------------------------------
def _angles(c, st):
    """cos and sin [B, 1, L, d/2]; the angle itself in float64, where far positions keep their fraction of a turn."""
    sections = SECTIONS[c["d"]]
    axis = torch.repeat_interleave(torch.arange(3, device="cuda"), torch.tensor(sections, device="cuda"))
    if c["spectrum"] == "whole":
        part = torch.arange(c["d"] // 2, device="cuda", dtype=torch.float64) / (c["d"] // 2)
    else:
        part = torch.cat([torch.arange(m, device="cuda", dtype=torch.float64) / m for m in sections])
    a = st["pos"][axis].permute(1, 2, 0).double() * BASE ** -part
    return a.cos().float()[:, None], a.sin().float()[:, None]


def _turn(x, cos, sin):
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)


def _plain_axes(c, st):
    cos, sin = _angles(c, st)
    out = []
    for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])):
        f = x.float()
        if c["norm"]:
            f = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS) * w
        out.append(_turn(f, cos, sin).to(x.dtype))
    return tuple(out)


def _plain_axes_bwd(c, st):
    cos, sin = _angles(c, st)
    dx, dw = [], []
    for x, w, dy in ((st["q"], st["wq"], st["dyq"]), (st["k"], st["wk"], st["dyk"])):
        g = _turn(dy.float(), cos, -sin)
        if c["norm"]:
            f = x.float()
            r = torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS)
            xh = f * r
            dw.append((g * xh).sum((0, 1, 2)))
            g = g * w
            g = r * (g - xh * (g * xh).mean(-1, keepdim=True))
        dx.append(g.to(dy.dtype))
    return tuple(dx + (dw or [None, None]))


# --------------------------------------------------------------------------------------------------
# the definitions in float64
# --------------------------------------------------------------------------------------------------
def exact(case, seed):
    c, st = case, prepare(case, seed)
    if c["op"] == "window":
        return _exact_window(c, st)
    if c["op"] == "tree":
        return _exact_tree(c, st)
    return _exact_axes(c, st)


def _order(c):
    """The natural position of every buffer row: the shards' positions, one shard after another."""
    L, n = c["L"], c["n"]
    S, rows = L // n, []
    for i in range(n):
        if c["layout"] == "contiguous":
            rows += range(i * S, (i + 1) * S)
        elif c["layout"] == "striped":
            rows += range(i, L, n)
        else:
            C = S // 2
            rows += list(range(i * C, (i + 1) * C)) + list(range((2 * n - 1 - i) * C, (2 * n - i) * C))
    return torch.tensor(rows, device="cuda")


def _exact_window(c, st):
    """Head by head over blocks of 2048 queries in natural order, each against the slice of keys from its first query's
    window to its last's, and the first keys before that slice (or behind it)."""
    B, H, Hkv, L, d, W, S = (c[x] for x in ("B", "H", "Hkv", "L", "d", "window", "sinks"))
    order = _order(c)
    at = torch.argsort(order)  # natural position -> buffer row
    f64 = dict(dtype=torch.float64, device="cuda")
    if c["backward"]:
        res = [torch.zeros((B, h, L, d), **f64) for h in (H, Hkv, Hkv)]
    else:
        res = [torch.zeros((B, H, L, d), **f64), torch.zeros((B, H, L), **f64)]
    for b in range(B):
        for h in range(H):
            g = h // (H // Hkv)
            k, v, q = st["k"][b, g, at].double(), st["v"][b, g, at].double(), st["q"][b, h, at].double()
            for a in range(0, L, 2048):
                e = min(L, a + 2048)
                lo, hi = max(0, a - W + 1), e if c["causal"] else min(L, e + W - 1)
                j = torch.cat([torch.arange(0, min(S, lo), device="cuda"), torch.arange(lo, hi, device="cuda"),
                               torch.arange(hi, 0 if c["causal"] else max(hi, min(S, L)), device="cuda") if not c["causal"] else
                               torch.arange(0, device="cuda")])
                p = torch.arange(a, e, device="cuda")[:, None]
                see = ((p - j).abs() < W) | (j < S)
                if c["causal"]:
                    see &= j <= p
                kj, vj, rows = k[j], v[j], at[a:e]
                s = (q[a:e] @ kj.T) * d ** -0.5
                s[~see] = -math.inf
                if not c["backward"]:
                    z = torch.logsumexp(s, -1)
                    res[1][b, h, rows] = z
                    res[0][b, h, rows] = torch.exp(s - z[:, None]) @ vj
                    continue
                do = st["dout"][b, h, rows].double()
                w = torch.exp(s - st["lse"][b, h, rows].double()[:, None])
                ds = w * (do @ vj.T - (do * st["out"][b, h, rows].double()).sum(-1, keepdim=True)) * d ** -0.5
                res[0][b, h, rows] = ds @ kj
                res[1][b, g].index_add_(0, at[j], ds.T @ q[a:e])
                res[2][b, g].index_add_(0, at[j], w.T @ do)
    return tuple(res)


def _exact_tree(c, st):
    B, H, Hkv, T, d, W, S = (c[x] for x in ("B", "H", "Hkv", "T", "d", "window", "sinks"))
    lens, counts = _lengths(c), _counts(c)
    out = torch.zeros((B, H, T, d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, T), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        n, t = lens[b] + counts[b], counts[b]
        where = torch.arange(n, device="cuda")[None, :]
        pos = torch.arange(lens[b], n, device="cuda")[:, None] if st["pos"] is None else st["pos"][b, :t].long()[:, None]
        see = (where > pos - W) | (where < S)
        see[:, lens[b]:] = torch.ones((t, t), device="cuda").tril().bool() if st["mask"] is None else st["mask"][b, :t, :t]
        hide = torch.zeros((t, n), dtype=torch.float64, device="cuda").masked_fill_(~see, -math.inf)
        keep = see.any(0)
        for g in range(Hkv):
            k, v = (x[b, g, :n][keep].double() for x in st["cache"][:2])
            if st["cache"][2] is not None:
                k, v = (x * torch.exp2(e[b, g, :n][keep].double() - 127.0)[:, None] for x, e in ((k, st["cache"][2]), (v, st["cache"][3])))
            for h in range(g * (H // Hkv), (g + 1) * (H // Hkv)):
                s = st["q"][b, h, :t].double() @ k.T * d ** -0.5 + hide[:, keep]
                z = torch.logsumexp(s, -1)
                lse[b, h, :t] = z
                out[b, h, :t] = torch.where(z[:, None] == -math.inf, 0.0, torch.exp(s - z[:, None]).nan_to_num(0.0) @ v)
    return out, lse


def _exact_axes(c, st):
    d, z = c["d"], []
    i = 0
    for axis, m in enumerate(SECTIONS[d]):  # the rotation as a complex factor, axis by axis
        for u in range(m):
            part = i / (d // 2) if c["spectrum"] == "whole" else u / m
            z.append(torch.exp(1j * st["pos"][axis].double() * math.exp(-part * math.log(BASE))))
            i += 1
    z = torch.stack(z, -1)[:, None]

    def turned(x, by):
        return torch.view_as_real(torch.view_as_complex(x.unflatten(-1, (d // 2, 2)).contiguous()) * by).flatten(-2)

    outs, grads = [], []
    for x, w, dy in (("q", "wq", "dyq"), ("k", "wk", "dyk")):
        ys, gw = [], torch.zeros(d, dtype=torch.float64, device="cuda") if c["norm"] else None
        for h in range(st[x].shape[1]):  # one head at a time keeps the float64 copies small
            v = st[x][:, h:h + 1].double()
            r = (v.pow(2).sum(-1, keepdim=True) / d + EPS).pow(-0.5)
            if not c["backward"]:
                ys.append(turned(v * r * st[w].double() if c["norm"] else v, z))
                continue
            g = turned(st[dy][:, h:h + 1].double(), z.conj())
            if c["norm"]:
                gw += (g * v * r).sum((0, 1, 2))
                u = g * st[w].double()
                g = u * r - v * r.pow(3) / d * (u * v).sum(-1, keepdim=True)
            ys.append(g)
        outs.append(torch.cat(ys, 1))
        if c["backward"]:
            grads.append(gw)
    return tuple(outs + grads)
