"""The operators as they are used together: a prompt through the norms, the rotation, the ring attention and the
cache, then steps of drafted tokens over it, each step's accepted tokens kept; every output against float64
attention over the whole sequence."""

import pytest
import torch

import cache_util as cu
import sequence_sharded_exact_gb300 as ra

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("cdt", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("d,G", [(128, 4), (64, 8)])
def test_prompt_then_drafted_tokens(cdt, d, G):
    torch.cuda.set_device(0)
    ra.device_status()
    B, Hkv, L, n, T, steps = 2, 2, 1024, 4, 4, 3
    H = Hkv * G
    g = torch.Generator().manual_seed(d)
    w = [(1 + 0.2 * torch.randn(d, generator=g)).to(DEV) for _ in range(2)]
    proj = lambda rows: torch.randn((B, rows, H + 2 * Hkv, d), generator=g).to(torch.bfloat16).to(DEV)  # noqa: E731

    def heads(x):
        return tuple(t.transpose(1, 2) for t in x.split([H, Hkv, Hkv], dim=2))

    # the prompt, in the zigzag order of four shards
    q, k, v = heads(proj(L))
    q, k = ra.qk_norm_rope(q, k, *w, n, "zigzag")
    v = v.contiguous()
    out, lse = ra.fwd(q, k, v, n, True, "zigzag")
    cache = ra.cache_alloc(B, Hkv, L + 64, d, cdt)
    ra.cache_write(cache, k, v)
    # the cache gives back the prompt's keys and values
    rk, rv = ra.cache_read(cache, L)
    # e4m3: half a step of a normal value is at most 2^-4 of it, of a subnormal one 2^-10 times the row's scale 2^e,
    # and a row's amax is above 224 * 2^e: 2^-10 / 224 = 2^-17.8 of amax
    for a, b in ((rk, k), (rv, v)):
        step, sub = (0.0, 0.0) if cdt == torch.bfloat16 else (2.0 ** -4, 2.0 ** -10 / 224)
        amax = b.float().abs().amax(-1, keepdim=True)
        over = (a.float() - b.float()).abs() - (step * b.float().abs() + sub * amax)
        assert float(over.max()) <= 0
    lens = torch.full((B,), L, dtype=torch.int32, device=DEV)
    for step in range(steps):
        q, k, v = heads(proj(T))
        mask = cu.random_tree(B, T, 100 * d + step).to(DEV)
        depth = mask.sum(-1).to(torch.int32) - 1  # a drafted token stands at its depth behind the prefix
        pos = (lens[:, None] + depth).to(torch.int32)
        q, k = ra.qk_norm_rope(q, k, *w, positions=pos)
        ra.cache_write(cache, k, v, lens)
        got = ra.tree_fwd(q, cache, lens, mask=mask)
        ck, cv = cu.cache_values(cache)
        cu.check_tree(got, cu.tree(q, ck, cv, lens.tolist(), mask.cpu(), None), 2.0 ** -8, torch.bfloat16, f"step {step}")
        # keep a path of the tree: token 0's deepest descendant by index, written again in order
        keep = [torch.nonzero(mask[b, T - 1].cpu()).flatten() for b in range(B)]
        idx = torch.zeros((B, T), dtype=torch.long)
        for b in range(B):
            idx[b, :len(keep[b])] = keep[b]
        at = idx.to(DEV)[:, None, :, None].expand(B, Hkv, T, d)
        count = torch.tensor([len(x) for x in keep], dtype=torch.int32, device=DEV)
        ra.cache_write(cache, k.gather(2, at), v.gather(2, at), lens, ntok=count)
        lens = lens + count
    assert ra.device_status() == 0


def test_the_step_of_single_tokens_equals_the_ring_forward():
    """The last row of the causal ring forward is the decoding of that token over the others' cache."""
    torch.cuda.set_device(0)
    B, H, Hkv, L, d = 1, 8, 2, 2048, 128
    g = torch.Generator().manual_seed(9)
    q, k, v = (torch.randn((B, h, L, d), generator=g).to(torch.bfloat16).to(DEV) for h in (H, Hkv, Hkv))
    out, lse = ra.fwd(q, k, v, 1, True, "contiguous")
    cache = ra.cache_alloc(B, Hkv, L, d, torch.bfloat16)
    ra.cache_write(cache, k, v)
    lens = torch.tensor([L - 1], dtype=torch.int32, device=DEV)
    o, l = ra.tree_fwd(q[:, :, -1:].contiguous(), cache, lens)
    ck, cv = cu.cache_values(cache)
    ref = cu.tree(q[:, :, -1:], ck, cv, [L - 1], None, None)
    cu.check_tree((o, l), ref, 2.0 ** -8, torch.bfloat16)
    # both are bf16 roundings of values within the weights' rounding of the exact one
    tol = 2 * (2.0 ** -8 * ref[2] + 2.0 ** -8 * ref[0].abs()) + 1e-4
    assert float(((out[:, :, -1:].cpu().double() - o.cpu().double()).abs() - tol).max()) <= 0
    assert float((lse[:, :, -1:] - l).abs().max()) <= 1e-4
