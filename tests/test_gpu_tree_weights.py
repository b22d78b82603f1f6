"""The normaliser of the attention over a cache: many keys that share a weight, in float32 output."""
import pytest
import torch

import cache_util as cu
import sequence_sharded_exact_gb300 as ra

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def _clean_status():
    torch.cuda.set_device(0)
    ra.device_status()
    yield
    assert ra.device_status() == 0


@pytest.mark.parametrize("cdt", [BF, E4M3])
@pytest.mark.parametrize("H,Hkv,T,d", [(8, 1, 8, 128), (8, 1, 8, 64), (4, 1, 64, 128), (4, 1, 64, 64)])
@pytest.mark.parametrize("n", [128, 700])
def test_keys_that_share_a_weight_are_averaged(H, Hkv, T, d, n, cdt):
    """Of every 128 keys the first 32 score 0 and the others alike, 3 to 7.5 binades above (each query its own): a running
    reference that follows the maximum in steps of 2^8 stays at the low ones, and all the high keys' weights are rounded
    the same way.  They are sums of 64 or 256 query rows per kv head.

    With e_j the relative rounding of weight j, out = sum (1 + e_j) w_j v_j / sum (1 + e_j) w_j: the high keys' common
    rounding cancels, the low keys' differs from it by at most 2^-8 + 2^-8, so out is off by at most
    1.02 * 2^-7 sum_low w_j |v_j - out|, and by the float32 sums, 2 n 2^-24 of sum w |v|, and the scores' and
    exponentials' error, 2 (2^-18 (1 + |s|) + 2^-20) between low and high keys.  A normaliser of unrounded weights leaves
    up to 2^-8 |out|, far above that."""
    x = torch.linspace(3.0, 7.5, H * T).view(1, H, T, 1)
    q = (x / (d ** 0.5 * 1.4426950408889634)).expand(1, H, T, d).to(BF).to(DEV).contiguous()
    low = torch.arange(n) % 128 < 32
    k = (~low).float().view(1, 1, n, 1).expand(1, Hkv, n, d)
    v = 1.0 + 0.1 * torch.randn((1, Hkv, n, d), generator=torch.Generator().manual_seed(n))
    cap = n + T
    cache = ra.cache_alloc(1, Hkv, cap, d, cdt)
    ra.cache_write(cache, k.to(BF).to(DEV).contiguous(), v.to(BF).to(DEV))
    mask = torch.zeros(T, T, dtype=torch.bool)
    out, lse = ra.tree_fwd(q, cache, torch.tensor([n], dtype=torch.int32, device=DEV), mask=mask.to(DEV), out_dtype=F32)
    kk, vv = cu.cache_values(cache)
    ref, ref_lse, mag, big = cu.tree(q, kk, vv, [n], mask, None)
    s_err = 2.0 ** -18 * (1 + big)
    assert float(((lse.cpu().double() - ref_lse).abs() - s_err - 2.0 ** -22 * ref_lse.abs()).max()) <= 0
    s = torch.einsum("htd,nd->htn", q[0].float().cpu().double(), kk[0, 0, :n]) / d ** 0.5
    w = torch.softmax(s, -1)
    apart = torch.einsum("htn,htnd->htd", w[..., low], (vv[0, 0, None, None, :n][:, :, low] - ref[0].unsqueeze(2)).abs())
    tol = (1.02 * 2.0 ** -7 + 2 * (s_err[0].unsqueeze(-1) + 2.0 ** -20)) * apart + 2 * n * 2.0 ** -24 * mag[0]
    over = (out[0].cpu().double() - ref[0]).abs() - tol
    assert float(over.max()) <= 0, f"off by {float(over.max()):.3e} beyond its bound ({float(tol.max()):.3e})"


@pytest.mark.parametrize("cdt", [BF, E4M3])
@pytest.mark.parametrize("H,Hkv,T,d", [(2, 1, 1, 128), (4, 2, 4, 64), (8, 2, 4, 128), (8, 2, 5, 128), (4, 1, 32, 64), (4, 1, 32, 128),
                                       (4, 1, 64, 128), (4, 1, 64, 64)])
@pytest.mark.parametrize("n", [90, 1500])
def test_float32_output_is_as_exact_as_its_sums(H, Hkv, T, d, n, cdt):
    """bfloat16 queries, output in float32: the weights go into the product as two bfloat16 parts, off by at most 2^-15 of
    themselves (over an e4m3 cache with up to 16 query rows per kv head as one float16, 2^-11), and the sums of n terms
    are float32's, (n / 16 + 16) 2^-23 of sum w |v|.  One bfloat16 weight would be off by up to 2^-8 of itself."""
    cap = n + T
    cache = ra.cache_alloc(1, Hkv, cap, d, cdt)
    g = torch.Generator().manual_seed(n)
    ra.cache_write(cache, *(torch.randn((1, Hkv, cap, d), generator=g).to(BF).to(DEV) for _ in range(2)))
    q, mask = torch.randn((1, H, T, d), generator=g).to(BF).to(DEV), cu.random_tree(1, T, 5)
    got = ra.tree_fwd(q, cache, torch.tensor([n], dtype=torch.int32, device=DEV), mask=mask.to(DEV), out_dtype=F32)
    weight_eps = 2.0 ** -11 if cdt == E4M3 and H // Hkv * T <= 16 else 2.0 ** -15
    cu.check_tree(got, cu.tree(q, *cu.cache_values(cache), [n], mask, None), weight_eps + (n / 16 + 16) * 2.0 ** -23, F32)
