"""The workspace of the norms' backward is what its blocks write."""
import pytest

from sequence_sharded_exact_gb300 import binding


@pytest.mark.parametrize("d", [64, 128])
def test_a_pair_of_partial_sums_per_block_and_no_more(d):
    """Two blocks on each SM, each with a float32 sum per weight of q and of k; 160 SMs bound the chips it is built for (152)."""
    need = binding.library().ring_attn_qk_norm_rope_bwd_workspace_size(d)
    assert 152 * 2 * 2 * d * 4 <= need <= 160 * 2 * 2 * d * 4 + 255
