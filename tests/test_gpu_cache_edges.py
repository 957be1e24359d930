"""Cache operators on the GPU at edges of their kernels and at their limits."""
import pytest
import torch

import cache_util as cu
import permuted_block_sparse_b200 as pbs
from test_gpu_cache import inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("M,N,window,n_sink", [(2048, 2048, 512, 0), (2048, 2048, 512, 128), (2176, 4000, 1024, 113),
                                               (1500, 1500, 384, 0)])
def test_one_head_per_kv_head_windows_on_tile_bounds(M, N, window, n_sink, d):
    """One head per KV head: a slot holds 128 positions, so the second one's window
    starts a whole tile after the first's and its products run a tile ahead."""
    for seed in range(4):
        Q, K, V = inputs(400 + 3 * seed, 1, 4, 4, d, M, N)
        O, lse = pbs.pbs_attn_window(Q, K, V, window, n_sink)
        pbs.pbs_check_device()
        for h in range(4):
            one = [t[:, h:h + 1] for t in (Q, K, V)]
            cu.assert_attention(O[:, h:h + 1], lse[:, h:h + 1], cu.reference(*one, window, n_sink),
                                torch.ones(1, M, dtype=torch.bool, device="cuda"), f"seed {seed}, head {h}")


def test_head_groups_past_the_limit_are_refused():
    Q, K, V = inputs(1, 1, 129, 1, 64, 4, 300)
    lse = torch.zeros((1, 129, 4), device="cuda")
    for call in (lambda: pbs.pbs_attn_window(Q, K, V), lambda: pbs.pbs_attn_prefix(Q, K, V, K, V),
                 lambda: pbs.pbs_key_mass(Q, K, lse)):
        with pytest.raises(pbs.PbsError) as e:
            call()
        assert e.value.code == -2
