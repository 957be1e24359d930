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


# B, Hq, Hkv, d, M, N, window, n_sink: every kernel of the mass, groups that fill a tile of rows and that do not
MASS_FORMS = [(2, 8, 2, 128, 1, 500, 200, 5), (1, 6, 2, 64, 4, 500, 200, 5), (1, 8, 2, 128, 40, 500, 64, 3),
              (1, 6, 2, 64, 40, 700, 64, 0), (1, 8, 2, 128, 300, 300, 64, 0), (1, 6, 2, 64, 300, 500, 64, 130),
              (1, 32, 1, 64, 1100, 2000, 300, 0)]


@pytest.mark.parametrize("case", MASS_FORMS, ids=str)
def test_mass_of_rows_that_are_nan(case):
    """A NaN key makes the LSE of the rows that see it NaN; those make NaN of every
    key that they see and of no other.  A row of LSE -inf adds nothing to any key."""
    B, Hq, Hkv, d, M, N, window, n_sink = case
    G = Hq // Hkv
    Q, K, V = inputs(500 + M, B, Hq, Hkv, d, M, N)
    see, _ = cu.visible(B, M, N, window, n_sink, None, None, Q.device)
    at = N - max(M // 2, 1) - 20
    bad_key = torch.zeros((B, Hkv, N), dtype=torch.bool, device="cuda")
    for where, alone, off in ((at, False, False), (None, True, False), (None, False, True), (at, True, True)):
        K2, bad_key[:] = K.clone(), False
        if where is not None:
            K2[:, 0, where, 5], bad_key[:, 0, where] = float("nan"), True
        _, lse, _, _ = cu.reference(Q, K2, V, window, n_sink)
        lse = lse.float()
        if alone:
            lse[0, Hq - 1, M // 3] = float("nan")
        if off:                                                 # the second head of every group counts for nothing
            lse[:, 1::G] = -float("inf")
        prev = torch.rand((B, Hkv, N), device="cuda")
        got = pbs.pbs_key_mass(Q, K2, lse, prev, 0.5, window, n_sink)
        pbs.pbs_check_device()
        nan_row = torch.isnan(lse).reshape(B, Hkv, G, M, 1)
        live = (lse != -float("inf")).reshape(B, Hkv, G, M, 1)
        nan = (see[:, None, None] & live & (nan_row | bad_key[:, :, None, None])).any(3).any(2)
        assert torch.equal(torch.isnan(got), nan), (where, alone, off)
        want, tol = cu.reference_mass(Q, K, torch.where(torch.isnan(lse), -float("inf"), lse), prev, 0.5, window, n_sink)
        assert ((got.double() - want).abs() <= tol)[~nan].all()


@pytest.mark.parametrize("case", MASS_FORMS, ids=str)
def test_mass_of_keys_of_weight_zero(case):
    """An infinity in a key that makes every logit -inf gives the weight zero; in
    rows that are switched off by LSE -inf a logit of +inf counts for nothing."""
    B, Hq, Hkv, d, M, N, window, n_sink = case
    Q, K, V = inputs(600 + M, B, Hq, Hkv, d, M, N)
    Q[..., 3] = -Q[..., 3].abs() - 1
    clean = K.clone()
    inf_at = [N - M // 2 - 1, N - M // 2 - 30]
    K[:, :, inf_at, 3] = float("inf")
    _, lse, _, _ = cu.reference(Q, K, V, window, n_sink)
    lse = lse.float()
    got = pbs.pbs_key_mass(Q, K, lse, window=window, n_sink=n_sink)
    assert (got[:, :, inf_at] == 0).all() and torch.isfinite(got).all()
    want, tol = cu.reference_mass(Q, clean, lse, window=window, n_sink=n_sink)
    want[:, :, inf_at], tol[:, :, inf_at] = 0.0, 0.0
    assert ((got.double() - want).abs() <= tol).all()
    off = torch.full_like(lse, -float("inf"))
    K[:, :, inf_at, 3] = -float("inf")
    assert (pbs.pbs_key_mass(Q, K, off, window=window, n_sink=n_sink) == 0).all()
    pbs.pbs_check_device()
