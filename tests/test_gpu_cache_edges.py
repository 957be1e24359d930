"""Cache operators on the GPU at edges of their kernels and at their limits."""
import pytest
import torch

import cache_util as cu
import permuted_block_sparse_b200 as pbs
from test_gpu_cache import inputs, lens

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


# B, Hq, Hkv, d, M, N, P: few rows (8, 16 and 32 a KV head) and tiles, with and without a prefix
VALUE_FORMS = [(2, 4, 2, 128, 1, 900, 0), (2, 8, 2, 64, 2, 900, 0), (1, 16, 1, 128, 1, 5000, 0), (1, 16, 1, 64, 2, 900, 0),
               (2, 8, 2, 128, 150, 900, 0), (2, 4, 2, 128, 1, 700, 600), (9, 8, 2, 64, 1, 700, 600)]


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("case", VALUE_FORMS, ids=str)
def test_infinite_values_that_every_row_sees(case, bad):
    """In the middle of the cache, where groups and tiles are wholly visible: with
    weights of every rounding, the one that is exactly 1 among them."""
    B, Hq, Hkv, d, M, N, P = case
    Q, K, V = inputs(700 + N + M, B, Hq, Hkv, d, M, N)
    Kp, Vp = (inputs(800 + P, 1, Hkv, Hkv, d, P, P)[1:] if P else (None, None))
    run = (lambda K, V, Vp: pbs.pbs_attn_prefix(Q, Kp, Vp, K, V)) if P else (lambda K, V, Vp: pbs.pbs_attn_window(Q, K, V))
    K[:, :, 400] = 3 * Q[:, ::Hq // Hkv, 0].sign()          # the largest logit of the groups' first heads
    want, want_lse = run(K, V, Vp)
    V2, Vp2 = V.clone(), None if Vp is None else Vp.clone()
    at = [200 + 7 * c for c in range(d // 2)]               # column 2 c holds one at key 200 + 7 c
    for c, j in enumerate(at):
        V2[:, :, 400 if c == 3 else j, 2 * c] = bad
    if P:
        Vp2[:, :, 111, 1] = bad
    O, lse = run(K, V2, Vp2)
    pbs.pbs_check_device()
    hit = torch.zeros(d, dtype=torch.bool, device="cuda")
    hit[::2], hit[1] = True, bool(P)
    assert torch.equal(lse, want_lse) and torch.equal(O[..., ~hit], want[..., ~hit])
    got = O[..., hit].float()
    assert torch.isnan(got).all() if bad != bad else (got == bad).all()


def test_infinite_values_of_both_signs():
    Q, K, V = inputs(900, 1, 4, 2, 128, 1, 900)
    V[:, :, 300, 5], V[:, :, 500, 5], V[:, :, 300, 6] = float("inf"), -float("inf"), float("inf")
    O, _ = pbs.pbs_attn_window(Q, K, V)
    assert torch.isnan(O[..., 5]).all() and (O[..., 6] == float("inf")).all()
    assert torch.isfinite(O[..., :5]).all() and torch.isfinite(O[..., 7:]).all()


@pytest.mark.parametrize("B,Hkv,N,budget", [(3, 4, 900, 300), (1, 2, 70000, 5000), (2, 1, 140000, 3000), (5, 8, 64, 64)])
def test_evict_with_lengths_in_place(B, Hkv, N, budget):
    """One tensor of lengths goes in and comes out, with one CTA a row and with clusters."""
    mass = torch.rand((B, Hkv, N), generator=torch.Generator(device="cuda").manual_seed(N), device="cuda")
    K, V = inputs(11, B, 1, 1, 64, 1, N)[1:]
    K, V = K.expand(B, Hkv, N, 64), V.expand(B, Hkv, N, 64)
    start = torch.tensor([N - 7 * b if b != 1 else budget - 1 for b in range(B)], dtype=torch.int32, device="cuda")
    want = pbs.pbs_evict(mass, K, V, budget, 20, 4, kv_len=start)
    for _ in range(4):
        n = start.clone()
        got = pbs.pbs_evict(mass, K, V, budget, 20, 4, kv_len=n, new_len=n)
        assert got[4] is n and n.tolist() == [min(int(x), budget) for x in start]
        assert torch.equal(got[0], want[0])
        for b in range(B):
            m = int(n[b])
            assert all(torch.equal(x[b, :, :m], y[b, :, :m]) for x, y in zip(got[1:4], want[1:4]))
    pbs.pbs_check_device()


def test_evict_with_one_output_given():
    """The other one gets its room."""
    _, K, V = inputs(21, 2, 2, 2, 64, 1, 300)
    mass = torch.rand((2, 2, 300), device="cuda")
    want = pbs.pbs_evict(mass, K, V, 50)
    for name in ("K_out", "V_out"):
        room = torch.zeros((2, 2, 90, 64), dtype=torch.bfloat16, device="cuda")
        _, Ko, Vo, _, _ = pbs.pbs_evict(mass, K, V, 50, **{name: room})
        assert Ko.shape == Vo.shape == room.shape
        assert torch.equal(Ko[:, :, :50], want[1]) and torch.equal(Vo[:, :, :50], want[2])


@pytest.mark.parametrize("M", [1, 3])
def test_mass_of_a_shared_prefix(M):
    """Each row as a sequence of its own over the broadcast prefix, and the own keys as
    they lie: what all rows give in all is one per row and head.  A logit of 64 products
    is off by 64 2^-24 of its absolute sum, which is below 8 here, and the LSE by as
    much: 2^-14 of a weight in all."""
    B, Hq, Hkv, d, P, N = 3, 8, 2, 64, 300, 90
    Q, K, V = inputs(31, B, Hq, Hkv, d, M, N)
    _, Kp, Vp = inputs(41, 1, Hkv, Hkv, d, 1, P)
    kv = lens([90, 3, 40])
    _, lse = pbs.pbs_attn_prefix(Q, Kp, Vp, K, V, kv_len=kv)
    rows, rows_lse = Q.transpose(1, 2).reshape(B * M, Hq, 1, d), lse.transpose(1, 2).reshape(B * M, Hq, 1)
    shared = pbs.pbs_key_mass(rows, Kp.expand(B * M, -1, -1, -1), rows_lse)
    own = pbs.pbs_key_mass(Q, K, lse, kv_len=kv)
    pbs.pbs_check_device()
    want = torch.exp(rows.double() @ Kp.double().repeat_interleave(Hq // Hkv, 1).transpose(2, 3) * d ** -0.5
                     - rows_lse.double()[..., None])
    want = want.reshape(B * M, Hkv, Hq // Hkv, P).sum(2)
    assert (shared.double() - want).abs().max() <= 2.0 ** -14 * float(want.max())
    total = shared.reshape(B, M, -1).sum((1, 2)) + own.sum((1, 2))
    assert (total - M * Hq).abs().max() <= 2.0 ** -12 * M * Hq
