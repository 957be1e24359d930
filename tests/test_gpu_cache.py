"""The cache operators on the GPU against fp64 references: windowed attention
with sinks, shared-prefix attention, key mass and eviction, alone and as a
decode loop uses them."""
import math

import numpy as np
import pytest
import torch

import cache_util as cu
import oracle
import permuted_block_sparse_b200 as pbs

pytestmark = pytest.mark.gpu
INF, NAN = math.inf, math.nan


def rand(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def lens(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def inputs(seed, B, Hq, Hkv, d, M, N, scale=1.0):
    return (rand(seed, B, Hq, M, d, scale=scale), rand(seed + 1, B, Hkv, N, d, scale=scale),
            rand(seed + 2, B, Hkv, N, d))


def check_window(Q, K, V, window=0, n_sink=0, kv=None, ql=None, what="", **kw):
    kv, ql = lens(kv), lens(ql)
    O, lse = pbs.pbs_attn_window(Q, K, V, window, n_sink, kv_len=kv, q_len=ql, **kw)
    pbs.pbs_check_device()
    ref = cu.reference(Q, K, V, window, n_sink, kv, ql, kw.get("softmax_scale"))
    _, rows = cu.visible(Q.shape[0], Q.shape[2], K.shape[2], window, n_sink, kv, ql, Q.device)
    cu.assert_attention(O, lse, ref, rows, what)
    return O, lse


# ---------------------------------------------------------------- attention
# B, Hq, Hkv, d, M, N, window, n_sink, kv_len, q_len
WINDOW_CASES = [
    (1, 1, 1, 64, 1, 1, 0, 0, None, None),
    (1, 1, 1, 128, 1, 1, 1, 1, None, None),
    (1, 8, 8, 128, 1, 15, 7, 2, None, None),              # one head per KV head
    (2, 8, 2, 128, 1, 1000, 0, 0, [1000, 1], None),
    (3, 32, 8, 128, 1, 2049, 300, 4, [0, 2049, 301], None),
    (2, 8, 1, 64, 1, 777, 100, 130, [777, 140], None),    # more sinks than window
    (1, 10, 2, 64, 3, 513, 64, 16, None, None),           # 15 rows per KV head
    (1, 16, 1, 128, 1, 4100, 4096, 17, None, None),
    (2, 6, 2, 64, 5, 333, 50, 5, [333, 3], None),         # rows before the first key
    (1, 9, 1, 128, 2, 700, 0, 0, None, None),             # 18 rows per KV head
    (1, 64, 1, 128, 2, 400, 129, 1, None, None),
    (1, 4, 1, 128, 33, 33, 0, 0, None, None),             # prompts
    (1, 4, 2, 64, 129, 129, 1, 0, None, None),            # each row sees itself alone
    (1, 4, 1, 128, 300, 300, 128, 128, None, None),
    (2, 6, 2, 128, 257, 400, 100, 3, [400, 257], None),
    (2, 7, 1, 64, 140, 300, 63, 70, [300, 20], None),     # a cache shorter than the chunk
    (3, 4, 2, 128, 200, 200, 64, 4, [200, 77, 0], [200, 77, 0]),   # padded prompts
    (1, 5, 1, 128, 1000, 1500, 517, 33, None, None),
    (1, 64, 1, 64, 20, 260, 31, 2, None, None),
    (1, 1, 1, 128, 520, 520, 200, 9, None, None),
    (1, 1, 1, 64, 700, 2000, 0, 0, [1999], None),
    (2, 16, 2, 128, 64, 3001, 700, 40, [3001, 1203], [64, 61]),
    (1, 32, 1, 128, 1, 5000, 0, 0, None, None),           # 32 rows per KV head
    (2, 12, 2, 64, 5, 900, 333, 9, [900, 11], [5, 3]),    # 30
    (1, 33, 1, 64, 1, 1, 0, 0, None, None),               # 33 rows, one key
    (1, 3, 1, 128, 64, 1, 5, 1, None, None),              # a chunk over one key
    (300, 2, 2, 64, 1, 70, 20, 2, None, None),            # more sequences than places on the chip
]


@pytest.mark.parametrize("case", WINDOW_CASES, ids=str)
def test_window(case):
    B, Hq, Hkv, d, M, N, window, n_sink, kv, ql = case
    check_window(*inputs(M + N, B, Hq, Hkv, d, M, N), window, n_sink, kv, ql)


# B, Hq, Hkv, d, M, P, N, kv_len, q_len
PREFIX_CASES = [
    (1, 1, 1, 64, 1, 1, 1, None, None),
    (1, 4, 1, 128, 1, 17, 5, [0], None),                  # the prefix alone
    (4, 32, 8, 128, 1, 2048, 100, [1, 100, 63, 64], None),
    (3, 10, 2, 64, 5, 1007, 333, [5, 333, 2], None),
    (33, 4, 1, 128, 1, 700, 40, None, None),              # more rows than one tile holds
    (70, 4, 1, 64, 1, 300, 33, None, None),
    (17, 20, 4, 128, 3, 515, 65, None, None),
    (2, 8, 1, 128, 40, 260, 90, [90, 40], None),          # 320 rows per KV head
    (2, 3, 1, 64, 100, 129, 100, [100, 30], [100, 30]),
    (5, 64, 1, 128, 2, 1000, 300, None, None),
    (2, 4, 4, 128, 1, 5000, 2000, [2000, 0], None),
    (3, 8, 2, 128, 1, 300, 50, [50, 0, 7], [1, 0, 1]),
    (3, 12, 2, 64, 5, 300, 50, [50, 4, 7], [5, 0, 2]),
    (40, 8, 1, 128, 1, 40, 1, None, None),
    (2, 33, 1, 128, 1, 1, 3, None, None),
    (1, 2, 2, 64, 70, 1, 70, [3], None),
]


@pytest.mark.parametrize("case", PREFIX_CASES, ids=str)
def test_prefix(case):
    B, Hq, Hkv, d, M, P, N, kv, ql = case
    Q, K, V = inputs(P + N, B, Hq, Hkv, d, M, N)
    Kp, Vp = rand(1, 1, Hkv, P, d), rand(2, 1, Hkv, P, d)
    kv, ql = lens(kv), lens(ql)
    O, lse = pbs.pbs_attn_prefix(Q, Kp, Vp, K, V, kv_len=kv, q_len=ql)
    pbs.pbs_check_device()
    ref = cu.reference(Q, K, V, kv_len=kv, q_len=ql, Kp=Kp, Vp=Vp)
    _, rows = cu.visible(B, M, N, 0, 0, kv, ql, Q.device)
    cu.assert_attention(O, lse, ref, rows)


SMALL_AND_LARGE = [(2, 8, 2, 128, 1, 900, 200, 5), (2, 8, 2, 64, 2, 900, 200, 5), (2, 9, 1, 128, 5, 900, 0, 0),
                   (2, 8, 2, 128, 150, 900, 200, 5)]     # every kernel: few rows, some, a chunk


@pytest.mark.parametrize("case", SMALL_AND_LARGE, ids=str)
def test_strides_and_broadcast_views(case):
    """Token-major queries and outputs, caches inside larger buffers, keys and
    values shared by all sequences or heads."""
    B, Hq, Hkv, d, M, N, window, n_sink = case
    Q, K, V = inputs(7, B, Hq, Hkv, d, M, N)
    want, want_lse = check_window(Q, K, V, window, n_sink)
    Qt = Q.transpose(1, 2).contiguous().transpose(1, 2)
    both = torch.stack([K, V], 3).reshape(B, Hkv, N, 2 * d)          # keys and values interleaved
    out = torch.full((B, M, Hq, d + 8), 5.0, dtype=torch.bfloat16, device="cuda")
    O, lse = pbs.pbs_attn_window(Qt, both[..., :d], both[..., d:], window, n_sink,
                                 out=out[..., :d].transpose(1, 2))
    assert torch.equal(O, want) and torch.equal(lse, want_lse)
    assert (out[..., d:] == 5.0).all()
    one = K[:1, :1].expand(B, Hkv, N, d), V[:1, :1].expand(B, Hkv, N, d)
    O, lse = pbs.pbs_attn_window(Q, *one, window, n_sink)
    full, full_lse = pbs.pbs_attn_window(Q, one[0].contiguous(), one[1].contiguous(), window, n_sink)
    assert torch.equal(O, full) and torch.equal(lse, full_lse)
    m = pbs.pbs_key_mass(Q, one[0], lse, window=window, n_sink=n_sink)
    assert torch.equal(m, pbs.pbs_key_mass(Q, one[0].contiguous(), lse, window=window, n_sink=n_sink))
    pbs.pbs_check_device()


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("case", SMALL_AND_LARGE, ids=str)
def test_unseen_keys_and_values_do_not_matter(case, bad):
    """NaN and infinities in every slot behind the sequence and in keys that
    some rows see and others do not change only the rows that see them."""
    B, Hq, Hkv, d, M, N, window, n_sink = case
    Q, K, V = inputs(11, B, Hq, Hkv, d, M, N)
    kv = lens([N - 100, N - 333])
    clean, clean_lse = pbs.pbs_attn_window(Q, K, V, window, n_sink, kv_len=kv)
    mass = pbs.pbs_key_mass(Q, K, clean_lse, window=window, n_sink=n_sink, kv_len=kv)
    see, _ = cu.visible(B, M, N, window, n_sink, kv, None, Q.device)
    K2, V2 = K.clone(), V.clone()
    hidden = ~see.any(1)[:, None, :, None].expand_as(K)
    K2[hidden], V2[hidden] = bad, bad
    O, lse = pbs.pbs_attn_window(Q, K2, V2, window, n_sink, kv_len=kv)
    assert torch.equal(O, clean) and torch.equal(lse, clean_lse)
    assert torch.equal(pbs.pbs_key_mass(Q, K2, lse, window=window, n_sink=n_sink, kv_len=kv), mass)
    some = [int(kv[0]) - 1, int(kv[0]) - M // 2 - 1, int(kv[0]) - window + 1]     # seen by some rows of sequence 0
    for col, j in zip((0, 3, d - 1), some):
        V2[0, :, j, col] = bad
    O, lse = pbs.pbs_attn_window(Q, K2, V2, window, n_sink, kv_len=kv)
    assert torch.equal(lse, clean_lse)
    hit = torch.zeros_like(O, dtype=torch.bool)
    for col, j in zip((0, 3, d - 1), some):
        hit[0, :, :, col] |= see[0, :, j]
    fine = torch.isfinite(O)
    assert (fine == ~hit).all()
    ref = cu.reference(Q, K, V, window, n_sink, kv)
    # the values beside the bad ones keep the bound (zeroing the bad ones would too)
    err = (O.double() - ref[0]).abs()
    assert (err <= 2 * cu.HALF * (ref[0].abs() + ref[2]) + 2.0 ** -12)[fine].all()
    if not math.isnan(bad):
        assert (O[hit] == bad).all()
    pbs.pbs_check_device()


@pytest.mark.parametrize("case", SMALL_AND_LARGE, ids=str)
def test_rows_past_q_len_stay_as_they_were(case):
    B, Hq, Hkv, d, M, N, window, n_sink = case
    M += 3
    Q, K, V = inputs(13, B, Hq, Hkv, d, M, N)
    ql = [M - 3, 0]
    Q[0, :, M - 3:] = NAN
    out = torch.full_like(Q, 3.0)
    lse = torch.full((B, Hq, M), 7.0, device="cuda")
    check_window(Q, K, V, window, n_sink, [N, N - 9], ql, out=out, lse=lse)
    assert (out[0, :, M - 3:] == 3.0).all() and (out[1] == 3.0).all()
    assert (lse[0, :, M - 3:] == 7.0).all() and (lse[1] == 7.0).all()
    before = out.clone()
    O, none = pbs.pbs_attn_window(Q, K, V, window, n_sink, kv_len=lens([N, N - 9]), q_len=lens(ql), out=out,
                                  want_lse=False)
    assert none is None and torch.equal(O, before)


@pytest.mark.parametrize("case", SMALL_AND_LARGE, ids=str)
def test_rows_that_see_nothing(case):
    """A cache shorter than the chunk: the rows before its first key give 0 and -inf, and add no mass."""
    B, Hq, Hkv, d, M, N, window, n_sink = case
    Q, K, V = inputs(17, B, Hq, Hkv, d, M, N)
    for kv in ([0, M - 1], [M // 2, 1]):
        O, lse = check_window(Q, K, V, window, n_sink, kv)
        for b in range(B):
            empty = max(0, M - kv[b])
            assert (O[b, :, :empty] == 0).all() and (lse[b, :, :empty] == -INF).all()
        m = pbs.pbs_key_mass(Q, K, lse, window=window, n_sink=n_sink, kv_len=lens(kv))
        assert float(m.sum()) == pytest.approx(Hq * sum(min(M, x) for x in kv), rel=1e-4)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hkv,G,M,N,kv,ql", [(1, 64, 4, 40, 2, 4), (2, 7, 369, 149, 44, 251), (1, 7, 369, 149, 103, 245),
                                             (1, 1, 256, 60, 50, 256)])
def test_tiles_without_a_visible_key_beside_others(Hkv, G, M, N, kv, ql, d):
    """Of the two row tiles that run together the first may see no key at all; its
    rows are zeros and the second's are right, every time."""
    for seed in range(12):
        Q, K, V = inputs(60 + seed, 1, Hkv * G, Hkv, d, M, N)
        out = torch.full_like(Q, 3.0)
        check_window(Q, K, V, 0, 0, [kv], [ql], out=out, what=f"seed {seed}")
        assert (out[0, :, :ql - kv] == 0).all() and (out[0, :, ql:] == 3.0).all()


@pytest.mark.parametrize("case", SMALL_AND_LARGE, ids=str)
def test_large_logits_and_scale(case):
    B, Hq, Hkv, d, M, N, window, n_sink = case
    Q, K, V = inputs(19, B, Hq, Hkv, d, M, N, scale=8.0)
    check_window(Q, K, V, window, n_sink)
    check_window(Q, K, V, window, n_sink, softmax_scale=1.0)
    check_window(Q, K, V, window, n_sink, softmax_scale=1e-4)
    low = K.clone()
    low[:, :, ::2] = torch.finfo(torch.bfloat16).min / 2 ** 100       # far below every other logit
    check_window(Q.abs(), low, V, window, n_sink)


@pytest.mark.parametrize("case", SMALL_AND_LARGE, ids=str)
def test_bad_lengths_are_reported(case):
    B, Hq, Hkv, d, M, N, window, n_sink = case
    Q, K, V = inputs(23, B, Hq, Hkv, d, M, N)
    for kv, ql, kv2, ql2 in (([N + 5, 40], None, [N, 40], None), ([40, -3], None, [40, 0], None),
                             ([N, N], [M + 1, -1], [N, N], [M, 0])):
        a = [torch.zeros_like(Q), torch.zeros((B, Hq, M), device="cuda")]
        b = [x.clone() for x in a]
        pbs.pbs_attn_window(Q, K, V, window, n_sink, kv_len=lens(kv), q_len=lens(ql), out=a[0], lse=a[1])
        with pytest.raises(pbs.PbsError) as e:
            pbs.pbs_check_device()
        assert e.value.code == -6
        pbs.pbs_attn_window(Q, K, V, window, n_sink, kv_len=lens(kv2), q_len=lens(ql2), out=b[0], lse=b[1])
        pbs.pbs_check_device()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    pbs.pbs_key_mass(Q, K, b[1], kv_len=lens([N + 1, 5]))
    with pytest.raises(pbs.PbsError):
        pbs.pbs_check_device()
    pbs.pbs_evict(torch.rand(B, Hkv, N, device="cuda"), K, V, 64, kv_len=lens([N, -1]))
    with pytest.raises(pbs.PbsError):
        pbs.pbs_check_device()


@pytest.mark.parametrize("M", [1, 40])
def test_offsets_past_32_bits(M):
    """A cache of 2.6 G elements per tensor, of which the window and the sinks are read."""
    Hkv, N, d, window, n_sink = 4, 5_000_000, 128, 300, 5
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB")
    K, V = (torch.empty((1, Hkv, N, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    n = window + M
    for t, s in ((K, 1), (V, 2)):
        t[:, :, :n_sink], t[:, :, N - n:] = rand(s, 1, Hkv, n_sink, d), rand(s + 9, 1, Hkv, n, d)
    Q = rand(5, 1, 16, M, d)
    O, lse = pbs.pbs_attn_window(Q, K, V, window, n_sink)
    pbs.pbs_check_device()
    near = [torch.cat([t[:, :, :n_sink], t[:, :, N - n:]], 2) for t in (K, V)]
    ref = cu.reference(Q, *near, window, n_sink)
    cu.assert_attention(O, lse, ref, torch.ones(1, M, dtype=torch.bool, device="cuda"))
    mass = pbs.pbs_key_mass(Q, K, lse, window=window, n_sink=n_sink)
    want, tol = cu.reference_mass(Q, near[0], lse, window=window, n_sink=n_sink)
    got = torch.cat([mass[:, :, :n_sink], mass[:, :, N - n:]], 2)
    assert ((got.double() - want).abs() <= tol).all()
    assert (mass[:, :, n_sink:N - n] == 0).all()
    score = torch.zeros((1, Hkv, N), device="cuda")
    score[:, :, N - n] = 1.0
    keep, Ko, Vo, _, _ = pbs.pbs_evict(score, K, V, n_sink + window + 1, recent=window, n_sink=n_sink)
    at = torch.tensor([*range(n_sink), N - n, *range(N - window, N)], dtype=torch.int32, device="cuda")
    assert (keep == at).all()
    assert torch.equal(Ko, K[:, :, at.long()]) and torch.equal(Vo, V[:, :, at.long()])


# --------------------------------------------------------------------- mass
MASS_CASES = [
    (1, 1, 1, 64, 1, 1, 0, 0, None, None),
    (2, 8, 2, 128, 1, 1000, 0, 0, [1000, 3], None),
    (3, 32, 8, 128, 1, 700, 100, 4, [0, 700, 301], None),
    (1, 10, 2, 64, 3, 513, 64, 16, None, None),
    (1, 9, 1, 128, 2, 700, 0, 0, None, None),
    (1, 64, 1, 128, 1, 300, 0, 0, None, None),
    (1, 4, 1, 128, 300, 300, 0, 0, None, None),
    (2, 6, 2, 64, 257, 400, 100, 3, [400, 257], None),
    (3, 4, 2, 128, 200, 200, 64, 4, [200, 77, 0], [200, 77, 0]),
    (2, 7, 1, 64, 140, 300, 63, 140, [300, 20], None),
    (1, 5, 1, 128, 61, 2001, 900, 7, None, None),
    (1, 64, 2, 64, 40, 260, 0, 0, None, None),
    (1, 1, 1, 128, 700, 1300, 500, 0, None, None),
    (2, 4, 1, 128, 64, 1111, 100, 30, [1111, 70], [64, 9]),          # one or two boxes of rows
    (1, 4, 2, 64, 33, 4000, 0, 0, None, None),
    (3, 5, 1, 128, 25, 700, 300, 140, [700, 0, 25], [25, 25, 0]),
    (1, 3, 1, 64, 90, 50, 0, 0, None, None),                         # more rows than keys
    (1, 8, 1, 128, 600, 5000, 0, 0, None, None),                     # parts of the rows
    (300, 2, 2, 64, 1, 70, 20, 2, None, None),
    (4, 2, 2, 64, 1, 4099, 17, 33, [4099, 66, 34, 1], None),         # sinks, a gap, the window, the unfilled end
    (5, 4, 1, 128, 2, 2000, 1, 0, [2000, 17, 16, 15, 0], [2, 1, 2, 0, 2]),
    (3, 3, 3, 64, 9, 700, 5, 16, [700, 40, 9], [9, 3, 9]),
    (2, 2, 1, 128, 1, 65, 1, 65, [65, 64], None),
    (40, 8, 4, 64, 200, 300, 0, 0, None, None),                      # several launches, each adding to the last
    (75, 8, 2, 128, 150, 200, 70, 9, [200, 0, 150, 31, 199] * 15, [150, 0, 64, 65, 128] * 15),
    (1, 8, 4, 128, 512, 9500, 3000, 5, None, None),
    (38, 5, 1, 64, 151, 1100, 0, 0, None, [151, 50, 51, 100, 1, 150, 0] * 5 + [2, 3, 101]),
    (37, 10, 2, 128, 60, 500, 0, 0, None, None),                     # ... and the most tiles of one launch
]


@pytest.mark.parametrize("decay", [None, 0.0, 0.75])
@pytest.mark.parametrize("case", MASS_CASES, ids=str)
def test_key_mass(case, decay):
    B, Hq, Hkv, d, M, N, window, n_sink, kv, ql = case
    Q, K, V = inputs(3 * M + N, B, Hq, Hkv, d, M, N)
    kv, ql = lens(kv), lens(ql)
    _, lse, _, _ = cu.reference(Q, K, V, window, n_sink, kv, ql)
    lse = lse.float()
    _, rows = cu.visible(B, M, N, window, n_sink, kv, ql, Q.device)
    lse[~rows[:, None].expand_as(lse)] = NAN                 # rows that are not queries are not read
    prev = None if decay is None else torch.rand((B, Hkv, N), device="cuda")
    got = pbs.pbs_key_mass(Q, K, lse, prev, 1.0 if decay is None else decay, window, n_sink, kv_len=kv, q_len=ql)
    pbs.pbs_check_device()
    want, tol = cu.reference_mass(Q, K, lse, prev, 1.0 if decay is None else decay, window, n_sink, kv, ql)
    assert ((got.double() - want).abs() <= tol).all(), float(((got.double() - want).abs() - tol).max())
    if decay is not None:                                    # in place, in rows of a larger buffer
        room = torch.full((B, Hkv, N + 5), -1.0, device="cuda")
        room[..., :N] = prev
        out = pbs.pbs_key_mass(Q, K, lse, room[..., :N], decay, window, n_sink, kv_len=kv, q_len=ql,
                               out=room[..., :N])
        assert torch.equal(out, got) and (room[..., N:] == -1.0).all()


@pytest.mark.parametrize("M", [1, 40, 300])
def test_key_mass_without_earlier_mass_ignores_decay(M):
    Q, K, V = inputs(8, 2, 4, 2, 64, M, 400)
    _, lse = pbs.pbs_attn_window(Q, K, V)
    want = pbs.pbs_key_mass(Q, K, lse)
    for decay in (0.5, NAN, INF, -1.0):
        assert torch.equal(pbs.pbs_key_mass(Q, K, lse, None, decay), want), decay


def test_key_mass_repeats_bit_for_bit():
    Q, K, _ = inputs(5, 2, 8, 2, 128, 500, 3000)
    lse = torch.full((2, 8, 500), 9.0, device="cuda")
    a = [pbs.pbs_key_mass(Q, K, lse) for _ in range(3)]
    assert torch.equal(a[0], a[1]) and torch.equal(a[0], a[2])


# ------------------------------------------------------------------ evict
def check_evict(mass, K, V, budget, recent, n_sink, kv):
    B, Hkv, N, d = K.shape
    keep, Ko, Vo, mo, n = pbs.pbs_evict(mass, K, V, budget, recent, n_sink, kv_len=lens(kv))
    pbs.pbs_check_device()
    want = oracle.evict(mass.cpu().numpy(), budget, recent, n_sink, kv)
    assert np.array_equal(keep.cpu().numpy(), want)
    assert n.tolist() == [min(budget, N if kv is None else kv[b]) for b in range(B)]
    for b in range(B):
        m = int(n[b])
        at = keep[b, :, :m].long()
        rows = at[..., None].expand(-1, -1, d)
        assert torch.equal(Ko[b, :, :m], torch.gather(K[b], 1, rows))
        assert torch.equal(Vo[b, :, :m], torch.gather(V[b], 1, rows))
        assert torch.equal(mo[b, :, :m].view(torch.int32), torch.gather(mass[b], 1, at).view(torch.int32))


@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "zeros", "special", "negative"])
@pytest.mark.parametrize("B,Hkv,d,N,budget,recent,n_sink,kv", [
    (1, 1, 64, 1, 1, 0, 0, None), (1, 1, 128, 1, 1, 1, 0, [0]), (2, 2, 64, 33, 32, 7, 3, [33, 20]),
    (1, 8, 128, 4096, 2048, 512, 4, None), (3, 1, 64, 1025, 100, 0, 0, [1025, 100, 101]),
    (2, 3, 128, 5003, 777, 300, 130, [5003, 900]), (1, 2, 64, 3000, 3000, 1000, 2000, None),
    (1, 1, 64, 70001, 33001, 5, 7, [70000]), (1, 1, 128, 300, 10, 5, 5, None),
])
def test_evict(B, Hkv, d, N, budget, recent, n_sink, kv, kind):
    g = torch.Generator(device="cuda").manual_seed(N)
    mass = torch.exp(3 * torch.randn((B, Hkv, N), generator=g, device="cuda"))
    if kind == "ties":
        mass = torch.randint(0, 4, (B, Hkv, N), generator=g, device="cuda").float()
    elif kind in ("equal", "zeros"):
        mass.fill_(0.25 if kind == "equal" else 0.0)
    elif kind == "special":
        pick = torch.randint(0, 6, (B, Hkv, N), generator=g, device="cuda")
        for i, x in enumerate((NAN, INF, -INF, -0.0, 0.0)):
            mass[pick == i] = x
    elif kind == "negative":
        mass = -mass
    _, K, V = inputs(N, B, Hkv, Hkv, d, 1, N)
    check_evict(mass, K, V, budget, recent, n_sink, kv)


@pytest.mark.parametrize("levels", [1 << 30, 50])
@pytest.mark.parametrize("B,Hkv,N,budget", [(40, 2, 41003, 9000), (3, 25, 20000, 700), (1, 1, 400000, 100001),
                                            (1, 3, 131072, 4096)])
def test_evict_long_caches(B, Hkv, N, budget, levels):
    """Rows held in shared memory by one CTA or a cluster, and rows too long for it."""
    g = torch.Generator(device="cuda").manual_seed(N)
    mass = torch.randint(0, levels, (B, Hkv, N), generator=g, device="cuda").float()
    K = torch.zeros((B, 1, N, 64), dtype=torch.bfloat16, device="cuda").expand(B, Hkv, N, 64)
    keep, *_ = pbs.pbs_evict(mass, K, K, budget, 100, 4)
    pbs.pbs_check_device()
    x = mass.cpu().numpy()
    always = np.zeros(N, bool)
    always[:4] = always[N - 100:] = True
    for b in range(B):
        for h in range(Hkv):
            order = np.lexsort((np.arange(N), -x[b, h].astype(np.float64), ~always))
            assert np.array_equal(keep[b, h].cpu().numpy(), np.sort(order[:budget])), (b, h)


def test_evict_into_larger_buffers():
    """Kept rows at the start of caches with room to grow; everything behind them stays."""
    B, Hkv, d, N, budget = 2, 2, 64, 500, 120
    _, K, V = inputs(1, B, Hkv, Hkv, d, 1, N)
    both = torch.stack([K, V], 3).reshape(B, Hkv, N, 2 * d)
    mass = torch.rand((B, Hkv, N + 3), device="cuda")[..., :N]
    kv = lens([500, 90])
    keep, Ko, Vo, mo, _ = pbs.pbs_evict(mass, K, V, budget, 10, 4, kv_len=kv)
    K2, V2 = (torch.full((B, N, Hkv, d), 9.0, dtype=torch.bfloat16, device="cuda").transpose(1, 2) for _ in range(2))
    m2 = torch.full((B, Hkv, 300), 9.0, device="cuda")
    keep2, *_ = pbs.pbs_evict(mass, both[..., :d], both[..., d:], budget, 10, 4, kv_len=kv, K_out=K2, V_out=V2,
                              mass_out=m2)
    assert torch.equal(keep2, keep)
    for b, n in enumerate((120, 90)):
        assert torch.equal(K2[b, :, :n], Ko[b, :, :n]) and torch.equal(V2[b, :, :n], Vo[b, :, :n])
        assert torch.equal(m2[b, :, :n], mo[b, :, :n])
        assert (K2[b, :, n:] == 9).all() and (V2[b, :, n:] == 9).all() and (m2[b, :, n:] == 9).all()


def test_views_of_one_buffer():
    """Inputs and outputs that lie between one another in a buffer, sharing no
    element, are taken: K beside V per sequence, heads or elements in turn, and
    the short cache behind the long one."""
    B, Hkv, d, N, budget = 3, 2, 64, 300, 70
    Q, K, V = inputs(5, B, 4, Hkv, d, 1, N)
    mass = torch.rand((B, Hkv, N), device="cuda")
    want = pbs.pbs_evict(mass, K, V, budget, 10, 4)
    room = torch.zeros((B, 2, Hkv, N + budget, d), dtype=torch.bfloat16, device="cuda")     # K beside V
    turns = torch.zeros((B, N + budget, Hkv, 2, d), dtype=torch.bfloat16, device="cuda").permute(0, 3, 2, 1, 4)
    side = torch.zeros((B, Hkv, N + budget, 2, d), dtype=torch.bfloat16, device="cuda").permute(0, 3, 1, 2, 4)
    for buf in (room, turns, side):
        m = torch.zeros((B, Hkv, N + budget), device="cuda")
        buf[:, 0, :, :N], buf[:, 1, :, :N], m[..., :N] = K, V, mass
        got = pbs.pbs_evict(m[..., :N], buf[:, 0, :, :N], buf[:, 1, :, :N], budget, 10, 4, K_out=buf[:, 0, :, N:],
                            V_out=buf[:, 1, :, N:], mass_out=m[..., N:])
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        assert torch.equal(buf[:, 0, :, :N], K) and torch.equal(buf[:, 1, :, :N], V)
    _, lse = pbs.pbs_attn_window(Q, K, V)
    pair = torch.zeros((B, Hkv, 2, N), device="cuda")
    pair[:, :, 0] = mass
    pbs.pbs_key_mass(Q, K, lse, pair[:, :, 0], 0.5, out=pair[:, :, 1])
    assert torch.equal(pair[:, :, 1], pbs.pbs_key_mass(Q, K, lse, mass, 0.5)) and torch.equal(pair[:, :, 0], mass)


# ---------------------------------------------------- as a program uses them
def test_prefill_mass_evict_decode():
    """Prefill by the sparse attention, mass of every key from its LSE, a cache
    cut to a third, then decode steps over the short cache that keep adding mass
    -- against the oracle run step by step on the same numbers."""
    B, Hq, Hkv, N, d, budget, extra = 1, 8, 2, 512, 128, 170, 4
    Q, K, V = inputs(31, B, Hq, Hkv, d, N, N)
    perm = pbs.pbs_permute(Q, K, 128, 256)
    counts, idx = pbs.pbs_select(Q, K, perm, 128, 256, "topk", 1.0)
    O, lse = pbs.pbs_attn_fwd(Q, K, V, perm, counts, idx, 128, 256)
    O2, lse2 = check_window(Q, K, V)
    assert (lse - lse2).abs().max() < 1e-3
    mass = pbs.pbs_key_mass(Q, K, lse)
    assert float(mass.sum()) == pytest.approx(Hq * N, rel=1e-3)
    Kc, Vc = (torch.zeros((B, Hkv, budget + extra, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    mc = torch.zeros((B, Hkv, budget + extra), device="cuda")
    keep, _, _, _, n = pbs.pbs_evict(mass, K, V, budget, 32, 4, K_out=Kc, V_out=Vc, mass_out=mc)
    want = oracle.evict(mass.cpu().numpy(), budget, 32, 4)
    assert np.array_equal(keep.cpu().numpy(), want)
    for step in range(extra):
        q, k, v = inputs(100 + step, B, Hq, Hkv, d, 1, 1)
        at = int(n[0])
        Kc[:, :, at], Vc[:, :, at] = k[:, :, 0], v[:, :, 0]
        n += 1
        O, lse = pbs.pbs_attn_window(q, Kc, Vc, kv_len=n)
        ref = cu.reference(q, Kc, Vc, kv_len=n)
        cu.assert_attention(O, lse, ref, torch.ones(B, 1, dtype=torch.bool, device="cuda"))
        want, tol = cu.reference_mass(q, Kc, lse, mc, 0.9, kv_len=n)
        pbs.pbs_key_mass(q, Kc, lse, mc, 0.9, kv_len=n, out=mc)
        assert ((mc.double() - want).abs() <= tol).all()
    keep, Ko, *_ = pbs.pbs_evict(mc, Kc, Vc, budget, 32, 4, kv_len=n)
    assert np.array_equal(keep.cpu().numpy(), oracle.evict(mc.cpu().numpy(), budget, 32, 4, n.tolist()))
    pbs.pbs_check_device()


def test_prefix_equals_window_over_the_joined_cache():
    B, Hq, Hkv, d, P, N = 3, 8, 2, 128, 400, 70
    Q, K, V = inputs(41, B, Hq, Hkv, d, 2, N)
    Kp, Vp = rand(1, 1, Hkv, P, d), rand(2, 1, Hkv, P, d)
    O, lse = pbs.pbs_attn_prefix(Q, Kp, Vp, K, V)
    joined = [torch.cat([p.expand(B, -1, -1, -1), t], 2) for p, t in ((Kp, K), (Vp, V))]
    O2, lse2 = pbs.pbs_attn_window(Q, *joined)
    assert (lse - lse2).abs().max() < 2.0 ** -14
    assert (O.float() - O2.float()).abs().max() <= 4 * cu.HALF * float(V.float().abs().max())


@pytest.mark.parametrize("M", [1, 3, 9, 130])
def test_streams_and_graphs(M):
    """Two calls at once on two streams, and two captured graphs of one shape
    that replay one after the other with new inputs, give the bits of calls
    made alone."""
    B, Hq, Hkv, d, N, P = 2, 8, 2, 128, 1500, 600
    sets = [inputs(51 + 10 * i, B, Hq, Hkv, d, M, N) for i in range(2)]
    Kp, Vp = rand(1, 1, Hkv, P, d), rand(2, 1, Hkv, P, d)
    kv = lens([N, N - 700])

    def step(Q, K, V, stream=None):
        O, lse = pbs.pbs_attn_window(Q, K, V, 512, 4, kv_len=kv, stream=stream)
        O2, lse2 = pbs.pbs_attn_prefix(Q, Kp, Vp, K, V, kv_len=kv, stream=stream)
        mass = pbs.pbs_key_mass(Q, K, lse, window=512, n_sink=4, kv_len=kv, stream=stream)
        return (O, lse, O2, lse2, mass, *pbs.pbs_evict(mass, K, V, 256, 64, 4, kv_len=kv, stream=stream))

    alone = [step(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        got = [step(*x, stream=s) for x, s in zip(sets, streams)]
    torch.cuda.synchronize()
    for a, b in zip(alone, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    held = [tuple(t.clone() for t in s) for s in sets]
    graphs, outs = [], []
    for x in held:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(*x))
        graphs.append(g)
    for i in (0, 1):
        for x, s in zip(held, (sets[i], sets[1 - i])):
            for t, src in zip(x, s):
                t.copy_(src)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for o, want in zip(outs, (alone[i], alone[1 - i])):
            assert all(torch.equal(a, b) for a, b in zip(o, want))
    pbs.pbs_check_device()


@pytest.mark.parametrize("B,M,d,P,N,ql", [
    (12, 1, 128, 5000, 900, None), (40, 1, 64, 1500, 300, None), (70, 1, 128, 900, 130, None),   # tiles beside rows
    (17, 5, 64, 3001, 333, [5, 0, 3] * 5 + [1, 0]), (12, 1, 128, 700, 400, [0] * 12),             # (the last ends at once)
    (4, 20, 128, 3000, 800, None), (5, 33, 64, 1111, 257, [33, 1, 0, 20, 0]),                     # tiles beside tiles
])
@pytest.mark.parametrize("graph", [False, True])
def test_prefix_beside_own_keys(graph, B, M, d, P, N, ql):
    """The prefix's kernel and the sequences' own run side by side: calls whose
    inputs the stream rewrites right before and right after them, the lengths and
    the workspace included, give the bits of calls made alone."""
    Hq, Hkv = 8, 2
    sets = []
    for i in range(3):
        Q, K, V = inputs(300 + 10 * i, B, Hq, Hkv, d, M, N)
        kv = torch.randint(0, N + 1, (B,), generator=torch.Generator().manual_seed(i), dtype=torch.int32).cuda()
        sets.append((Q, rand(7 + i, 1, Hkv, P, d), rand(17 + i, 1, Hkv, P, d), K, V, kv))
    q_len = lens(ql)
    held = [t.clone() for t in sets[0]]
    outs = [(torch.full_like(held[0], 7.0), torch.full((B, Hq, M), 7.0, device="cuda")) for _ in range(12)]

    def step(x, out):
        pbs.pbs_attn_prefix(*x[:5], kv_len=x[5], q_len=q_len, out=out[0], lse=out[1])

    def run():
        for i, out in enumerate(outs):
            for t, x in zip(held, sets[i % 3]):
                t.copy_(x)
            step(held, out)

    alone = [(torch.full_like(o, 7.0), torch.full_like(l, 7.0)) for o, l in outs[:3]]
    for x, out in zip(sets, alone):
        step(x, out)
        torch.cuda.synchronize()
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        run = g.replay
    for _ in range(5):
        for o, l in outs:
            o.fill_(7.0), l.fill_(7.0)
        run()
        torch.cuda.synchronize()
        for i, (o, l) in enumerate(outs):
            assert torch.equal(o, alone[i % 3][0]) and torch.equal(l, alone[i % 3][1]), i
    pbs.pbs_check_device()
