"""Host-side checks of the cache operators: the fp64 oracle against torch and
brute force, and every refusal of the C ABI and the binding, before any GPU
call."""
import ctypes
import itertools
import math

import numpy as np
import pytest
import torch

import oracle
import permuted_block_sparse_b200 as pbs
from permuted_block_sparse_b200 import _binding as bd
import cache_util as cu


@pytest.fixture(scope="module")
def lib():
    from permuted_block_sparse_b200 import build
    build.build()
    return pbs.load()


# ------------------------------------------------------------------ oracle
@pytest.mark.parametrize("pos,window,n_sink", list(itertools.product((-2, 0, 3, 9), (0, 1, 4, 20), (0, 2, 12))))
def test_visible_keys_by_enumeration(pos, window, n_sink):
    want = [j for j in range(30) if j <= pos and (window == 0 or j > pos - window or j < n_sink)]
    assert list(oracle.visible_keys(pos, window, n_sink)) == want


@pytest.mark.parametrize("window,n_sink,kv,ql,prefix", [
    (0, 0, None, None, 0), (5, 0, None, None, 0), (5, 3, [11, 7], None, 0), (4, 2, [0, 9], [3, 6], 0),
    (0, 0, [13, 2], [6, 0], 7),
])
def test_attention_and_mass_oracle_against_masked_torch(window, n_sink, kv, ql, prefix):
    g = torch.Generator().manual_seed(3)
    B, Hq, Hkv, M, N, d = 2, 4, 2, 6, 13, 8
    Q, K, V = (torch.randn(B, h, n, d, generator=g, dtype=torch.float64) for h, n in ((Hq, M), (Hkv, N), (Hkv, N)))
    Kp, Vp = (torch.randn(1, Hkv, prefix, d, generator=g, dtype=torch.float64) if prefix else None for _ in range(2))
    kvt = None if kv is None else torch.tensor(kv, dtype=torch.int32)
    qlt = None if ql is None else torch.tensor(ql, dtype=torch.int32)
    args = [None if x is None else x.numpy() for x in (Kp, Vp)]
    O, lse = oracle.attn_cache(Q.numpy(), K.numpy(), V.numpy(), window, n_sink, kv, ql, Kp=args[0], Vp=args[1])
    Or, lr, _, _ = cu.reference(Q, K, V, window, n_sink, kvt, qlt, Kp=Kp, Vp=Vp)
    rows = ~np.isnan(lse)
    assert np.allclose(O[rows], Or.numpy()[rows], atol=1e-12)
    assert np.allclose(lse[rows], lr.numpy()[rows], atol=1e-12)
    if prefix:
        return
    prev = torch.rand(B, Hkv, N, generator=g)
    l32 = torch.from_numpy(np.where(rows, lse, 0.0)).float()
    got = oracle.key_mass(Q.numpy(), K.numpy(), l32.numpy(), prev.numpy(), 0.5, window, n_sink, kv, ql)
    want, _ = cu.reference_mass(Q, K, l32, prev, 0.5, window, n_sink, kvt, qlt)
    assert np.allclose(got, want.numpy(), atol=1e-12)
    # without decayed mass, the weights of each computed row that sees a key add to one
    total = oracle.key_mass(Q.numpy(), K.numpy(), lse, None, 1.0, window, n_sink, kv, ql).sum()
    assert total == pytest.approx(np.isfinite(lse[rows]).sum(), abs=1e-9)


def test_evict_oracle_by_brute_force():
    rng = np.random.default_rng(5)
    for trial in range(40):
        N, L = 9, int(rng.integers(0, 10))
        budget = int(rng.integers(1, N + 1))
        n_sink = int(rng.integers(0, budget + 1))
        recent = int(rng.integers(0, budget - n_sink + 1))
        mass = rng.integers(-2, 3, (1, 1, N)).astype(np.float32)
        mass[0, 0, rng.integers(0, N)] = rng.choice([np.nan, np.inf, -np.inf, -0.0])
        keep = oracle.evict(mass, budget, recent, n_sink, [L])[0, 0]
        n = min(L, budget)
        assert (keep[n:] == -1).all() and (np.diff(keep[:n]) > 0).all()
        always = {j for j in range(L) if j < n_sink or j >= L - recent}
        assert always <= set(keep[:n])

        def value(j):
            x = mass[0, 0, j]
            return (-math.inf, 0) if np.isnan(x) else (float(x), 1)

        best = None
        for some in itertools.combinations(sorted(set(range(L)) - always), n - len(always)):
            score = (sorted((value(j) for j in some), reverse=True), [-j for j in some])
            best = score if best is None or score > best else best
        chosen = [j for j in keep[:n] if j not in always]
        assert (sorted((value(j) for j in chosen), reverse=True), [-j for j in chosen]) == best


# ---------------------------------------------------------------- refusals
def _desc(B=1, H=2, N=256, D=128, ptr=0x100000, **kw):
    t = bd.PbsTensor(ptr, B, H, N, D, H * N * D, N * D, D)
    for name, v in kw.items():
        setattr(t, name, v)
    return t


P = ctypes.c_void_p


def _window(lib, q=None, k=None, v=None, o=None, window=16, n_sink=0, scale=0.1, ws=0x4000, n=1 << 40):
    q = q or _desc(H=4, N=3)
    k = k or _desc()
    return lib.pbs_attn_window(q, k, v or _desc(B=k.B, H=k.H, N=k.N, D=k.D), None, None, window, n_sink, scale,
                               o or _desc(B=q.B, H=q.H, N=q.N, D=q.D), None, P(ws), n, None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(q=_desc(H=4, N=3, ptr=0)), -1, b"null"),
    (dict(q=_desc(H=4, N=3, D=96)), -2, b"head dim"),
    (dict(q=_desc(H=4, N=3, ptr=0x100008)), -2, b"aligned"),
    (dict(k=_desc(sN=132)), -2, b"strides"),
    (dict(q=_desc(H=3, N=3)), -1, b"multiple"),
    (dict(q=_desc(H=130, N=3)), -2, b"64"),
    (dict(q=_desc(B=2, H=4, N=3)), -1, b"disagree"),
    (dict(q=_desc(H=4, N=3, sH=0)), -2, b"broadcast"),
    (dict(o=_desc(H=4, N=3, sH=0)), -2, b"broadcast"),
    (dict(o=_desc(H=4, N=4)), -1, b"O shape"),
    (dict(v=_desc(N=128)), -1, b"V shape"),
    (dict(window=-1), -1, b"negative"),
    (dict(n_sink=-1), -1, b"negative"),
    (dict(scale=0.0), -1, b"softmax_scale"),
    (dict(scale=float("nan")), -1, b"softmax_scale"),
    (dict(scale=float("inf")), -1, b"softmax_scale"),
    (dict(scale=3e38), -1, b"softmax_scale"),
    (dict(q=_desc(B=300, H=256, N=1), k=_desc(B=300, H=256)), -2, b"65535"),
])
def test_attn_window_refusals(lib, kw, code, word):
    assert _window(lib, **kw) == code
    assert word in lib.pbs_get_last_error()


def test_workspace_is_checked(lib):
    q, k = _desc(B=1, H=4, N=1), _desc(N=1 << 20)
    need = lib.pbs_workspace_size(pbs.PBS_OP_ATTN_WINDOW, q, k, 0, 0)
    if need:
        assert _window(lib, q=q, k=k, n=need - 1) == -1
        assert _window(lib, q=q, k=k, ws=0x4010) == -1
        assert _window(lib, q=q, k=k, ws=0) == -1
    for op in (pbs.PBS_OP_ATTN_WINDOW, pbs.PBS_OP_ATTN_PREFIX, pbs.PBS_OP_KEY_MASS, pbs.PBS_OP_EVICT):
        assert lib.pbs_workspace_size(op, _desc(D=96), k, 0, 0) == 0


def test_attn_prefix_refusals(lib):
    q, k, o = _desc(B=3, H=4, N=1), _desc(B=3), _desc(B=3, H=4, N=1)

    def call(kp, vp):
        return lib.pbs_attn_prefix(q, kp, vp, k, _desc(B=3), None, None, 0.1, o, None, P(0x4000), 1 << 40, None)

    for kp, vp, word in ((_desc(B=3), _desc(B=3), b"Kp"), (_desc(H=1), _desc(H=1), b"Kp"),
                         (_desc(D=64), _desc(D=64), b"Kp"), (_desc(), _desc(N=255), b"Vp shape")):
        assert call(kp, vp) == -1 and word in lib.pbs_get_last_error()
    assert call(None, _desc()) == -1


def test_key_mass_refusals(lib):
    q, k = _desc(H=4, N=3), _desc()

    def call(lse=0x2000, decay=1.0, prev=0x8000, s_prev=256, mass=0x9000, s_mass=256, window=0):
        return lib.pbs_key_mass(q, k, P(lse), None, None, window, 0, decay, 0.1, P(prev), s_prev, P(mass), s_mass,
                                P(0x4000), 1 << 40, None)

    for kw in (dict(lse=0), dict(mass=0), dict(s_mass=255), dict(s_prev=255), dict(decay=-1.0),
               dict(decay=float("nan")), dict(decay=float("inf")), dict(window=-1),
               dict(prev=0x9000, s_prev=512), dict(prev=0x9004), dict(prev=0x9000 - 4 * 300)):
        assert call(**kw) == -1, kw


def test_evict_refusals(lib):
    k = _desc(ptr=0x1000000)

    def call(budget=64, recent=8, n_sink=4, ko=None, vo=None, mass=0x2000, s=256, keep=0x3000, out=0x5000, s_out=64):
        return lib.pbs_evict(P(mass), s, k, _desc(ptr=0x2000000), None, budget, recent, n_sink, P(keep), None,
                             ko or _desc(N=64, ptr=0x3000000), vo or _desc(N=64, ptr=0x4000000), P(out), s_out,
                             P(0x4000), 1 << 40, None)

    for kw, code in ((dict(budget=0), -1), (dict(budget=257), -1), (dict(budget=65), -1), (dict(recent=61), -1),
                     (dict(recent=-1), -1), (dict(n_sink=-1), -1), (dict(mass=0), -1), (dict(keep=0), -1),
                     (dict(out=0), -1), (dict(s=255), -1), (dict(s_out=63), -1), (dict(out=0x2000), -1),
                     (dict(out=0x2000 + 4 * 100), -1), (dict(vo=_desc(N=64, ptr=0x3000100)), -1),
                     (dict(ko=_desc(N=64, ptr=0x1000000)), -1), (dict(vo=_desc(N=64, ptr=0x2000100)), -1),
                     (dict(ko=_desc(H=1, N=64, ptr=0x3000000)), -1), (dict(ko=_desc(N=70, ptr=0x3000000)), -1),
                     (dict(ko=_desc(N=64, ptr=0x3000000, sH=0)), -2)):
        assert call(**kw) == code, kw


def test_overlapping_views_are_refused(lib):
    """Arrays of equal strides that lie in one another and share an element."""
    def evict(ko, vo, k=None, out=0x5000, s=256, s_out=64):
        return lib.pbs_evict(P(0x2000), s, k or _desc(ptr=0x1000000), _desc(ptr=0x2000000), None, 64, 8, 4, P(0x3000),
                             None, ko, vo, P(out), s_out, P(0x4000), 1 << 40, None)

    ko = _desc(N=64, ptr=0x3000000)
    row, head = 2 * 128, 2 * 64 * 128                       # bytes
    wide = dict(N=64, sH=2 * 64 * 128, sB=4 * 64 * 128)     # heads of K_out and V_out in turn
    for ko, vo in ((ko, _desc(N=64, ptr=0x3000000 + head)), (ko, _desc(N=64, ptr=0x3000000 - head)),
                   (_desc(ptr=0x3000000, **wide), _desc(ptr=0x3000000 + head - row, **wide)),
                   (_desc(ptr=0x3000000, **wide), _desc(ptr=0x3000000 - head + 16, **wide)),
                   (_desc(N=64, ptr=0x3000000, sN=256, sH=64 * 256),                  # elements in turn
                    _desc(N=64, ptr=0x3000000 + 2 * 128 - 16, sN=256, sH=64 * 256))):
        assert evict(ko, vo) == -1 and b"overlap" in lib.pbs_get_last_error()
    ko, vo = _desc(N=64, ptr=0x3000000), _desc(N=64, ptr=0x4000000)
    for off, s in ((255, 256), (256, 319), (-63, 320), (-1, 256)):                    # behind and before mass's rows
        assert evict(ko, vo, out=0x2000 + 4 * off, s=s, s_out=s) == -1 and b"overlap" in lib.pbs_get_last_error()


def test_binding_refusals(lib):
    x = torch.zeros(1, 2, 16, 64, dtype=torch.bfloat16)
    for call in (lambda: pbs.pbs_attn_window(x, x, x), lambda: pbs.pbs_attn_prefix(x, x, x, x, x),
                 lambda: pbs.pbs_key_mass(x, x, torch.zeros(1, 2, 16)),
                 lambda: pbs.pbs_evict(torch.zeros(1, 2, 16), x, x, 8)):
        with pytest.raises(ValueError):          # not CUDA tensors
            call()
    with pytest.raises(ValueError):
        pbs.pbs_attn_prefix(x, None, None, x, x)
    with pytest.raises(ValueError):
        bd._lengths("kv_len", torch.zeros(2, dtype=torch.int64), 2)
    with pytest.raises(ValueError):
        bd._lengths("kv_len", torch.zeros(3, dtype=torch.int32), 2)
    with pytest.raises(ValueError):
        bd._row_stride("mass", torch.zeros(2, 3, 8)[:, :2], (2, 2, 8))      # rows not evenly spaced
    with pytest.raises(ValueError):
        bd._row_stride("mass", torch.zeros(2, 3, 8).transpose(1, 2), (2, 8, 3))
    with pytest.raises(TypeError):
        bd._row_stride("mass", torch.zeros(2, 3, 8, dtype=torch.float64), (2, 3, 8))
    assert bd._row_stride("mass", torch.zeros(2, 3, 20)[..., :8], (2, 3, 8)) == 20
    with pytest.raises(ValueError):
        bd._int32("n_sink", 1 << 31)
