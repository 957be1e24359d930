"""Workspace queries and workspace checks of the cache operators at and past the
limits of their shapes, on the host."""
import ctypes

import pytest

import permuted_block_sparse_b200 as pbs
from permuted_block_sparse_b200 import _binding as bd

P = ctypes.c_void_p
OPS = (pbs.PBS_OP_ATTN_WINDOW, pbs.PBS_OP_ATTN_PREFIX, pbs.PBS_OP_KEY_MASS)


@pytest.fixture(scope="module")
def lib():
    from permuted_block_sparse_b200 import build
    build.build()
    return pbs.load()


def desc(B, H, N, D=64, ptr=0x100000):
    return bd.PbsTensor(ptr, B, H, N, D, H * N * D, N * D, D)


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("M", [1, 4, 300])
def test_workspace_of_head_groups_past_the_limit(lib, op, M):
    """Groups larger than a tile of query rows give size 0, and the call its refusal."""
    for G in (65, 128, 129, 256, 1 << 20):
        q, k = desc(1, G, M), desc(1, 1, 300)
        assert lib.pbs_workspace_size(op, q, k, 0, 0) == 0
        assert b"64" in lib.pbs_get_last_error()
        assert bd._cache_ws_bytes(op, 1, G, M, 64, 1, 300) == 0
    q, k, o = desc(1, 129, M), desc(1, 1, 300), desc(1, 129, M)
    rc = {pbs.PBS_OP_ATTN_WINDOW: lambda: lib.pbs_attn_window(q, k, k, None, None, 0, 0, 0.1, o, None, None, 0, None),
          pbs.PBS_OP_ATTN_PREFIX: lambda: lib.pbs_attn_prefix(q, k, k, k, k, None, None, 0.1, o, None, None, 0, None),
          pbs.PBS_OP_KEY_MASS: lambda: lib.pbs_key_mass(q, k, P(0x2000), None, None, 0, 0, 1.0, 0.1, None, 0,
                                                        P(0x9000), 300, None, 0, None)}[op]()
    assert rc == -2 and b"64" in lib.pbs_get_last_error()


@pytest.mark.parametrize("op", OPS)
def test_workspace_of_refused_shapes(lib, op):
    for q, k in ((desc(1, 3, 4), desc(1, 2, 300)), (desc(1, 2, 4), desc(1, 4, 300)), (desc(2, 4, 4), desc(1, 2, 300)),
                 (desc(1, 4, 4), desc(1, 2, 300, D=128)), (desc(1 << 32, 1 << 32, 4), desc(1 << 32, 1 << 32, 300)),
                 (desc(300, 256, 1), desc(300, 256, 64)), (desc(64, 64, 1 << 30), desc(64, 1, 64))):
        assert lib.pbs_workspace_size(op, q, k, 0, 0) == 0


def test_evict_refuses_overlapping_lengths(lib):
    k, v = desc(3, 2, 256, ptr=0x1000000), desc(3, 2, 256, ptr=0x2000000)
    ko, vo = desc(3, 2, 64, ptr=0x3000000), desc(3, 2, 64, ptr=0x4000000)

    def call(kv_len, new_len, keep=0x30000):
        return lib.pbs_evict(P(0x2000), 256, k, v, P(kv_len), 64, 8, 4, P(keep), P(new_len), ko, vo, P(0x50000), 64,
                             None, 0, None)

    end = 0x30000 + 4 * 3 * 2 * 64                          # of keep
    for kv_len, new_len in ((0x9000, 0x9004), (0x9008, 0x9000), (0x30000, 0x9000), (end - 4, 0x9000),
                            (0x9000, end - 4), (0x9000, 0x30000 - 8), (0, 0x30010)):
        assert call(kv_len, new_len) == -1 and b"overlap" in lib.pbs_get_last_error(), (hex(kv_len), hex(new_len))


@pytest.mark.parametrize("op", OPS)
def test_workspace_refusals(lib, op):
    """Too small, misaligned and null, for shapes whose keys or rows are cut into parts."""
    q, k = (desc(1, 4, 4000), desc(1, 1, 4000)) if op == pbs.PBS_OP_KEY_MASS else (desc(1, 4, 3), desc(1, 2, 1 << 20))
    o = desc(q.B, q.H, q.N, ptr=0x80000000)
    need = lib.pbs_workspace_size(op, q, k, 0, 0)
    assert need > 0 and need % 256 == 0

    def call(ws, n):
        if op == pbs.PBS_OP_ATTN_WINDOW:
            return lib.pbs_attn_window(q, k, k, None, None, 0, 0, 0.1, o, None, P(ws), n, None)
        if op == pbs.PBS_OP_ATTN_PREFIX:
            return lib.pbs_attn_prefix(q, k, k, k, k, None, None, 0.1, o, None, P(ws), n, None)
        return lib.pbs_key_mass(q, k, P(0x2000), None, None, 0, 0, 1.0, 0.1, None, 0, P(0x90000000), k.N, P(ws), n, None)

    for ws, n in ((0x4000, need - 1), (0x4000, 0), (0x4010, need), (0, need)):
        assert call(ws, n) == -1 and b"workspace" in lib.pbs_get_last_error(), (hex(ws), n)
