"""ctypes binding of libpbs.so: argument marshalling only.

Every function here checks types, builds the C descriptors, allocates the
caller-side buffers the C ABI asks for (outputs, workspace) with torch, and
calls the library on torch's current CUDA stream.  All computation happens in
the library's sm_100a kernels; there is no fallback: if libpbs.so is missing
or fails to load, every call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import os
from typing import Optional, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpbs.so")

PBS_OP_PERMUTE, PBS_OP_SELECT, PBS_OP_ATTN, PBS_OP_PERMUTE_SEGMENTED, PBS_OP_SELECT_SEGMENTED = 0, 1, 2, 3, 4
PBS_OP_SELECT_SAMPLE = 5
PBS_OP_PERMUTE_QUERIES = 6
PBS_OP_ATTN_WINDOW, PBS_OP_ATTN_PREFIX, PBS_OP_KEY_MASS, PBS_OP_EVICT = 7, 8, 9, 10
PBS_SELECT_TOPK, PBS_SELECT_TAU, PBS_SELECT_SAMPLE = 0, 1, 2
_MODES = {"topk": PBS_SELECT_TOPK, "tau": PBS_SELECT_TAU, "sample": PBS_SELECT_SAMPLE}
PBS_SELECT_SCORE_ORDER, PBS_SELECT_PERM_PER_SEGMENT = 0x10, 0x20
PBS_ATTN_EARLY_STOP, PBS_ATTN_PERM_PER_SEGMENT, PBS_ATTN_CTA_PAIR = 1, 2, 4
STATUS = {0: "PBS_OK", -1: "PBS_ERR_INVALID_ARG", -2: "PBS_ERR_UNSUPPORTED", -3: "PBS_ERR_CAPACITY",
          -4: "PBS_ERR_CUDA", -5: "PBS_ERR_TIMEOUT", -6: "PBS_ERR_DEVICE_CHECK"}
EXPORTS = ("pbs_workspace_size", "pbs_permute", "pbs_permute_segmented", "pbs_select_capacity", "pbs_select",
           "pbs_attn_fwd", "pbs_attn_fwd_early_stop", "pbs_attn_fwd_ex", "pbs_check_device",
           "pbs_get_last_error", "pbs_version", "pbs_permute_noalloc", "pbs_test_inject_timeout",
           "pbs_permute_queries", "pbs_select_qperm", "pbs_attn_fwd_qperm",
           "pbs_attn_window", "pbs_attn_prefix", "pbs_key_mass", "pbs_evict")


class PbsError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{STATUS.get(code, code)}: {msg}")
        self.code = code


class PbsTensor(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p),
                ("B", ctypes.c_int64), ("H", ctypes.c_int64), ("N", ctypes.c_int64), ("D", ctypes.c_int64),
                ("sB", ctypes.c_int64), ("sH", ctypes.c_int64), ("sN", ctypes.c_int64)]


_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libpbs.so and declare its signatures (raises if missing)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"libpbs.so not built at {path}; run python -m permuted_block_sparse_b200.build")
    lib = ctypes.CDLL(path)
    P = ctypes.POINTER(PbsTensor)
    vp, i32, i64, dbl, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_double, ctypes.c_size_t
    lib.pbs_workspace_size.argtypes = [i32, P, P, i32, i32]
    lib.pbs_workspace_size.restype = sz
    lib.pbs_permute.argtypes = [P, P, i32, i32, i32, vp, vp, sz, vp]
    lib.pbs_permute.restype = i32
    lib.pbs_permute_segmented.argtypes = [P, P, i32, i32, i32, vp, vp, sz, vp]
    lib.pbs_permute_segmented.restype = i32
    lib.pbs_attn_fwd_ex.argtypes = [P, P, P, vp, vp, vp, i32, i32, i32, ctypes.c_uint, vp, ctypes.c_float,
                                    ctypes.c_float, P, vp, vp, vp]
    lib.pbs_attn_fwd_ex.restype = i32
    lib.pbs_select_capacity.argtypes = [i64, i32, i32, i32, dbl, i32, i32]
    lib.pbs_select_capacity.restype = i32
    lib.pbs_select.argtypes = [P, P, vp, i32, i32, i32, dbl, i32, i32, vp, vp, i32, vp, sz, vp]
    lib.pbs_select.restype = i32
    lib.pbs_attn_fwd.argtypes = [P, P, P, vp, vp, vp, i32, i32, i32, vp, ctypes.c_float, P, vp, vp, vp, sz, vp]
    lib.pbs_attn_fwd.restype = i32
    lib.pbs_attn_fwd_early_stop.argtypes = [P, P, P, vp, vp, vp, i32, i32, i32, ctypes.c_float, ctypes.c_float,
                                            P, vp, vp, vp]
    lib.pbs_attn_fwd_early_stop.restype = i32
    lib.pbs_check_device.argtypes = [vp]
    lib.pbs_check_device.restype = i32
    lib.pbs_permute_queries.argtypes = [P, P, i32, i32, vp, vp, sz, vp]
    lib.pbs_permute_queries.restype = i32
    lib.pbs_select_qperm.argtypes = [P, P, vp, vp, i32, i32, i32, dbl, i32, vp, vp, i32, vp, sz, vp]
    lib.pbs_select_qperm.restype = i32
    lib.pbs_attn_fwd_qperm.argtypes = [P, P, P, vp, vp, vp, vp, i32, i32, i32, ctypes.c_float, P, vp, vp, vp]
    lib.pbs_attn_fwd_qperm.restype = i32
    f32 = ctypes.c_float
    lib.pbs_attn_window.argtypes = [P, P, P, vp, vp, i64, i32, f32, P, vp, vp, sz, vp]
    lib.pbs_attn_window.restype = i32
    lib.pbs_attn_prefix.argtypes = [P, P, P, P, P, vp, vp, f32, P, vp, vp, sz, vp]
    lib.pbs_attn_prefix.restype = i32
    lib.pbs_key_mass.argtypes = [P, P, vp, vp, vp, i64, i32, f32, f32, vp, i64, vp, i64, vp, sz, vp]
    lib.pbs_key_mass.restype = i32
    lib.pbs_evict.argtypes = [vp, i64, P, P, vp, i32, i32, i32, vp, vp, P, P, vp, i64, vp, sz, vp]
    lib.pbs_evict.restype = i32
    lib.pbs_test_inject_timeout.argtypes = [ctypes.c_uint]
    lib.pbs_test_inject_timeout.restype = None
    lib.pbs_get_last_error.argtypes = []
    lib.pbs_get_last_error.restype = ctypes.c_char_p
    lib.pbs_version.argtypes = []
    lib.pbs_version.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _check(rc: int) -> None:
    if rc != 0:
        raise PbsError(rc, load().pbs_get_last_error().decode())


def describe(t: torch.Tensor) -> PbsTensor:
    """pbs_tensor for a [B, H, N, D] bf16 CUDA tensor with unit D stride."""
    if t.dim() != 4:
        raise ValueError("expected a [B, H, N, D] tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError("expected bfloat16")
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if t.stride(3) != 1:
        raise ValueError("the D dimension must be contiguous")
    B, H, N, D = t.shape
    sB, sH, sN, _ = t.stride()
    return PbsTensor(t.data_ptr(), B, H, N, D, sB, sH, sN)


_HERE_AND_NOW = contextlib.nullcontext()


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _workspace(nbytes: int, device) -> Optional[torch.Tensor]:
    if nbytes == 0:
        return None
    return torch.empty(nbytes + 256, dtype=torch.uint8, device=device)


def _aligned(ws: Optional[torch.Tensor]) -> Tuple[Optional[int], int]:
    if ws is None:
        return None, 0
    p = ws.data_ptr()
    a = (p + 255) & ~255
    return a, ws.numel() - (a - p)


def workspace_size(op: int, Q: torch.Tensor, K: torch.Tensor, blk: int, seg: int) -> int:
    q, k = describe(Q), describe(K)
    return load().pbs_workspace_size(op, ctypes.byref(q), ctypes.byref(k), blk, seg)


def select_capacity(N: int, blk: int, seg: int, mode: str, density_or_tau: float,
                    band: int = 0, n_sink: int = 0) -> int:
    if mode not in _MODES:
        raise ValueError(f"unknown selection mode {mode!r}; expected one of {sorted(_MODES)}")
    m = _MODES[mode]
    rc = load().pbs_select_capacity(N, blk, seg, m, float(density_or_tau), band, n_sink)
    _check(min(rc, 0))
    return rc


def pbs_permute(Q: torch.Tensor, K: torch.Tensor, blk: int, seg: int, n_sink: int = 0,
                perm: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """perm [B, Hkv, N] int32: per-segment stable descending sort of keys."""
    lib = load()
    q, k = describe(Q), describe(K)
    B, Hkv, N, _ = K.shape
    if perm is None:
        perm = torch.empty((B, Hkv, N), dtype=torch.int32, device=K.device)
    if ws is None:
        ws = _workspace(lib.pbs_workspace_size(PBS_OP_PERMUTE, ctypes.byref(q), ctypes.byref(k), blk, seg), K.device)
    wp, wn = _aligned(ws)
    _check(lib.pbs_permute(ctypes.byref(q), ctypes.byref(k), blk, seg, n_sink, perm.data_ptr(), wp, wn,
                           _stream(stream)))
    return perm


def pbs_permute_segmented(Q: torch.Tensor, K: torch.Tensor, blk: int, seg: int, n_sink: int = 0,
                          perm: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                          stream=None) -> torch.Tensor:
    """perm [B, Hkv, nseg, N] int32: one permutation per query segment (its
    history's key segments sorted by the segment's pooled query)."""
    lib = load()
    q, k = describe(Q), describe(K)
    B, Hkv, N, _ = K.shape
    nseg = (N + seg - 1) // seg
    if perm is None:
        perm = torch.empty((B, Hkv, nseg, N), dtype=torch.int32, device=K.device)
    if ws is None:
        ws = _workspace(lib.pbs_workspace_size(PBS_OP_PERMUTE_SEGMENTED, ctypes.byref(q), ctypes.byref(k), blk, seg),
                        K.device)
    wp, wn = _aligned(ws)
    _check(lib.pbs_permute_segmented(ctypes.byref(q), ctypes.byref(k), blk, seg, n_sink, perm.data_ptr(), wp, wn,
                                     _stream(stream)))
    return perm


def pbs_select(Q: torch.Tensor, K: torch.Tensor, perm: torch.Tensor, blk: int, seg: int,
               mode: str = "topk", density_or_tau: float = 1.0, band: int = 0, n_sink: int = 0,
               cap: Optional[int] = None, counts: Optional[torch.Tensor] = None,
               idx: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
               stream=None, score_order: bool = False) -> Tuple[torch.Tensor, torch.Tensor]:
    """(counts [B, Hq, nb] int32, idx [B, Hq, nb, cap] int32) block lists,
    ascending, or in visiting order (forced blocks, then descending block
    score) with ``score_order``."""
    lib = load()
    q, k = describe(Q), describe(K)
    B, Hq, N, _ = Q.shape
    nb = N // blk
    if mode not in _MODES:
        raise ValueError(f"unknown selection mode {mode!r}; expected one of {sorted(_MODES)}")
    m = _MODES[mode]
    if score_order:
        m |= PBS_SELECT_SCORE_ORDER
    op = PBS_OP_SELECT_SAMPLE if mode == "sample" else PBS_OP_SELECT
    if perm is not None and perm.dim() == 4:   # one permutation per query segment
        m |= PBS_SELECT_PERM_PER_SEGMENT
        op = PBS_OP_SELECT_SEGMENTED
    if cap is None:
        cap = max(1, select_capacity(N, blk, seg, mode, density_or_tau, band, n_sink))
    if counts is None:
        counts = torch.empty((B, Hq, nb), dtype=torch.int32, device=Q.device)
    if idx is None:
        idx = torch.empty((B, Hq, nb, cap), dtype=torch.int32, device=Q.device)
    if ws is None:
        ws = _workspace(lib.pbs_workspace_size(op, ctypes.byref(q), ctypes.byref(k), blk, seg), Q.device)
    wp, wn = _aligned(ws)
    _check(lib.pbs_select(ctypes.byref(q), ctypes.byref(k), _ptr(perm), blk, seg, m, float(density_or_tau),
                          band, n_sink, counts.data_ptr(), idx.data_ptr(), cap, wp, wn, _stream(stream)))
    return counts, idx


def pbs_attn_fwd(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, perm: torch.Tensor,
                 counts: torch.Tensor, idx: torch.Tensor, blk: int, seg: int,
                 gate_thr: Optional[torch.Tensor] = None, softmax_scale: Optional[float] = None,
                 out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                 want_lse: bool = True, stats: Optional[torch.Tensor] = None,
                 stream=None, cta_pair: bool = False) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """(O [B, Hq, N, D] bf16, LSE [B, Hq, N] fp32 or None).  ``cta_pair``
    runs the CTA-pair kernel where it applies (d = blk = 128, query heads per
    KV head a multiple of 4, no gate); its results are the same."""
    lib = load()
    B, Hq, N, D = Q.shape
    if out is None:
        out = torch.empty_like(Q)
    if lse is None and want_lse:
        lse = torch.empty((B, Hq, N), dtype=torch.float32, device=Q.device)
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    if gate_thr is not None and gate_thr.dtype != torch.float32:
        raise TypeError("gate_thr must be float32")
    if stats is not None and stats.dtype != torch.int64:
        raise TypeError("stats must be int64")
    q, k, v, o = describe(Q), describe(K), describe(V), describe(out)
    flags = (PBS_ATTN_PERM_PER_SEGMENT if perm.dim() == 4 else 0) | (PBS_ATTN_CTA_PAIR if cta_pair else 0)
    if flags:                                # one permutation per query segment / one-CTA kernel
        _check(lib.pbs_attn_fwd_ex(ctypes.byref(q), ctypes.byref(k), ctypes.byref(v), perm.data_ptr(),
                                   counts.data_ptr(), idx.data_ptr(), idx.shape[-1], blk, seg,
                                   flags, _ptr(gate_thr), 0.0, float(softmax_scale),
                                   ctypes.byref(o), _ptr(lse), _ptr(stats), _stream(stream)))
        return out, lse
    _check(lib.pbs_attn_fwd(ctypes.byref(q), ctypes.byref(k), ctypes.byref(v), perm.data_ptr(),
                            counts.data_ptr(), idx.data_ptr(), idx.shape[-1], blk, seg, _ptr(gate_thr),
                            float(softmax_scale), ctypes.byref(o), _ptr(lse), _ptr(stats), None, 0,
                            _stream(stream)))
    return out, lse


def pbs_permute_queries(Q: torch.Tensor, K: torch.Tensor, blk: int, seg: int,
                        qperm: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    """qperm [B, Hq, N] int32: S2O's query permutation (per segment, queries
    by descending score against the KV head's guide vector)."""
    lib = load()
    q, k = describe(Q), describe(K)
    B, Hq, N, _ = Q.shape
    if qperm is None:
        qperm = torch.empty((B, Hq, N), dtype=torch.int32, device=Q.device)
    if ws is None:
        ws = _workspace(lib.pbs_workspace_size(PBS_OP_PERMUTE_QUERIES, ctypes.byref(q), ctypes.byref(k), blk, seg),
                        Q.device)
    wp, wn = _aligned(ws)
    _check(lib.pbs_permute_queries(ctypes.byref(q), ctypes.byref(k), blk, seg, qperm.data_ptr(), wp, wn,
                                   _stream(stream)))
    return qperm


def pbs_select_qperm(Q: torch.Tensor, K: torch.Tensor, perm: torch.Tensor, qperm: torch.Tensor, blk: int,
                     seg: int, mode: str = "topk", density_or_tau: float = 1.0, n_sink: int = 0,
                     cap: Optional[int] = None, counts: Optional[torch.Tensor] = None,
                     idx: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                     stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(counts, idx) block lists of the permuted query blocks (ascending)."""
    lib = load()
    q, k = describe(Q), describe(K)
    B, Hq, N, _ = Q.shape
    nb = N // blk
    if mode not in ("topk", "tau"):
        raise ValueError(f"permuted queries take mode 'topk' or 'tau', not {mode!r}")
    if cap is None:
        cap = max(1, select_capacity(N, blk, seg, mode, density_or_tau, 0, n_sink))
    if counts is None:
        counts = torch.empty((B, Hq, nb), dtype=torch.int32, device=Q.device)
    if idx is None:
        idx = torch.empty((B, Hq, nb, cap), dtype=torch.int32, device=Q.device)
    if ws is None:
        ws = _workspace(lib.pbs_workspace_size(PBS_OP_SELECT, ctypes.byref(q), ctypes.byref(k), blk, seg), Q.device)
    wp, wn = _aligned(ws)
    _check(lib.pbs_select_qperm(ctypes.byref(q), ctypes.byref(k), perm.data_ptr(), qperm.data_ptr(), blk, seg,
                                _MODES[mode], float(density_or_tau), n_sink, counts.data_ptr(), idx.data_ptr(), cap,
                                wp, wn, _stream(stream)))
    return counts, idx


def pbs_attn_fwd_qperm(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, perm: torch.Tensor,
                       qperm: torch.Tensor, counts: torch.Tensor, idx: torch.Tensor, blk: int, seg: int,
                       softmax_scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                       lse: Optional[torch.Tensor] = None, want_lse: bool = True,
                       stats: Optional[torch.Tensor] = None,
                       stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """(O, LSE) at the queries' original positions, for lists indexed by
    permuted query block."""
    lib = load()
    B, Hq, N, D = Q.shape
    if out is None:
        out = torch.empty_like(Q)
    if lse is None and want_lse:
        lse = torch.empty((B, Hq, N), dtype=torch.float32, device=Q.device)
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    if stats is not None and stats.dtype != torch.int64:
        raise TypeError("stats must be int64")
    q, k, v, o = describe(Q), describe(K), describe(V), describe(out)
    _check(lib.pbs_attn_fwd_qperm(ctypes.byref(q), ctypes.byref(k), ctypes.byref(v), perm.data_ptr(),
                                  qperm.data_ptr(), counts.data_ptr(), idx.data_ptr(), idx.shape[-1], blk, seg,
                                  float(softmax_scale), ctypes.byref(o), _ptr(lse), _ptr(stats), _stream(stream)))
    return out, lse


def pbs_attn_fwd_early_stop(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, perm: torch.Tensor,
                            counts: torch.Tensor, idx: torch.Tensor, blk: int, seg: int, stop_tau: float,
                            softmax_scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                            lse: Optional[torch.Tensor] = None, want_lse: bool = True,
                            stats: Optional[torch.Tensor] = None,
                            stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """(O, LSE): S2O's two passes with the early-stopping rule; ``idx`` holds
    each block's list in visiting order."""
    lib = load()
    B, Hq, N, D = Q.shape
    if out is None:
        out = torch.empty_like(Q)
    if lse is None and want_lse:
        lse = torch.empty((B, Hq, N), dtype=torch.float32, device=Q.device)
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    if stats is not None and stats.dtype != torch.int64:
        raise TypeError("stats must be int64")
    q, k, v, o = describe(Q), describe(K), describe(V), describe(out)
    if perm.dim() == 4:                      # one permutation per query segment
        _check(lib.pbs_attn_fwd_ex(ctypes.byref(q), ctypes.byref(k), ctypes.byref(v), perm.data_ptr(),
                                   counts.data_ptr(), idx.data_ptr(), idx.shape[-1], blk, seg,
                                   PBS_ATTN_EARLY_STOP | PBS_ATTN_PERM_PER_SEGMENT, None, float(stop_tau),
                                   float(softmax_scale), ctypes.byref(o), _ptr(lse), _ptr(stats),
                                   _stream(stream)))
        return out, lse
    _check(lib.pbs_attn_fwd_early_stop(ctypes.byref(q), ctypes.byref(k), ctypes.byref(v), perm.data_ptr(),
                                       counts.data_ptr(), idx.data_ptr(), idx.shape[-1], blk, seg,
                                       float(stop_tau), float(softmax_scale), ctypes.byref(o), _ptr(lse),
                                       _ptr(stats), _stream(stream)))
    return out, lse


# --------------------------------------------------------- cache operators
# Stream handle of a device's current stream; the private function is the one
# torch's own code generators launch by, 3 us cheaper than a Stream object.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _place(stream, first: torch.Tensor, *others: Optional[torch.Tensor]):
    """Context in which a cache operator allocates and launches: the tensors'
    device, and ``stream`` where one is given, so that what is allocated here
    belongs to the stream that uses it."""
    dev = first.get_device()
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensors on {first.device} and {t.device}")
    if stream is not None:
        if stream.device != first.device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {first.device}")
        return torch.cuda.stream(stream)
    if dev >= 0 and dev != torch.cuda.current_device():
        return torch.cuda.device(dev)
    return _HERE_AND_NOW


@functools.lru_cache(maxsize=512)
def _cache_ws_bytes(op: int, B: int, Hq: int, M: int, D: int, Hkv: int, N: int) -> int:
    q = PbsTensor(256, B, Hq, M, D, Hq * M * D, M * D, D)        # only the shapes are read
    k = PbsTensor(256, B, Hkv, N, D, Hkv * N * D, N * D, D)
    return load().pbs_workspace_size(op, q, k, 0, 0)


def _cache_ws(ws: Optional[torch.Tensor], nbytes: int, like: torch.Tensor):
    """(owner, address, bytes) of the caller's workspace or a new one."""
    if ws is None:
        if nbytes == 0:
            return None, None, 0
        ws = like.new_empty(nbytes + 256, dtype=torch.uint8)
    return ws, *_aligned(ws)


def _lengths(name: str, t: Optional[torch.Tensor], B: int) -> Optional[int]:
    if t is None:
        return None
    if t.dtype != torch.int32 or t.shape != (B,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape ({B},)")
    return t.data_ptr()


def _int32(name: str, x: int) -> int:
    if not -2 ** 31 <= x < 2 ** 31:          # ctypes would drop the upper bits
        raise ValueError(f"{name} = {x} does not fit 32 bits")
    return x


def _row_stride(name: str, t: torch.Tensor, shape: Tuple[int, ...]) -> int:
    """Elements between successive (b, hkv) rows of an fp32 [B, Hkv, n] tensor."""
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be float32")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    sB, sH, sn = t.stride()
    B, H, n = shape
    if H == 1:
        sH = sB if B > 1 else n
    if (sn != 1 and n > 1) or (B > 1 and sB != H * sH):
        raise ValueError(f"{name} must have unit stride within rows and evenly spaced (b, hkv) rows")
    return sH


def _check_out(name: str, t: torch.Tensor, dtype, shape: Tuple[int, ...]) -> None:
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape}")


def _cache_attn(Q, Kp, Vp, K, V, window, n_sink, kv_len, q_len, softmax_scale, out, lse, want_lse, ws, stream):
    lib = _lib or load()
    q, k, v = describe(Q), describe(K), describe(V)
    B, Hq, M, D = Q.shape
    kv, ql = _lengths("kv_len", kv_len, B), _lengths("q_len", q_len, B)
    _int32("n_sink", n_sink)
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    with _place(stream, Q, K, V, Kp, Vp, kv_len, q_len, out, lse, ws):
        if out is None:
            out = torch.empty_like(Q)
        if lse is not None:
            _check_out("lse", lse, torch.float32, (B, Hq, M))
        elif want_lse:
            lse = Q.new_empty((B, Hq, M), dtype=torch.float32)
        op = PBS_OP_ATTN_WINDOW if Kp is None else PBS_OP_ATTN_PREFIX
        ws, wp, wn = _cache_ws(ws, _cache_ws_bytes(op, B, Hq, M, D, k.H, k.N), Q)
        o, s = describe(out), _raw_stream(Q.get_device())
        if Kp is None:
            rc = lib.pbs_attn_window(q, k, v, kv, ql, window, n_sink, softmax_scale, o, _ptr(lse), wp, wn, s)
        else:
            rc = lib.pbs_attn_prefix(q, describe(Kp), describe(Vp), k, v, kv, ql, softmax_scale, o, _ptr(lse), wp, wn,
                                     s)
    _check(rc)
    return out, lse


def pbs_attn_window(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, window: int = 0, n_sink: int = 0,
                    kv_len: Optional[torch.Tensor] = None, q_len: Optional[torch.Tensor] = None,
                    softmax_scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                    lse: Optional[torch.Tensor] = None, want_lse: bool = True, ws: Optional[torch.Tensor] = None,
                    stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """(O [B, Hq, M, D] bf16, LSE [B, Hq, M] fp32 or None) of the newest M
    tokens over a cache of N keys per sequence, ``kv_len`` [B] int32 of them
    filled: every row sees the last ``window`` keys up to its own (0: all) and
    the first ``n_sink``.  With ``q_len`` [B] int32 only that many rows of each
    sequence are queries; the other rows of the outputs are not written."""
    return _cache_attn(Q, None, None, K, V, window, n_sink, kv_len, q_len, softmax_scale, out, lse, want_lse, ws,
                       stream)


def pbs_attn_prefix(Q: torch.Tensor, Kp: torch.Tensor, Vp: torch.Tensor, K: torch.Tensor, V: torch.Tensor,
                    kv_len: Optional[torch.Tensor] = None, q_len: Optional[torch.Tensor] = None,
                    softmax_scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                    lse: Optional[torch.Tensor] = None, want_lse: bool = True, ws: Optional[torch.Tensor] = None,
                    stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """(O, LSE) of a batch over one shared prefix ``Kp``, ``Vp``
    [1, Hkv, P, D], read once for the batch, and each sequence's own cache
    ``K``, ``V`` after it (lengths as for :func:`pbs_attn_window`)."""
    if Kp is None or Vp is None:
        raise ValueError("Kp and Vp are needed")
    return _cache_attn(Q, Kp, Vp, K, V, 0, 0, kv_len, q_len, softmax_scale, out, lse, want_lse, ws, stream)


def pbs_key_mass(Q: torch.Tensor, K: torch.Tensor, lse: torch.Tensor, mass: Optional[torch.Tensor] = None,
                 decay: float = 1.0, window: int = 0, n_sink: int = 0, kv_len: Optional[torch.Tensor] = None,
                 q_len: Optional[torch.Tensor] = None, softmax_scale: Optional[float] = None,
                 out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """[B, Hkv, N] fp32: ``decay`` times the earlier ``mass`` (None: zero) plus
    the attention weight that the rows of ``Q`` give each key, from the ``lse``
    of their attention.  ``out`` may be ``mass`` itself.  Rows are causal as in
    :func:`pbs_attn_window`: for the mass of a shared prefix that every row sees
    whole, pass each row as a sequence of its own over the broadcast prefix."""
    lib = _lib or load()
    q, k = describe(Q), describe(K)
    B, Hq, M, D = Q.shape
    shape = (B, k.H, k.N)
    kv, ql = _lengths("kv_len", kv_len, B), _lengths("q_len", q_len, B)
    _int32("n_sink", n_sink)
    _check_out("lse", lse, torch.float32, (B, Hq, M))
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    s_in = 0 if mass is None else _row_stride("mass", mass, shape)
    with _place(stream, Q, K, lse, mass, kv_len, q_len, out, ws):
        if out is None:
            out = Q.new_empty(shape, dtype=torch.float32)
        s_out = _row_stride("out", out, shape)
        ws, wp, wn = _cache_ws(ws, _cache_ws_bytes(PBS_OP_KEY_MASS, B, Hq, M, D, k.H, k.N), Q)
        rc = lib.pbs_key_mass(q, k, lse.data_ptr(), kv, ql, window, n_sink, decay, softmax_scale, _ptr(mass), s_in,
                              out.data_ptr(), s_out, wp, wn, _raw_stream(Q.get_device()))
    _check(rc)
    return out


def pbs_evict(mass: torch.Tensor, K: torch.Tensor, V: torch.Tensor, budget: int, recent: int = 0, n_sink: int = 0,
              kv_len: Optional[torch.Tensor] = None, keep: Optional[torch.Tensor] = None,
              K_out: Optional[torch.Tensor] = None, V_out: Optional[torch.Tensor] = None,
              mass_out: Optional[torch.Tensor] = None, new_len: Optional[torch.Tensor] = None,
              ws: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, ...]:
    """(keep [B, Hkv, budget] int32, K_out, V_out, mass_out, new_len [B] int32):
    every cache cut to ``budget`` keys, of which the first ``n_sink`` and the
    last ``recent`` always stay and the rest are those of highest ``mass``.
    ``K_out`` and ``V_out`` [B, Hkv, n >= budget, D] and ``mass_out``
    [B, Hkv, n >= budget] take the kept rows at their start.  ``new_len`` may be
    ``kv_len`` itself.  No workspace is needed; ``ws`` is not read."""
    lib = _lib or load()
    k, v = describe(K), describe(V)
    B, Hkv, N, D = K.shape
    kv = _lengths("kv_len", kv_len, B)
    s_in = _row_stride("mass", mass, (B, Hkv, N))
    if not 1 <= budget <= N:
        raise ValueError(f"budget {budget} is not in [1, N = {N}]")
    _int32("recent", recent), _int32("n_sink", n_sink)
    with _place(stream, K, V, mass, kv_len, keep, K_out, V_out, mass_out, new_len, ws):
        if keep is None:
            keep = K.new_empty((B, Hkv, budget), dtype=torch.int32)
        else:
            _check_out("keep", keep, torch.int32, (B, Hkv, budget))
        if K_out is None:
            K_out = K.new_empty((B, Hkv, budget if V_out is None else V_out.shape[2], D))
        if V_out is None:
            V_out = K.new_empty((B, Hkv, K_out.shape[2], D))
        if mass_out is None:
            mass_out = mass.new_empty((B, Hkv, budget))
        s_out = _row_stride("mass_out", mass_out, (B, Hkv) + tuple(mass_out.shape[2:]))
        if mass_out.shape[2] < budget:
            raise ValueError(f"mass_out has room for {mass_out.shape[2]} of {budget} keys")
        if new_len is None:
            new_len = K.new_empty((B,), dtype=torch.int32)
        else:
            _check_out("new_len", new_len, torch.int32, (B,))
        rc = lib.pbs_evict(mass.data_ptr(), s_in, k, v, kv, budget, recent, n_sink, keep.data_ptr(),
                           new_len.data_ptr(), describe(K_out), describe(V_out), mass_out.data_ptr(), s_out, None, 0,
                           _raw_stream(K.get_device()))
    _check(rc)
    return keep, K_out, V_out, mass_out, new_len


def pbs_check_device(stream=None) -> None:
    """Synchronise and raise if a device-side check or bounded wait failed."""
    _check(load().pbs_check_device(_stream(stream)))


def test_inject_timeout(limit_polls: int) -> None:
    """Failure-path test hook (see pbs.h): > 0 makes later attention launches
    time out on purpose (bounded waits, no fault); 0 turns it off."""
    load().pbs_test_inject_timeout(int(limit_polls))


def version() -> str:
    return load().pbs_version().decode()
