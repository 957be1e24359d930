"""Helpers shared by the tests of the cache operators: a masked dense
reference in fp64 torch (either device), and tolerances that follow from the
number formats."""
from __future__ import annotations

import math

import torch

# Half a step of bf16, relative: one rounding is off by at most this.
HALF = torch.finfo(torch.bfloat16).eps / 2


def visible(B, M, N, window, n_sink, kv_len, q_len, device):
    """bool [B, M, N], and bool [B, M]: the rows that are computed."""
    L = torch.full((B,), N, device=device) if kv_len is None else kv_len.to(device).long()
    n = torch.full((B,), M, device=device) if q_len is None else q_len.to(device).long()
    r = torch.arange(M, device=device)
    pos = (L - n)[:, None] + r
    j = torch.arange(N, device=device)
    see = j <= pos[..., None]
    if window:
        see &= (j > pos[..., None] - window) | (j < n_sink)
    return see & (r < n[:, None])[..., None], r < n[:, None]


def reference(Q, K, V, window=0, n_sink=0, kv_len=None, q_len=None, scale=None, Kp=None, Vp=None):
    """fp64 (O, lse, A, S): A is the attention-weighted mean of |V| per output,
    S the largest scale * sum |q||k| over the keys a row sees.  Unseen keys and
    values are zeroed first, so what they hold does not matter; each row's own
    visible set is applied to the logits."""
    B, Hq, M, d = Q.shape
    G = Hq // K.shape[1]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    see, rows = visible(B, M, K.shape[2], window, n_sink, kv_len, q_len, Q.device)
    q = torch.where(rows[:, None, :, None], Q.double(), 0.0)
    used = see.any(1)[:, None, :, None]
    k = torch.where(used, K.double(), 0.0).repeat_interleave(G, 1)
    v = torch.where(used, V.double(), 0.0).repeat_interleave(G, 1)
    see = see[:, None].expand(B, Hq, M, see.shape[-1])
    if Kp is not None:
        k = torch.cat([Kp.double().repeat_interleave(G, 1).expand(B, -1, -1, -1), k], 2)
        v = torch.cat([Vp.double().repeat_interleave(G, 1).expand(B, -1, -1, -1), v], 2)
        see = torch.cat([rows[:, None, :, None].expand(B, Hq, M, Kp.shape[2]), see], 3)
    x = (q @ k.transpose(2, 3) * scale).masked_fill(~see, -math.inf)
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - torch.where(lse == -math.inf, 0.0, lse)[..., None])
    S = (q.abs() @ k.abs().transpose(2, 3) * scale).masked_fill(~see, 0.0).amax(-1)
    return p @ v, lse, p @ v.abs(), S


def assert_attention(O, lse, ref, rows, what=""):
    """Every computed element within the bound of its roundings: the weights
    once to bf16 and the output once to bf16 (HALF each, the first relative to
    the weighted mean of |V|, the second to a value that already carries the
    first), fp32 logits of at most 128 products (2^-16 of their absolute sum),
    and fp32 exponentials and sums (2^-18)."""
    Or, lr, A, S = ref
    rows = rows[:, None].expand(lr.shape)
    fp32 = (2.0 ** -16 * S + 2.0 ** -18)[..., None]
    tol = HALF * A + HALF * (Or.abs() + HALF * A) + 2 * fp32 * A
    err = (O.double() - Or).abs()
    bad = (~(err <= tol)) & rows[..., None]
    assert not bad.any(), f"{what}: {int(bad.sum())} outputs off, worst {(err / tol)[bad].max():.3g} of the bound"
    if lse is not None:
        finite = rows & torch.isfinite(lr)
        lerr = (lse.double() - lr).abs()
        ltol = 2.0 ** -16 * S + 2.0 ** -18 + 2.0 ** -22 * lr.abs()
        assert (lerr <= ltol)[finite].all(), f"{what}: lse off by {float(lerr[finite].max()):.3g}"
        assert (lse[rows & ~torch.isfinite(lr)] == -math.inf).all(), what


def reference_mass(Q, K, lse, prev=None, decay=1.0, window=0, n_sink=0, kv_len=None, q_len=None, scale=None):
    """fp64 (mass, tolerance).  A term exp(x - lse) is off by the relative error
    of its exponent: 2^-16 of the logit's absolute sum, 2^-22 of |lse| (its
    conversion to base 2), and 2^-20 for the exponential and the sums."""
    B, Hq, M, d = Q.shape
    Hkv, N = K.shape[1], K.shape[2]
    G = Hq // Hkv
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    see, rows = visible(B, M, N, window, n_sink, kv_len, q_len, Q.device)
    q = torch.where(rows[:, None, :, None], Q.double(), 0.0)
    k = torch.where(see.any(1)[:, None, :, None], K.double(), 0.0).repeat_interleave(G, 1)
    see = see[:, None] & (lse != -math.inf)[..., None]
    y = torch.where(rows[:, None] & (lse != -math.inf), lse.double(), 0.0)
    p = torch.exp(q @ k.transpose(2, 3) * scale - y[..., None]).masked_fill(~see, 0.0)
    S = (q.abs() @ k.abs().transpose(2, 3) * scale).masked_fill(~see, 0.0)
    part = p.reshape(B, Hkv, G * M, N).sum(2)
    tol = (p * (2.0 ** -16 * S + 2.0 ** -22 * y.abs()[..., None] + 2.0 ** -20)).reshape(B, Hkv, G * M, N).sum(2)
    if prev is not None:
        L = torch.full((B,), N, device=Q.device) if kv_len is None else kv_len.long()
        live = torch.arange(N, device=Q.device) < L[:, None, None]
        old = torch.where(live, decay * prev.double(), 0.0)
        part, tol = part + old, tol + 2.0 ** -22 * (old.abs() + part)
    return part, tol
