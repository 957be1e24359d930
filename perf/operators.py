"""Measured cases of the cache operators that follow a prefill: attention with a
sliding window and visible first tokens, attention of a batch over a shared
prefix, attention mass per key, and eviction by that mass.

``run`` computes each operator in plain torch operations (fp32 inside, rounded
once at the end), or, with ``own`` set, through the package's entry points.
Shapes are those of the package's workloads (Hq 32, Hkv 8, d 128; up to 32K
tokens; 128 sink keys) and generic odd ones.
"""
import math

import numpy as np
import torch

own = False

_INF = float("inf")


# ------------------------------------------------------------------- the cases
def listed():
    return [
        # one new token of one conversation, short window: launch latency
        dict(name="window_decode_one", op="window", B=1, Hq=32, Hkv=8, d=128, M=1, N=1024, window=256, n_sink=4,
             ragged=False),
        # one decode step of a serving batch, caches of unequal length
        dict(name="window_decode_batch", op="window", B=64, Hq=32, Hkv=8, d=128, M=1, N=8192, window=4096, n_sink=4,
             ragged=True),
        # whole-prompt prefill at the package's 32K shape, one 128-key sink block
        dict(name="window_prefill_32k", op="window", B=1, Hq=32, Hkv=8, d=128, M=32768, N=32768, window=2048,
             n_sink=128, ragged=False),
        # a chunk of a chunked prefill: odd lengths, three query heads per KV head, d = 64
        dict(name="window_chunk_odd", op="window", B=2, Hq=6, Hkv=2, d=64, M=777, N=5003, window=1000, n_sink=5,
             ragged=True),
        # four requests just behind a short system prompt
        dict(name="prefix_decode_small", op="prefix", B=4, Hq=32, Hkv=8, d=128, M=1, P=2048, N=128, ragged=True),
        # a batch of answers over one 32K document
        dict(name="prefix_decode_batch", op="prefix", B=64, Hq=32, Hkv=8, d=128, M=1, P=32768, N=1024, ragged=True),
        # five drafted tokens per request, odd everything, d = 64
        dict(name="prefix_draft_odd", op="prefix", B=17, Hq=10, Hkv=2, d=64, M=5, P=10007, N=333, ragged=True),
        # a decode step's share of attention added to the running mass
        dict(name="mass_decode", op="mass", B=32, Hq=32, Hkv=8, d=128, M=1, N=8192, window=0, n_sink=0, ragged=True,
             decay=1.0),
        # the mass of every key of a prompt, from the LSE of its attention
        dict(name="mass_prompt_8k", op="mass", B=1, Hq=32, Hkv=8, d=128, M=8192, N=8192, window=0, n_sink=0,
             ragged=False, decay=0.0),
        # the last 61 queries of two long prompts, under a window, d = 64
        dict(name="mass_window_odd", op="mass", B=2, Hq=12, Hkv=4, d=64, M=61, N=20011, window=9001, n_sink=7,
             ragged=True, decay=0.5),
        # a cache of one conversation halved
        dict(name="evict_one", op="evict", B=1, Hkv=8, d=128, N=4096, budget=2048, recent=512, n_sink=4,
             ragged=False),
        # a batch of 32K caches cut to an eighth
        dict(name="evict_batch", op="evict", B=16, Hkv=8, d=128, N=32768, budget=4097, recent=1024, n_sink=128,
             ragged=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    """One case of the listed ranges: batches, head groups, both head
    dimensions, lengths spread over their logarithm, ragged or not."""
    op = rng.choice(["window", "prefix", "mass", "evict"])
    d = rng.choice([64, 128, 128])
    Hkv, G = rng.choice([1, 2, 4, 8, 8]), rng.choice([1, 2, 3, 4, 4, 5, 8])
    same = [work(x) for x in listed() if x["op"] == op]
    cap_flops, cap_bytes = max(w["flops"] for w in same), max(w["bytes"] for w in same)
    c = dict(op=op, B=_log(rng, 1, 64), Hkv=Hkv, d=d, N=_log(rng, 256, 32768), ragged=rng.random() < 0.6)
    if op == "evict":
        budget = _log(rng, c["N"] // 16, c["N"] // 2)
        c.update(budget=budget, recent=rng.randint(0, budget // 2), n_sink=rng.randint(0, min(128, budget // 4)))
    elif op == "prefix":
        N = _log(rng, 16, 2048)
        c.update(Hq=Hkv * G, M=rng.choice([1, 1, _log(rng, 1, 8)]), P=_log(rng, 256, 32768), N=N)
    else:
        N = c["N"]
        c.update(Hq=Hkv * G, M=rng.choice([1, 1, _log(rng, 2, 64), _log(rng, N // 16, N)]), window=_log(rng, 16, N),
                 n_sink=rng.choice([0, rng.randint(1, 128)]))
        if op == "mass":
            c["decay"] = rng.choice([0.0, 0.5, 1.0])
            if rng.random() < 0.5:
                c.update(window=0, n_sink=0)                   # window 0: every earlier key

    def too_much(x):
        w = work(x)
        return (w["flops"] > cap_flops or w["bytes"] > cap_bytes
                or x.get("M", 1) * x.get("Hq", 1) * x["B"] * x["N"] > 4 << 30)

    while too_much(c):
        if c["B"] > 1:
            c["B"] //= 2
        elif c.get("M", 1) > 1:
            c["M"] //= 2
        else:
            c["Hkv"], c["N"] = max(1, c["Hkv"] // 2), max(64, c["N"] // 2)
    return c


def _lens(case):
    """Lengths of the sequences, in ascending order: N, or spread evenly from N/2 to N."""
    B, N = case["B"], case["N"]
    if not case["ragged"]:
        return [N] * B
    lo = max(case.get("M", 1), case.get("budget", 1), N // 2)
    return [lo + (N - lo) * (i + 1) // B for i in range(B)]


def work(case):
    """Every input element read and every output element written once, and the
    visible (query, key) pairs' products."""
    B, Hkv, d, N = case["B"], case["Hkv"], case["d"], case["N"]
    L = _lens(case)
    if case["op"] == "evict":
        row = 2 * d * 2 + 4                                    # K, V and mass of one key
        return {"bytes": Hkv * (sum(L) * 4 + B * case["budget"] * (2 * row - 4 + 4)), "flops": 0}
    Hq, M = case["Hq"], case["M"]
    if case["op"] == "prefix":
        P = case["P"]
        pairs = sum(M * P + M * n - M * (M - 1) // 2 for n in L)
        keys = P + sum(L)
        return {"bytes": 4 * d * Hkv * keys + B * M * Hq * (4 * d + 4), "flops": 4 * d * Hq * pairs}
    W = case["window"] or N
    S = case["n_sink"]
    pairs = keys = 0
    for n in L:
        at = np.arange(n - M, n, dtype=np.int64)               # positions of the query rows
        first = np.maximum(0, at - W + 1)
        pairs += int((at - first + 1 + np.minimum(S, first)).sum())
        keys += int(n - first[0] + min(S, first[0]))
    if case["op"] == "window":
        return {"bytes": 4 * d * Hkv * keys + B * M * Hq * (4 * d + 4), "flops": 4 * d * Hq * pairs}
    read = 4 if case["decay"] else 0
    return {"bytes": Hkv * (2 * d * keys + read * sum(L) + 4 * B * N) + B * M * Hq * (2 * d + 4),
            "flops": 2 * d * Hq * pairs}


# ------------------------------------------------------------------ the inputs
def prepare(case, seed):
    """Queries, keys and values with the clustered keys of long contexts (a few
    keys that draw much of the attention), cache lengths, and for the mass and
    the eviction what earlier steps left."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    B, Hkv, d, N = case["B"], case["Hkv"], case["d"], case["N"]
    order = torch.randperm(B, generator=torch.Generator().manual_seed(seed))
    st = dict(case)
    st["kv_len"] = torch.tensor(_lens(case), dtype=torch.int32)[order].cuda() if case["ragged"] else None
    u = normal(1, Hkv, 1, d)
    u = u / u.norm(dim=-1, keepdim=True)

    def cache(b, n):
        heavy = (torch.rand((b, Hkv, n, 1), generator=g, device="cuda") < 0.01).float()
        k = (normal(b, Hkv, n, d) + 4.0 * heavy * u).to(torch.bfloat16)
        return k, normal(b, Hkv, n, d).to(torch.bfloat16)

    st["K"], st["V"] = cache(B, N)
    if case["op"] == "evict":
        mass = torch.exp(2.0 * normal(B, Hkv, N))
        st["mass"] = torch.where(torch.rand((B, Hkv, N), generator=g, device="cuda") < 0.05, 0.0, mass)
        return st
    Hq, M = case["Hq"], case["M"]
    st["Q"] = (normal(B, Hq, M, d) + 1.5 * u.repeat_interleave(Hq // Hkv, dim=1)).to(torch.bfloat16)
    if case["op"] == "prefix":
        st["Kp"], st["Vp"] = cache(1, case["P"])
    if case["op"] == "mass":
        st["V"] = None
        st["prev"] = torch.exp(normal(B, Hkv, N)) if case["decay"] else None
        if st["prev"] is not None and st["kv_len"] is not None:
            st["prev"] *= torch.arange(N, device="cuda") < st["kv_len"][:, None, None]
        st["lse"] = _plain_lse(st)
    return st


# -------------------------------------------------------------- the plain form
def _band(st):
    """Index of the keys that each chunk of C query rows looks at: the sinks,
    then the chunk's span of the window.  Returns (index [B, chunks, n],
    visible [B, chunks, C, n], C)."""
    B, M, N, S = st["B"], st["M"], st["N"], min(st["n_sink"], st["N"])
    W = min(st["window"] or N, N)
    C = min(M, max(W, 64))
    chunks = -(-M // C)
    dev = st["Q"].device
    length = torch.full((B,), N, device=dev) if st["kv_len"] is None else st["kv_len"].long()
    start = (length - M)[:, None] + C * torch.arange(chunks, device=dev)         # position of each chunk's first row
    n_band = min(W + C - 1, N)
    lo = (start - W + 1).clamp(0, N - n_band)[:, :, None]
    band = lo + torch.arange(n_band, device=dev)
    sink = torch.arange(S, device=dev).expand(B, chunks, S)
    key = torch.cat([sink, band], dim=2)
    is_sink = torch.arange(S + n_band, device=dev) < S
    at = (start[:, :, None] + torch.arange(C, device=dev))[..., None]            # [B, chunks, C, 1]
    j = key[:, :, None, :]
    seen = (j <= at) & torch.where(is_sink, j <= at - W, j > at - W)             # a sink inside the window counts there
    return key, seen, C


def _rows(x, key):
    """x [B, H, N, d] at key [B, chunks, n], in fp32: [B, H, chunks, n, d]."""
    B, H, N, d = x.shape
    flat = key.reshape(B, 1, -1, 1).expand(B, H, -1, d)
    return torch.gather(x, 2, flat).float().reshape(B, H, key.shape[1], key.shape[2], d)


def _plain_scores(st):
    """Scaled logits [B, Hkv, G, chunks, C, n], -inf where a key is not visible."""
    key, seen, C = _band(st)
    B, Hq, M, d = st["Q"].shape
    Hkv, chunks = st["Hkv"], key.shape[1]
    q = torch.nn.functional.pad(st["Q"].float(), (0, 0, 0, chunks * C - M))
    q = q.reshape(B, Hkv, Hq // Hkv, chunks, C, d)
    s = torch.einsum("bhgcqd,bhckd->bhgcqk", q, _rows(st["K"], key))
    s = s.mul_(1.0 / math.sqrt(d)).masked_fill_(~seen[:, None, None], -_INF)
    return s, key


def _softmax_(s):
    """Softmax over the last axis in place, and its log normaliser; a row that sees nothing gives zeros and -inf."""
    m = s.amax(dim=-1, keepdim=True)
    m = torch.where(m == -_INF, 0.0, m)
    total = s.sub_(m).exp_().sum(dim=-1, keepdim=True)
    s.div_(torch.where(total == 0, 1.0, total))
    return s, (m + total.log()).squeeze(-1)


def _plain_lse(st):
    s, _ = _plain_scores(st)
    B, Hq, M, _ = st["Q"].shape
    return torch.logsumexp(s, dim=-1).reshape(B, Hq, -1)[:, :, :M].contiguous()


def _plain_window(st):
    s, key = _plain_scores(st)
    p, lse = _softmax_(s)
    B, Hq, M, d = st["Q"].shape
    o = torch.einsum("bhgcqk,bhckd->bhgcqd", p, _rows(st["V"], key))
    return o.reshape(B, Hq, -1, d)[:, :, :M].to(torch.bfloat16), lse.reshape(B, Hq, -1)[:, :, :M].contiguous()


def _plain_prefix(st):
    B, Hq, M, d = st["Q"].shape
    Hkv, N, P = st["Hkv"], st["N"], st["P"]
    q = st["Q"].float().reshape(B, Hkv, Hq // Hkv, M, d)
    length = torch.full((B,), N, device=q.device) if st["kv_len"] is None else st["kv_len"].long()
    at = (length - M)[:, None, None] + torch.arange(M, device=q.device)[:, None]
    seen = torch.arange(N, device=q.device) <= at
    mine = torch.einsum("bhgqd,bhkd->bhgqk", q, st["K"].float()).masked_fill_(~seen[:, None, None], -_INF)
    s = torch.cat([torch.einsum("bhgqd,hkd->bhgqk", q, st["Kp"][0].float()), mine], dim=-1).mul_(1.0 / math.sqrt(d))
    p, lse = _softmax_(s)
    o = torch.einsum("bhgqk,hkd->bhgqd", p[..., :P], st["Vp"][0].float())
    o += torch.einsum("bhgqk,bhkd->bhgqd", p[..., P:], st["V"].float())
    return o.reshape(B, Hq, M, d).to(torch.bfloat16), lse.reshape(B, Hq, M)


def _plain_mass(st):
    s, key = _plain_scores(st)
    B, Hq, M, _ = st["Q"].shape
    Hkv, N = st["Hkv"], st["N"]
    chunks, C = s.shape[3], s.shape[4]
    lse = torch.nn.functional.pad(st["lse"], (0, chunks * C - M), value=_INF).reshape(B, Hkv, Hq // Hkv, chunks, C, 1)
    part = s.sub_(lse).exp_().sum(dim=(2, 4), dtype=torch.float64)               # [B, Hkv, chunks, n]
    out = torch.zeros((B, Hkv, N), dtype=torch.float64, device=s.device)
    out.scatter_add_(2, key.reshape(B, 1, -1).expand(B, Hkv, -1), part.reshape(B, Hkv, -1))
    if st["prev"] is not None:
        out += st["decay"] * st["prev"].double()
    return out.float()


def _plain_evict(st):
    K, V, mass = st["K"], st["V"], st["mass"]
    B, Hkv, N, d = K.shape
    n = st["budget"]
    length = torch.full((B, 1, 1), N, device=K.device) if st["kv_len"] is None else st["kv_len"].long()[:, None, None]
    j = torch.arange(N, device=K.device)
    score = torch.where(j < length, mass, -_INF)
    always = ((j < st["n_sink"]) | (j >= length - st["recent"])) & (j < length)
    order = score.sort(dim=-1, descending=True, stable=True).indices
    first = torch.gather(always.expand(B, Hkv, N), 2, order).float().sort(dim=-1, descending=True, stable=True).indices
    keep = torch.gather(order, 2, first[..., :n]).sort(dim=-1).values
    rows = keep[..., None].expand(B, Hkv, n, d)
    return (keep.int(), torch.gather(K, 2, rows), torch.gather(V, 2, rows), torch.gather(mass, 2, keep),
            length.reshape(B).clamp(max=n).int())


# ---------------------------------------------------------------- one pass
def run(state):
    st = state
    if own:
        import permuted_block_sparse_b200 as pbs
        if st["op"] == "window":
            return pbs.pbs_attn_window(st["Q"], st["K"], st["V"], st["window"], st["n_sink"], kv_len=st["kv_len"])
        if st["op"] == "prefix":
            return pbs.pbs_attn_prefix(st["Q"], st["Kp"], st["Vp"], st["K"], st["V"], kv_len=st["kv_len"])
        if st["op"] == "mass":
            return pbs.pbs_key_mass(st["Q"], st["K"], st["lse"], mass=st["prev"], decay=st["decay"],
                                    window=st["window"], n_sink=st["n_sink"], kv_len=st["kv_len"])
        return pbs.pbs_evict(st["mass"], st["K"], st["V"], st["budget"], st["recent"], st["n_sink"],
                             kv_len=st["kv_len"])
    return {"window": _plain_window, "prefix": _plain_prefix, "mass": _plain_mass, "evict": _plain_evict}[st["op"]](st)


# ------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """The operators' definitions, one sequence and query head at a time, in fp64."""
    st = prepare(case, seed)
    B, N = case["B"], case["N"]
    length = [N] * B if st["kv_len"] is None else st["kv_len"].tolist()
    if case["op"] == "evict":
        return _exact_evict(st, length)
    Hq, Hkv, M, d = case["Hq"], case["Hkv"], case["M"], case["d"]
    G = Hq // Hkv
    if case["op"] != "mass":
        out = torch.empty((B, Hq, M, d), dtype=torch.float64, device="cuda")
        lse = torch.empty((B, Hq, M), dtype=torch.float64, device="cuda")
    total = torch.zeros((B, Hkv, N), dtype=torch.float64, device="cuda")
    if B * Hq * M * N > 6e10:
        return None
    step = max(1, (1 << 28) // (N + case.get("P", 0)))
    for b in range(B):
        for h in range(Hq):
            k = st["K"][b, h // G, :length[b]].double()
            if case["op"] == "prefix":
                k = torch.cat([st["Kp"][0, h // G].double(), k])
                v = torch.cat([st["Vp"][0, h // G].double(), st["V"][b, h // G, :length[b]].double()])
            elif case["op"] == "window":
                v = st["V"][b, h // G, :length[b]].double()
            j = torch.arange(k.shape[0], device="cuda")
            for r in range(0, M, step):
                rows = torch.arange(r, min(M, r + step), device="cuda")
                at = (k.shape[0] - M + rows)[:, None]
                hidden = j > at
                if case.get("window"):
                    hidden |= (at - j >= case["window"]) & (j >= case["n_sink"])
                x = st["Q"][b, h, rows].double() @ k.T / math.sqrt(d)
                x[hidden] = -_INF
                if case["op"] == "mass":
                    total[b, h // G, :length[b]] += torch.exp(x - st["lse"][b, h, rows].double()[:, None]).sum(0)
                else:
                    lse[b, h, rows] = torch.logsumexp(x, 1)
                    out[b, h, rows] = torch.softmax(x, 1) @ v
    if case["op"] != "mass":
        return out, lse
    return total if st["prev"] is None else total + case["decay"] * st["prev"].double()


def _exact_evict(st, length):
    mass = st["mass"].cpu().numpy()
    B, Hkv, N = mass.shape
    keep = np.empty((B, Hkv, st["budget"]), dtype=np.int64)
    for b in range(B):
        j = np.arange(length[b])
        spare = ~((j < st["n_sink"]) | (j >= length[b] - st["recent"]))
        for h in range(Hkv):
            keep[b, h] = np.sort(np.lexsort((j, -mass[b, h, :length[b]].astype(np.float64), spare))[:st["budget"]])
    at = torch.from_numpy(keep).cuda()
    rows = at[..., None].expand(-1, -1, -1, st["d"])
    return (at.int(), torch.gather(st["K"].double(), 2, rows), torch.gather(st["V"].double(), 2, rows),
            torch.gather(st["mass"].double(), 2, at),
            torch.tensor([min(n, st["budget"]) for n in length], dtype=torch.int32))
