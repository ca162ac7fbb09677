"""The serving operators around the quantized key cache: what is measured, in plain form and as the library's calls.

Four operators: attention over packed prompts, decode attention over a shared
quantized prefix, the accumulation of attention weights, and the eviction of
cache rows by them.  ``own`` selects the library's calls.
"""
import functools
import math
import random

import numpy as np
import torch

own = False

_TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_DEV = "cuda"


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # a handful of very short prompts, one of a single token: launch latency counts
        _prompt("prompt_short", "bf16", 128, 8, 4, 4, 1, 40, 0, 11),
        # a ragged batch of ordinary prompts, some continuing earlier chunks
        _prompt("prompt_packed", "bf16", 128, 8, 4, 12, 1, 1500, 700, 12),
        # one long document
        _prompt("prompt_long", "bf16", 128, 8, 4, 1, 8192, 8192, 0, 13),
        # the wide heads of the 16-bit float workloads
        _prompt("prompt_wide_f16", "f16", 256, 8, 2, 3, 500, 2300, 0, 14),
        # full precision
        _prompt("prompt_f32", "f32", 64, 4, 2, 5, 30, 900, 100, 15),
        # two short conversations on a short system prompt
        _shared("shared_small", "f16", 128, 4, 8, 4, 2, 300, 40, 21),
        # multi-head keys at three bits, a batch of eight on one document
        _shared("shared_mha_b3", "bf16", 128, 3, 32, 1, 8, 32768, 600, 22),
        # 32 conversations on a document of 128k tokens, four queries to a KV head
        _shared("shared_128k", "bf16", 128, 4, 8, 4, 32, 131072, 500, 23),
        # the weights of one decode step: a short cache, and a batch of four at 128k tokens
        _weights("weights_small", 8, 4, 1100, 31),
        _weights("weights_128k", 32, 4, 131072, 32),
        # a sliding budget that sheds a few rows, and the cut of a long prompt's cache
        _evict("evict_few", "bf16", 128, 4, 8, 1100, 1024, 100, 41),
        _evict("evict_prompt", "bf16", 128, 4, 32, 32768, 8192, 512, 42),
    ]


def _prompt(name, dtype, d, heads, group, batch, shortest, longest, past, lens_seed):
    return {"name": name, "op": "prompt", "dtype": dtype, "d": d, "heads": heads, "group": group, "batch": batch,
            "shortest": shortest, "longest": longest, "past": past, "lens_seed": lens_seed}


def _shared(name, dtype, d, b, heads, group, batch, prefix, longest, lens_seed):
    return {"name": name, "op": "shared", "dtype": dtype, "d": d, "b": b, "heads": heads, "group": group,
            "batch": batch, "prefix": prefix, "longest": longest, "lens_seed": lens_seed}


def _weights(name, heads, group, n, lens_seed):
    return {"name": name, "op": "weights", "heads": heads, "group": group, "n": n, "lens_seed": lens_seed}


def _evict(name, dtype, d, b, heads, n, keep, recent, lens_seed):
    return {"name": name, "op": "evict", "dtype": dtype, "d": d, "b": b, "heads": heads, "n": n, "keep": keep,
            "recent": recent, "lens_seed": lens_seed}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    seed = rng.randrange(1 << 30)
    op = rng.choice(["prompt", "prompt", "shared", "shared", "weights", "evict"])
    if op == "prompt":
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        d = rng.choice([64, 128, 256]) if dtype != "f32" else rng.choice([64, 128])
        longest = _log(rng, 2, 4096 if dtype != "f32" else 1024)
        case = _prompt("", dtype, d, rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4]), rng.randint(1, 6),
                       max(1, longest // rng.choice([1, 2, 8])), longest, rng.choice([0, 0, longest // 2]), seed)
    elif op == "shared":
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        prefix = _log(rng, 50, 60000 if dtype != "f32" else 6000)
        case = _shared("", dtype, rng.choice([64, 128]), rng.choice([2, 3, 4]), rng.choice([2, 4, 8]),
                       rng.choice([1, 3, 4, 8]), _log(rng, 1, 40), prefix, _log(rng, 2, 1500), seed)
    elif op == "weights":
        case = _weights("", rng.choice([1, 5, 8, 32]), rng.choice([1, 2, 4, 7]), _log(rng, 30, 131072), seed)
    else:
        n = _log(rng, 60, 40000)
        keep = max(2, int(n * rng.uniform(0.1, 0.95)))
        case = _evict("", rng.choice(["bf16", "f16", "f32"]), rng.choice([64, 128, 256]), rng.choice([2, 3, 4]),
                      rng.choice([1, 4, 8, 32]), n, keep, int(keep * rng.uniform(0, 0.5)), seed)
    del case["name"]
    return case


def _prompt_lens(case):
    r = random.Random(case["lens_seed"])
    lens_q = [r.randint(case["shortest"], case["longest"]) for _ in range(case["batch"])]
    if case["batch"] > 1:
        lens_q[1] = 1
    lens_k = [n + (r.randint(0, case["past"]) if case["past"] else 0) for n in lens_q]
    return lens_q, lens_k


def _shared_lens(case):
    """Own lengths of the sequences; one of several has none yet."""
    r = random.Random(case["lens_seed"])
    lens = [r.randint(0, case["longest"]) for _ in range(case["batch"])]
    if len(lens) > 1:
        lens[1] = 0
    return lens


def _head_lens(case):
    """Rows in use per KV head: most caches full, one head in four shorter."""
    r = random.Random(case["lens_seed"])
    n = case["n"]
    return [n if r.random() < 0.75 else r.randint((n + 1) // 2, n) for _ in range(case["heads"])]


def _size(dtype):
    return 4 if dtype == "f32" else 2


def work(case):
    if case["op"] == "prompt":
        lens_q, lens_k = _prompt_lens(case)
        hq, d, e = case["heads"] * case["group"], case["d"], _size(case["dtype"])
        pairs = sum(nq * (nk - nq) + nq * (nq + 1) // 2 for nq, nk in zip(lens_q, lens_k))
        return {"bytes": sum(lens_q) * hq * (2 * d * e + 4) + sum(lens_k) * case["heads"] * 2 * d * e,
                "flops": 4 * d * hq * pairs}
    if case["op"] == "shared":
        d, h, e = case["d"], case["heads"], _size(case["dtype"])
        row = d * case["b"] // 8 + 4 + d * e
        own_rows = sum(_shared_lens(case))
        hq = h * case["group"]
        return {"bytes": h * (case["prefix"] + own_rows) * row + case["batch"] * hq * (2 * d * e + 4),
                "flops": 4 * d * hq * (case["batch"] * case["prefix"] + own_rows)}
    lens = _head_lens(case)
    if case["op"] == "weights":
        return {"bytes": sum(lens) * 4 * (case["group"] + 2), "flops": 4 * case["group"] * sum(lens)}
    row = case["d"] * case["b"] // 8 + 8 + case["d"] * _size(case["dtype"])
    kept = sum(min(n, case["keep"]) for n in lens)
    return {"bytes": 4 * sum(lens) + kept * (2 * row + 4), "flops": 0}


# ---- the quantized cache, from its definition --------------------------------

@functools.lru_cache(maxsize=None)
def _centroids(b):
    """Lloyd-Max centroids of N(0, 1), ascending, in 64 bits."""
    m = 1 << (b - 1)
    p = [3.0 * (i + 0.5) / m for i in range(m)]
    phi = lambda x: math.exp(-0.5 * x * x) / math.sqrt(2 * math.pi) if x < 1e9 else 0.0  # noqa: E731
    tail = lambda x: 0.5 * math.erfc(x / math.sqrt(2)) if x < 1e9 else 0.0  # noqa: E731
    for _ in range(20000):
        tau = [0.0] + [0.5 * (p[i] + p[i + 1]) for i in range(m - 1)] + [1e10]
        q = [(phi(tau[i]) - phi(tau[i + 1])) / (tail(tau[i]) - tail(tau[i + 1])) for i in range(m)]
        moved = max(abs(x - y) for x, y in zip(p, q))
        p = q
        if moved < 1e-15:
            break
    return tuple([-x for x in reversed(p)] + p)


def _codebook(d, b, device):
    c = (np.array(_centroids(b)) / math.sqrt(d)).astype(np.float32)
    return torch.from_numpy(c).to(device)


def _hadamard(d, dtype, device):
    i = torch.arange(d, device=device)
    x = i[:, None] & i[None, :]
    odd = torch.zeros_like(x)
    for s in range(10):
        odd ^= (x >> s) & 1
    return (1 - 2 * odd).to(dtype)


def _write_cache(g, heads, n, d, b, signs):
    """Packed codes and norms of seeded keys: rows of N(0, 1) times LogNormal(0, 0.5)."""
    idx = torch.zeros((heads, n, d * b // 8), dtype=torch.uint8, device=_DEV)
    norms = torch.zeros((heads, n), device=_DEV)
    if not n:
        return idx, norms
    c = _codebook(d, b, _DEV)
    edges = (c[1:] + c[:-1]) / 2
    rot = _hadamard(d, torch.float32, _DEV) * signs.float()[:, None] / math.sqrt(d)
    shift = b * torch.arange(8, device=_DEV, dtype=torch.int32)
    step = max(1, (1 << 18) // n)
    for h in range(0, heads, step):
        k = torch.randn((min(step, heads - h), n, d), generator=g, device=_DEV)
        k *= torch.exp(0.5 * torch.randn((k.shape[0], n, 1), generator=g, device=_DEV))
        r = k.norm(dim=2)
        code = torch.bucketize((k @ rot) / r[..., None], edges).to(torch.int32)
        word = (code.view(k.shape[0], n, d // 8, 8) << shift).sum(-1, dtype=torch.int32)
        byte = torch.stack([(word >> (8 * i)) & 255 for i in range(b)], dim=-1)
        idx[h:h + step] = byte.reshape(k.shape[0], n, -1).to(torch.uint8)
        norms[h:h + step] = r
    return idx, norms


def _read_cache(idx, b, centroids):
    """Centroids of packed rows (..., P) as (..., d): eight codes sit in every b bytes."""
    by = idx.reshape(idx.shape[:-1] + (idx.shape[-1] // b, b)).to(torch.int32)
    word = (by << (8 * torch.arange(b, device=idx.device, dtype=torch.int32))).sum(-1, dtype=torch.int32)
    shift = b * torch.arange(8, device=idx.device, dtype=torch.int32)
    code = (word[..., None] >> shift) & ((1 << b) - 1)
    return centroids[code.reshape(idx.shape[:-1] + (8 * word.shape[-1],))]


# ---- inputs ------------------------------------------------------------------

def _starts(lens):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)


def prepare(case, seed):
    g = torch.Generator(device=_DEV).manual_seed(1_000_003 * (seed % (1 << 40)) + 17)
    state = dict(case)
    if case["op"] == "prompt":
        lens_q, lens_k = _prompt_lens(case)
        t, h, d = _TYPES[case["dtype"]], case["heads"], case["d"]
        nq, nk = sum(lens_q), sum(lens_k)
        # token-major projections seen head by head, as a model's linear layers leave them
        state["q"] = torch.randn((nq, h * case["group"], d), generator=g, device=_DEV).to(t).transpose(0, 1)
        state["K"] = (1.5 * torch.randn((nk, h, d), generator=g, device=_DEV)).to(t).transpose(0, 1)
        state["V"] = torch.randn((nk, h, d), generator=g, device=_DEV).to(t).transpose(0, 1)
        state["cu_q"], state["cu_k"] = _starts(lens_q).to(_DEV), _starts(lens_k).to(_DEV)
        state["longest_q"], state["longest_k"] = max(lens_q), max(lens_k)
        return state
    if case["op"] == "shared":
        t, h, d, b, n = _TYPES[case["dtype"]], case["heads"], case["d"], case["b"], case["prefix"]
        lens = _shared_lens(case)
        cap = (max(lens) + 64) // 16 * 16
        signs = torch.randint(0, 2, (d,), generator=g, device=_DEV, dtype=torch.int8) * 2 - 1
        state["signs"] = signs
        state["prefix_idx"], state["prefix_norms"] = _write_cache(g, h, n, d, b, signs)
        state["prefix_V"] = torch.randn((h, n, d), generator=g, device=_DEV).to(t)
        state["idx"], state["norms"] = _write_cache(g, case["batch"] * h, cap, d, b, signs)
        state["own_V"] = torch.randn((case["batch"] * h, cap, d), generator=g, device=_DEV).to(t)
        state["lengths"] = torch.tensor(lens, dtype=torch.int32, device=_DEV)
        state["q"] = torch.randn((case["batch"] * h * case["group"], d), generator=g, device=_DEV).to(t)
        return state
    lens = _head_lens(case)
    state["lengths"] = torch.tensor(lens, dtype=torch.int32, device=_DEV)
    h, n = case["heads"], case["n"]
    if case["op"] == "weights":
        state["scores"] = 1.5 * torch.randn((h * case["group"], n), generator=g, device=_DEV)
        state["weights"] = torch.rand((h, n), generator=g, device=_DEV)
        return state
    t, d, b, keep = _TYPES[case["dtype"]], case["d"], case["b"], case["keep"]
    state["idx"] = torch.randint(0, 256, (h, n, d * b // 8), generator=g, device=_DEV, dtype=torch.uint8)
    state["norms"] = torch.rand((h, n), generator=g, device=_DEV) + 0.5
    state["V"] = torch.randn((h, n, d), generator=g, device=_DEV).to(t)
    # heavy-tailed sums, coarse enough that some are equal
    heavy = torch.exp(1.5 * torch.randn((h, n), generator=g, device=_DEV))
    state["weights"] = torch.round(heavy * 1024) / 1024
    state["out"] = (torch.zeros((h, keep, d * b // 8), dtype=torch.uint8, device=_DEV),
                    torch.zeros((h, keep), device=_DEV), torch.zeros((h, keep, d), dtype=t, device=_DEV),
                    torch.zeros((h, keep), device=_DEV),
                    torch.full((h, keep), -1, dtype=torch.int32, device=_DEV),
                    torch.zeros(h, dtype=torch.int32, device=_DEV))
    return state


# ---- the operators -----------------------------------------------------------

def run(state):
    if own:
        return _run_own(state)
    return {"prompt": _plain_prompt, "shared": _plain_shared, "weights": _plain_weights,
            "evict": _plain_evict}[state["op"]](state)


def _run_own(s):
    from lut_attention_b200 import axr

    if s["op"] == "prompt":
        out, lse = axr.axr_prompt_attention(s["q"], s["K"], s["V"], s["cu_q"], s["cu_k"])
        return {"out": out, "lse": lse}
    if s["op"] == "shared":
        out, lse = axr.axr_attention_shared(s["q"], s["prefix_idx"], s["prefix_norms"], s["prefix_V"], s["idx"],
                                            s["norms"], s["own_V"], s["lengths"], s["group"], s["b"], s["signs"])
        return {"out": out, "lse": lse}
    if s["op"] == "weights":
        return axr.axr_accumulate_weights(s["scores"], s["weights"], s["group"], lengths=s["lengths"])
    return axr.axr_evict(s["idx"], s["norms"], s["V"], s["weights"], s["lengths"], s["keep"], s["recent"],
                         out=s["out"])


def _softmax(scores):
    """Softmax along the last axis and its log sum; rows without a visible key give 0 and -inf."""
    m = scores.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(scores - m)
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total == 0, torch.ones_like(total), total), (m + torch.log(total)).squeeze(-1)


def _plain_prompt(s):
    q, K, V, group = s["q"], s["K"], s["V"], s["group"]
    dev = q.device
    first_q, first_k = s["cu_q"].long(), s["cu_k"].long()
    len_q, len_k = first_q.diff(), first_k.diff()
    i, j = torch.arange(s["longest_q"], device=dev), torch.arange(s["longest_k"], device=dev)
    at_q = (first_q[:-1, None] + i).clamp(max=q.shape[1] - 1)               # (batch, longest_q)
    at_k = (first_k[:-1, None] + j).clamp(max=K.shape[1] - 1)
    heads, d = K.shape[0], K.shape[2]
    qp = q.float()[:, at_q].view(heads, group, len(at_q), -1, d)
    kp, vp = K.float()[:, at_k][:, None], V.float()[:, at_k][:, None]
    scores = qp @ kp.transpose(-1, -2) / math.sqrt(d)
    last = (len_k - len_q)[:, None] + i                                     # last key a query sees
    seen = (j <= last[..., None]) & (j < len_k[:, None, None])
    p, lse = _softmax(scores.masked_fill_(~seen, float("-inf")))
    del scores
    out = p @ vp
    rows = (i < len_q[:, None]).nonzero(as_tuple=True)                      # in packed order
    out = out.view(heads * group, len(at_q), -1, d)[:, rows[0], rows[1]]
    return {"out": out.to(q.dtype), "lse": lse.view(heads * group, len(at_q), -1)[:, rows[0], rows[1]]}


def _plain_shared(s):
    q, group, b = s["q"], s["group"], s["b"]
    heads, n, d = s["prefix_V"].shape
    batch = s["lengths"].shape[0]
    c = _codebook(d, b, q.device)
    rot = (q.float() * s["signs"].float()) @ _hadamard(d, torch.float32, q.device) / d
    rot = rot.view(batch, heads, group, d)
    k_pre = _read_cache(s["prefix_idx"], b, c) * s["prefix_norms"][..., None]
    k_own = _read_cache(s["idx"], b, c) * s["norms"][..., None]
    by_head = rot.transpose(0, 1).reshape(heads, batch * group, d)
    s_pre = (by_head @ k_pre.transpose(-1, -2)).view(heads, batch, group, n).transpose(0, 1)
    s_own = rot @ k_own.view(batch, heads, -1, d).transpose(-1, -2)
    cap = s_own.shape[-1]
    seen = torch.arange(cap, device=q.device) < s["lengths"][:, None]
    s_own = s_own.masked_fill(~seen[:, None, None], float("-inf"))
    p, lse = _softmax(torch.cat([s_pre, s_own], dim=-1))
    p_pre = p[..., :n].transpose(0, 1).reshape(heads, batch * group, n)
    out = (p_pre @ s["prefix_V"].float()).view(heads, batch, group, d).transpose(0, 1)
    out = out + p[..., n:] @ s["own_V"].float().view(batch, heads, cap, d)
    return {"out": out.reshape(-1, d).to(s["own_V"].dtype), "lse": lse.reshape(-1)}


def _plain_weights(s):
    heads, n = s["weights"].shape
    seen = torch.arange(n, device=s["scores"].device) < s["lengths"][:, None]
    scores = s["scores"].view(heads, -1, n).masked_fill(~seen[:, None], float("-inf"))
    s["weights"] += _softmax(scores)[0].sum(1)
    return s["weights"]


def _plain_evict(s):
    w, lens, keep, recent = s["weights"], s["lengths"].long(), s["keep"], s["recent"]
    heads, n = w.shape
    t = torch.arange(n, device=w.device)
    rank = w.masked_fill(t >= (lens - recent)[:, None], float("inf"))
    rank = rank.masked_fill(t >= lens[:, None], float("-inf"))
    order = torch.sort(rank, dim=1, descending=True, stable=True)[1][:, :keep]
    left = lens.clamp(max=keep)
    live = torch.arange(keep, device=w.device) < left[:, None]
    kept = torch.sort(torch.where(live, order, n), dim=1)[0]
    at = kept.clamp(max=n - 1)
    h = torch.arange(heads, device=w.device)[:, None]
    out = s["out"]
    for to, src in zip(out[:4], (s["idx"], s["norms"], s["V"], w)):
        got = src[h, at]
        to.copy_(torch.where(live.view(live.shape + (1,) * (got.dim() - 2)), got, to))
    out[4].copy_(torch.where(live, kept, -1))
    out[5].copy_(left)
    return out


# ---- the same in 64 bits -----------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"prompt": _exact_prompt, "shared": _exact_shared, "weights": _exact_weights,
            "evict": _exact_evict}[case["op"]](s)


def _attend(q, k, v, seen=None):
    """Rows q (r, d) over keys k (n, d) and values v in 64 bits: outputs and log sums."""
    if k.shape[0] == 0:
        return torch.zeros_like(q), torch.full((q.shape[0],), -math.inf, dtype=torch.float64, device=q.device)
    x = q @ k.T
    if seen is not None:
        x = torch.where(seen, x, -math.inf)
    lse = torch.logsumexp(x, dim=1)
    w = torch.exp(x - torch.where(torch.isinf(lse), 0.0, lse)[:, None])
    return w @ v, lse


def _exact_prompt(s):
    hq, nq, d = s["q"].shape
    out = torch.zeros((hq, nq, d), dtype=torch.float64, device=_DEV)
    lse = torch.zeros((hq, nq), dtype=torch.float64, device=_DEV)
    cu_q, cu_k = s["cu_q"].tolist(), s["cu_k"].tolist()
    for a, z, ka, kz in zip(cu_q, cu_q[1:], cu_k, cu_k[1:]):
        last = torch.arange(z - a, device=_DEV) + (kz - ka) - (z - a)
        seen = torch.arange(kz - ka, device=_DEV)[None] <= last[:, None]
        for h in range(hq):
            kv = h // s["group"]
            out[h, a:z], lse[h, a:z] = _attend(s["q"][h, a:z].double() / math.sqrt(d), s["K"][kv, ka:kz].double(),
                                               s["V"][kv, ka:kz].double(), seen)
    return {"out": out, "lse": lse}


def _exact_shared(s):
    heads, n, d = s["prefix_V"].shape
    group, batch = s["group"], s["lengths"].shape[0]
    c = _codebook(d, s["b"], _DEV).double()
    q = s["q"].double() * s["signs"].double()
    half = 1                                             # butterflies: the transform without its matrix
    while half < d:
        x = q.view(-1, d // (2 * half), 2, half)
        q = torch.stack([x[:, :, 0] + x[:, :, 1], x[:, :, 0] - x[:, :, 1]], dim=2).reshape(-1, d)
        half *= 2
    q = (q / d).view(batch, heads, group, d)
    out = torch.zeros((batch, heads, group, d), dtype=torch.float64, device=_DEV)
    lse = torch.zeros((batch, heads, group), dtype=torch.float64, device=_DEV)
    idx, norms = s["idx"].view(batch, heads, -1, s["idx"].shape[-1]), s["norms"].view(batch, heads, -1)
    V = s["own_V"].view(batch, heads, -1, d)
    for h in range(heads):
        k = _read_cache(s["prefix_idx"][h], s["b"], c) * s["prefix_norms"][h].double()[:, None]
        o1, l1 = _attend(q[:, h].reshape(-1, d), k, s["prefix_V"][h].double())
        for i, m in enumerate(s["lengths"].tolist()):
            k = _read_cache(idx[i, h, :m], s["b"], c) * norms[i, h, :m].double()[:, None]
            o2, l2 = _attend(q[i, h], k, V[i, h, :m].double())
            la, oa = l1[i * group:(i + 1) * group], o1[i * group:(i + 1) * group]
            both = torch.logaddexp(la, l2)
            out[i, h] = oa * torch.exp(la - both)[:, None] + o2 * torch.exp(l2 - both)[:, None]
            lse[i, h] = both
    return {"out": out.view(-1, d), "lse": lse.view(-1)}


def _exact_weights(s):
    w = s["weights"].double()
    for h, m in enumerate(s["lengths"].tolist()):
        for g in range(s["group"]):
            x = s["scores"][h * s["group"] + g, :m].double()
            w[h, :m] += torch.exp(x - torch.logsumexp(x, 0))
    return w


def _exact_evict(s):
    """What is copied, by a search on the host for the rows that stay."""
    out = [x.clone() for x in s["out"]]
    for h, m in enumerate(s["lengths"].tolist()):
        w = s["weights"][h, :m].cpu().numpy()
        old = max(0, m - s["recent"])
        stay = np.arange(m)
        if m > s["keep"]:
            by = np.lexsort((np.arange(old), -w[:old]))[:s["keep"] - (m - old)]
            stay = np.sort(np.concatenate([by, np.arange(old, m)]))
        at = torch.from_numpy(stay).to(_DEV)
        for to, src in zip(out[:4], (s["idx"], s["norms"], s["V"], s["weights"])):
            to[h, :len(stay)] = src[h, at]
        out[4][h, :len(stay)] = at.int()
        out[5][h] = len(stay)
    return (None, out[1].double(), out[2].double(), out[3].double(), out[4], out[5])
