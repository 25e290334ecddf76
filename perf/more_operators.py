"""Attention of many queries over the device pages, as measured cases.

Three operators beside those of ``operators.py``:

  query    several query tokens per sequence over its pages: cross attention to
           an encoder's states of another length, or (causal) a chunk of a
           prompt over what is cached and itself (``query_attention``);
  prefix   one new token per sequence, over a prefix that a group of sequences
           shares, read once for the group, and over the sequence's own pages
           (``prefix_attention``);
  merge    results over parts of the tokens, joined by their log-sums
           (``merge_attention``).

``own`` selects the library's calls; otherwise ``run`` computes the same from
elementary torch operations in 32 bits.  ``exact`` computes it in 64 bits, one
sequence and kv head at a time, from the definitions.
"""
from __future__ import annotations

import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
DEV = "cuda"


# ---- cases ----------------------------------------------------------------------

def _query(name, batch, min_q, max_q, min_kv, max_kv, q_heads, kv_heads, dim, page, causal=False, window=0,
           dtype="bf16", cache="same", empty=False, padded=0):
    return {"name": name, "op": "query", "batch": batch, "min_q": min_q, "max_q": max_q, "min_kv": min_kv,
            "max_kv": max_kv, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "page": page, "causal": causal,
            "window": window, "dtype": dtype, "cache": cache, "empty": empty, "padded": padded}


def _prefix(name, batch, groups, min_prefix, max_prefix, min_own, max_own, q_heads, kv_heads, dim, page,
            dtype="bf16", cache="same", empty=False, loose=0):
    return {"name": name, "op": "prefix", "batch": batch, "groups": groups, "min_prefix": min_prefix,
            "max_prefix": max_prefix, "min_own": min_own, "max_own": max_own, "q_heads": q_heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype, "cache": cache, "empty": empty,
            "loose": loose}


def _merge(name, tokens, parts, q_heads, dim, dtype="bf16", empty=False):
    return {"name": name, "op": "merge", "tokens": tokens, "parts": parts, "q_heads": q_heads, "dim": dim,
            "dtype": dtype, "empty": empty}


def listed():
    return [
        # one decoder token against one encoded input: latency
        _query("cross_1", 1, 1, 1, 1500, 1500, 16, 16, 64, 64, dtype="fp16"),
        # decoder prompts of a batch, each against its own encoded input; one input is not there yet
        _query("cross_32_ragged", 32, 1, 96, 200, 3000, 16, 16, 64, 16, dtype="fp16", empty=True),
        # long queries against long encoded inputs: compute
        _query("cross_8x2k", 8, 2048, 2048, 4001, 4001, 32, 8, 128, 64),
        # one prefill of a long prompt, nothing cached before it
        _query("chunk_8k", 1, 8191, 8191, 8191, 8191, 32, 8, 128, 64, causal=True),
        # a turn's new tokens after a long cached conversation
        _query("chunk_2k_at_32k", 1, 2048, 2048, 32768, 32768, 32, 8, 128, 64, causal=True),
        # chunks of several prompts in one batch, an 8-bit cache, a sliding window
        _query("chunks_e4m3_window", 6, 100, 1000, 1000, 12000, 32, 8, 128, 16, causal=True, window=4000, dtype="fp16",
               cache="e4m3", padded=40),
        # large heads
        _query("chunk_256", 2, 1500, 1500, 6001, 6001, 16, 4, 256, 128, causal=True),
        # a few samples of one request: latency
        _prefix("prefix_4x2k", 4, 1, 2000, 2000, 1, 64, 32, 8, 128, 64),
        # many requests on one long document
        _prefix("prefix_64x32k", 64, 1, 32768, 32768, 33, 1024, 32, 8, 128, 16),
        # several system prompts in one batch, an 8-bit cache, some requests that share nothing
        _prefix("prefix_96_groups_e4m3", 96, 6, 1000, 9000, 10, 500, 32, 8, 128, 16, dtype="fp16", cache="e4m3",
                empty=True, loose=5),
        # a decode batch's two parts
        _merge("merge_2x64", 64, 2, 32, 128),
        # a prefill chunk over a tree of prefixes, some of its levels empty
        _merge("merge_4x8k", 8191, 4, 32, 128, empty=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("cross", "chunk", "prefix", "prefix", "merge"))
    dtype = rng.choice(("bf16", "fp16"))
    page = rng.choice((1, 5, 16, 64, 128))
    dim = rng.choice((64, 80, 96, 128, 192, 256))
    kv = rng.choice((1, 2, 4, 8))
    cache = rng.choice(("same", "same", "e4m3"))
    if op == "merge":
        heads = rng.choice((1, 4, 7, 16, 32))
        c = _merge("", _log(rng, 1, 8000), rng.randint(1, 8), heads, dim, dtype, rng.random() < 0.5)
    elif op == "prefix":
        group = rng.choice((1, 2, 3, 4, 6, 8, 12, 16))
        longest = _log(rng, 1, 40000)
        batch = _log(rng, 1, 256)
        groups = rng.randint(1, max(1, min(batch, 60000 // longest, 12)))
        most = _log(rng, 1, max(1, min(2000, 100000 // batch)))
        # queries times tokens of the prefixes, as in the listed cases
        while batch * longest * kv * group > 64 * 32768 * 32:
            batch = max(1, batch // 2)
            groups = min(groups, batch)
        c = _prefix("", batch, groups, max(1, longest // rng.choice((1, 3, 20))), longest,
                    max(1, most // rng.choice((1, 4, 30))), most, kv * group, kv, dim, page, dtype, cache,
                    rng.random() < 0.3, rng.randint(0, batch // 8))
    else:
        group = rng.choice((1, 1, 2, 3, 4, 7, 8))
        causal = op == "chunk"
        longest = _log(rng, 1, 40000)
        most = _log(rng, 1, min(longest, 4096) if causal else 4096)
        batch = _log(rng, 1, 64)
        while batch > 1 and batch * most * longest * kv * group * dim > 2048 * 32768 * 32 * 128 // 2 or \
                batch > 1 and batch * longest > 200000:
            batch //= 2
        while batch * most * longest * kv * group * dim > 2048 * 32768 * 32 * 128:
            most = max(1, most // 2)
            longest = max(most, longest // 2)
        lo_q = max(1, most // rng.choice((1, 3, 30)))
        lo_kv = max(most if causal else 1, longest // rng.choice((1, 2, 10)))
        window = rng.choice((0, 0, rng.randint(1, longest))) if causal else 0
        c = _query("", batch, lo_q, most, lo_kv, longest, kv * group, kv, dim, page, causal, window, dtype, cache,
                   rng.random() < 0.3, rng.randint(0, 20))
    del c["name"]
    return c


# ---- sizes that follow from a case alone -------------------------------------------

def _spread(n, lo, hi, shift=0.5):
    """n sizes spread evenly over the logarithm between lo and hi, in mixed order."""
    at = [(i * 0.6180339887498949 + shift) % 1.0 for i in range(n)]
    sizes = [int(round(math.exp(math.log(lo) + (math.log(hi) - math.log(lo)) * x))) for x in at]
    sizes[0] = hi
    return sizes


def _query_sizes(case):
    q = _spread(case["batch"], case["min_q"], case["max_q"], 0.25)
    kv = _spread(case["batch"], case["min_kv"], case["max_kv"])
    if case["empty"] and case["batch"] > 1:
        kv[-1] = 0
    return q, kv


def _prefix_sizes(case):
    """(sequences of each group, prefix lengths, own lengths); the last `loose`
    sequences belong to no group."""
    n, g = case["batch"] - case["loose"], case["groups"]
    if n < g:
        g = max(1, n)
    cut = [n * i // g for i in range(g + 1)]
    members = [cut[i + 1] - cut[i] for i in range(g)] + [0] * (case["groups"] - g)
    prefix = _spread(case["groups"], case["min_prefix"], case["max_prefix"])
    mine = _spread(case["batch"], case["min_own"], case["max_own"])
    if case["empty"]:
        mine[-1] = 0
        if case["groups"] > 1:
            prefix[-1] = 0
    return members, prefix, mine


def _starts(sizes):
    at = [0]
    for n in sizes:
        at.append(at[-1] + n)
    return at


def _elem(case):
    return 1 if case["cache"] == "e4m3" else 2


# ---- inputs ------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _tables(case, lens, g):
    """One page table per list of lengths, of pages that nothing else has, from one
    shuffled pool; -1 behind each last page.  Returns the tables and the pool's pages."""
    p = case["page"]
    counts = [[-(-n // p) for n in some] for some in lens]
    total = sum(map(sum, counts))
    spare = max(1, total // 16)
    perm = torch.randperm(total + spare, generator=g, device=DEV).to(torch.int32)
    tables, at = [], 0
    for some in counts:
        width = max(1, max(some))
        n = torch.tensor(some, device=DEV)
        first = at + torch.cumsum(n, 0) - n
        col = torch.arange(width, device=DEV)
        index = (first[:, None] + col[None, :]).clamp_(max=total + spare - 1)
        tables.append(torch.where(col[None, :] < n[:, None], perm[index], -1).to(torch.int32))
        at += sum(some)
    return tables, total + spare


def _cache(case, pages, g):
    dt = DT[case["dtype"]]
    bufs = [torch.randn((pages * case["page"], case["kv_heads"] * case["dim"]), generator=g, device=DEV, dtype=dt)
            for _ in range(2)]
    if case["cache"] != "e4m3":
        return bufs, 1.0, 1.0
    scales = (0.0625, 0.03125)
    return [(x.float() / sc).to(torch.float8_e4m3fn) for x, sc in zip(bufs, scales)], *scales


def _int32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _prepare_query(case, seed):
    g = _generator(seed)
    dt, d, hq = DT[case["dtype"]], case["dim"], case["q_heads"]
    q_lens, kv_lens = _query_sizes(case)
    (table,), pages = _tables(case, [kv_lens], g)
    bufs, ks, vs = _cache(case, pages, g)
    n = sum(q_lens) + case["padded"]      # rows that only fill up the batch: left as they are
    return {"q": (2 * torch.randn((n, hq, d), generator=g, device=DEV)).to(dt), "table": table, "bufs": bufs,
            "pages": pages, "k_scale": ks, "v_scale": vs, "starts": _int32(_starts(q_lens)), "lens": _int32(kv_lens),
            "out": torch.zeros((n, hq, d), dtype=dt, device=DEV),
            "lse": torch.zeros((n, hq), dtype=torch.float32, device=DEV)}


def _prepare_prefix(case, seed):
    g = _generator(seed)
    dt, d, hq, b = DT[case["dtype"]], case["dim"], case["q_heads"], case["batch"]
    members, prefix, mine = _prefix_sizes(case)
    (shared, table), pages = _tables(case, [prefix, mine], g)
    bufs, ks, vs = _cache(case, pages, g)
    return {"q": (2 * torch.randn((b, hq, d), generator=g, device=DEV)).to(dt), "table": table, "bufs": bufs,
            "pages": pages, "k_scale": ks, "v_scale": vs, "shared": shared, "starts": _int32(_starts(members)),
            "prefix": _int32(prefix), "lens": _int32(mine), "out": torch.zeros((b, hq, d), dtype=dt, device=DEV),
            "lse": torch.zeros((b, hq), dtype=torch.float32, device=DEV)}


def _prepare_merge(case, seed):
    g = _generator(seed)
    dt, n, h, d = DT[case["dtype"]], case["tokens"], case["q_heads"], case["dim"]
    outs, lses = [], []
    for _ in range(case["parts"]):
        outs.append(torch.randn((n, h, d), generator=g, device=DEV, dtype=torch.float32).to(dt))
        lse = 8 + 3 * torch.randn((n, h), generator=g, device=DEV)
        if case["empty"]:                 # parts without a token for some rows: zeros there
            none = torch.rand((n, 1), generator=g, device=DEV) < 0.25
            lse = torch.where(none, -torch.inf, lse)
            outs[-1] = torch.where(none[:, :, None], 0.0, outs[-1]).to(dt)
        lses.append(lse)
    return {"outs": outs, "lses": lses, "out": torch.zeros((n, h, d), dtype=dt, device=DEV),
            "lse": torch.zeros((n, h), dtype=torch.float32, device=DEV)}


def prepare(case, seed):
    s = {"query": _prepare_query, "prefix": _prepare_prefix, "merge": _prepare_merge}[case["op"]](case, seed)
    s["case"] = case
    if own:
        _handles(s)
    return s


# ---- the library's calls -------------------------------------------------------------

def _handles(s):
    """What a serving program keeps: the pool's shape, the device buffers, a workspace."""
    import tiered_kv_cache_gb300 as hc

    case = s["case"]
    s["hc"] = hc
    if case["op"] == "merge":
        return
    s["desc"] = hc.PoolDesc(1, 2, case["page"], _elem(case), case["kv_heads"] * case["dim"], 1, hc.LAYER_FIRST, 0, 0, 0)
    s["kv"] = hc.DeviceKV(s["bufs"], s["pages"])
    if case["op"] == "query":
        n = hc.query_workspace(s["desc"], case["batch"], s["q"].shape[0], case["q_heads"], case["dim"],
                               s["table"].shape[1])
    else:
        n = hc.prefix_workspace(s["desc"], case["batch"], case["groups"], case["q_heads"], case["dim"],
                                s["shared"].shape[1], s["table"].shape[1])
    s["workspace"] = torch.zeros(n, dtype=torch.uint8, device=DEV)


def _own(s):
    hc, case = s["hc"], s["case"]
    if case["op"] == "query":
        hc.query_attention(s["kv"], s["desc"], 0, s["q"], s["starts"], s["table"], s["lens"], s["out"], s["workspace"],
                           causal=case["causal"], window=case["window"], lse=s["lse"], k_scale=s["k_scale"],
                           v_scale=s["v_scale"])
    elif case["op"] == "prefix":
        hc.prefix_attention(s["kv"], s["desc"], 0, s["q"], s["starts"], s["shared"], s["prefix"], s["table"], s["lens"],
                            s["out"], s["workspace"], lse=s["lse"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    else:
        hc.merge_attention(s["outs"], s["lses"], s["out"], lse=s["lse"])
    return [s["out"], s["lse"]]


# ---- the plain forms -------------------------------------------------------------------

def _rows(s, buf, table, n):
    """The first n tokens of a table's row, [kv_heads, n, dim] in 32 bits (without the scale)."""
    case = s["case"]
    p = case["page"]
    pages = table[:-(-n // p)].long()
    raw = buf.view(torch.uint8) if buf.element_size() == 1 else buf
    x = raw.view(s["pages"], p, -1)[pages].flatten(0, 1)[:n]
    return x.view(buf.dtype).float().view(n, case["kv_heads"], case["dim"]).transpose(0, 1)


def _softmax_product(x, v):
    """x [heads, rows, tokens] scores with -infinity where masked; v [heads, tokens, dim].
    Returns the products with their softmax, and its log-sums."""
    top = x.amax(-1, keepdim=True) if x.shape[-1] else x.new_full((*x.shape[:-1], 1), -torch.inf)
    top = torch.where(top == -torch.inf, 0.0, top)
    x = torch.exp(x - top)
    z = x.sum(-1, keepdim=True)
    return torch.matmul(x, v) / torch.where(z > 0, z, 1.0), (top + torch.log(z)).squeeze(-1)


_ROWS = 1024                             # query tokens of a sequence at a time: their scores are kept in memory


def _plain_query(s):
    case = s["case"]
    d, hk = case["dim"], case["kv_heads"]
    group = case["q_heads"] // hk
    q_lens, kv_lens = _query_sizes(case)
    at = 0
    for b, (nq, nk) in enumerate(zip(q_lens, kv_lens)):
        k, v = (_rows(s, buf, s["table"][b], nk) for buf in s["bufs"])
        for i in range(0, nq, _ROWS):
            m = min(_ROWS, nq - i)
            rows = slice(at + i, at + i + m)
            # [hk, group * m, d]
            q = s["q"][rows].float().view(m, hk, group, d).permute(1, 2, 0, 3).reshape(hk, group * m, d)
            x = torch.matmul(q, k.transpose(1, 2)) * (s["k_scale"] / math.sqrt(d))
            if case["causal"]:
                pos = torch.arange(nk - nq + i, nk - nq + i + m, device=DEV)[:, None]
                tok = torch.arange(nk, device=DEV)[None, :]
                seen = tok <= pos
                if case["window"]:
                    seen &= tok > pos - case["window"]
                x = torch.where(seen.repeat(group, 1), x, -torch.inf)
            y, z = _softmax_product(x, v)
            s["out"][rows] = (y * s["v_scale"]).view(hk, group, m, d).permute(2, 0, 1, 3).reshape(m, -1, d).to(s["out"].dtype)
            s["lse"][rows] = z.view(hk, group, m).permute(2, 0, 1).reshape(m, -1)
        at += nq
    return [s["out"], s["lse"]]


def _plain_prefix(s):
    case = s["case"]
    d, hk, p, b = case["dim"], case["kv_heads"], case["page"], case["batch"]
    group = case["q_heads"] // hk
    members, prefix, _ = _prefix_sizes(case)
    # each sequence's own pages, in one batch
    width = s["table"].shape[1]
    seen = torch.arange(width * p, device=DEV)[None, :] < s["lens"][:, None]
    page = s["table"].clamp(min=0).long()
    k, v = ((x.view(torch.uint8) if x.element_size() == 1 else x).view(s["pages"], p, hk, d)[page].view(x.dtype).float()
            .view(b, width * p, hk, d).transpose(1, 2) for x in s["bufs"])
    v = torch.where(seen[:, None, :, None], v, 0.0)
    q = s["q"].float().view(b, hk, group, d)
    scale = s["k_scale"] / math.sqrt(d)
    x = torch.where(seen[:, None, None, :], torch.matmul(q, k.transpose(2, 3)) * scale, -torch.inf)
    top = x.amax(-1)
    lift = torch.where(top == -torch.inf, 0.0, top)
    x = torch.exp(x - lift[..., None])
    total, y = x.sum(-1), torch.matmul(x, v)
    # each group's prefix, once for all of its sequences
    at = 0
    for i, (m, n) in enumerate(zip(members, prefix)):
        if m and n:
            k, v = (_rows(s, buf, s["shared"][i], n) for buf in s["bufs"])
            rows = slice(at, at + m)
            x = torch.matmul(q[rows].transpose(0, 1).reshape(hk, m * group, d), k.transpose(1, 2)) * scale
            there = x.amax(-1).view(hk, m, group).transpose(0, 1)
            now = torch.maximum(lift[rows], there)
            now = torch.where(top[rows] == -torch.inf, there, now)
            x = torch.exp(x - now.transpose(0, 1).reshape(hk, m * group, 1))
            was = torch.exp(lift[rows] - now)
            was = torch.where(top[rows] == -torch.inf, 0.0, was)
            total[rows] = total[rows] * was + x.sum(-1).view(hk, m, group).transpose(0, 1)
            y[rows] = y[rows] * was[..., None] + torch.matmul(x, v).view(hk, m, group, d).transpose(0, 1)
            lift[rows] = now
        at += m
    s["out"].copy_((y * (s["v_scale"] / torch.where(total > 0, total, 1.0))[..., None]).view(b, -1, d))
    s["lse"].copy_((lift + torch.log(total)).view(b, -1))
    return [s["out"], s["lse"]]


def _plain_merge(s):
    top = s["lses"][0]
    for z in s["lses"][1:]:
        top = torch.maximum(top, z)
    lift = torch.where(top == -torch.inf, 0.0, top)
    total, y = torch.zeros_like(top), 0.0
    for x, z in zip(s["outs"], s["lses"]):
        w = torch.exp(z - lift)
        total += w
        y = y + x.float() * w[..., None]
    s["out"].copy_(y / torch.where(total > 0, total, 1.0)[..., None])
    s["lse"].copy_(lift + torch.log(total))
    return [s["out"], s["lse"]]


def run(s):
    if own:
        return _own(s)
    op = s["case"]["op"]
    return _plain_query(s) if op == "query" else _plain_prefix(s) if op == "prefix" else _plain_merge(s)


# ---- 64 bits -----------------------------------------------------------------------------

def _head_rows(s, which, table, n, h):
    """Tokens 0..n-1 of one kv head in 64 bits, with the scale."""
    case = s["case"]
    p, d = case["page"], case["dim"]
    t = torch.arange(n, device=DEV)
    at = table[t // p].long() * p + t % p
    x = s["bufs"][which][:, h * d:(h + 1) * d]
    x = x.view(torch.uint8)[at].view(x.dtype) if x.element_size() == 1 else x[at]
    return x.double() * (s["k_scale"] if which == 0 else s["v_scale"])


def _exact_rows(q, k, v, keep, scale):
    """(out, lse) of rows q [n, d] over tokens k, v; keep [n, tokens] or None."""
    if k.shape[0] == 0:
        return torch.zeros_like(q), q.new_full((q.shape[0],), -torch.inf)
    x = (q @ k.T) * scale
    if keep is not None:
        x.masked_fill_(~keep, -torch.inf)
    z = torch.logsumexp(x, -1)
    w = torch.exp(x - torch.where(z == -torch.inf, 0.0, z)[:, None])
    return w @ v, z


def _exact_query(s, case):
    d, hk = case["dim"], case["kv_heads"]
    group = case["q_heads"] // hk
    q_lens, kv_lens = _query_sizes(case)
    out = s["out"].double()
    lse = s["lse"].double()
    at = 0
    for b, (nq, nk) in enumerate(zip(q_lens, kv_lens)):
        for h in range(hk):
            k, v = (_head_rows(s, w, s["table"][b], nk, h) for w in (0, 1))
            for j in range(h * group, (h + 1) * group):
                for i in range(0, nq, 2048):
                    m = min(2048, nq - i)
                    lo, hi = 0, nk
                    keep = None
                    if case["causal"]:   # only the tokens that some row of these sees
                        hi = max(0, nk - nq + i + m)
                        lo = max(0, nk - nq + i + 1 - case["window"]) if case["window"] else 0
                        pos = torch.arange(nk - nq + i, nk - nq + i + m, device=DEV)
                        off = pos[:, None] - torch.arange(lo, hi, device=DEV)[None, :]
                        keep = (off >= 0) & (off < case["window"]) if case["window"] else off >= 0
                    rows = slice(at + i, at + i + m)
                    out[rows, j], lse[rows, j] = _exact_rows(s["q"][rows, j].double(), k[lo:hi], v[lo:hi], keep,
                                                            1.0 / math.sqrt(d))
        at += nq
    return [out, lse]


def _exact_prefix(s, case):
    d, hk = case["dim"], case["kv_heads"]
    group = case["q_heads"] // hk
    members, prefix, mine = _prefix_sizes(case)
    out = torch.zeros((case["batch"], case["q_heads"], d), dtype=torch.float64, device=DEV)
    lse = torch.zeros((case["batch"], case["q_heads"]), dtype=torch.float64, device=DEV)
    owner = [g for g, m in enumerate(members) for _ in range(m)]
    owner += [-1] * (case["batch"] - len(owner))
    for h in range(hk):
        heads = slice(h * group, (h + 1) * group)
        shared = [[_head_rows(s, w, s["shared"][g], n, h) for w in (0, 1)] for g, n in enumerate(prefix)]
        for b, n in enumerate(mine):
            k, v = (_head_rows(s, w, s["table"][b], n, h) for w in (0, 1))
            if owner[b] >= 0:
                k, v = (torch.cat([a, c]) for a, c in zip(shared[owner[b]], (k, v)))
            out[b, heads], lse[b, heads] = _exact_rows(s["q"][b, heads].double(), k, v, None, 1.0 / math.sqrt(d))
    return [out, lse]


def _exact_merge(s):
    z = torch.stack(s["lses"]).double()
    lse = torch.logsumexp(z, 0)
    w = torch.exp(z - torch.where(lse == -torch.inf, 0.0, lse))
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    for x, f in zip(s["outs"], w):
        out += x.double() * f[..., None]
    return [out, lse]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    return _exact_query(s, case) if op == "query" else _exact_prefix(s, case) if op == "prefix" else _exact_merge(s)


# ---- what a pass cannot do without ---------------------------------------------------------

def _pairs(nq, nk, causal, window):
    """Pairs of a query and a token that it attends to."""
    if not causal:
        return nq * nk
    seen = lambda n: max(0, n) * (max(0, n) + 1) // 2    # noqa: E731  tokens seen by positions 0..n-1 in all
    full = seen(nk) - seen(nk - nq)
    if not window:
        return full
    return full - (seen(nk - window) - seen(nk - nq - window))   # without those before the windows


def work(case):
    h, d = case["q_heads"], case["dim"]
    if case["op"] == "merge":
        n, parts = case["tokens"] * h, case["parts"]
        return {"bytes": (parts + 1) * n * (2 * d + 4), "flops": 2 * parts * n * d}
    row = 2 * case["kv_heads"] * d * _elem(case)
    p = case["page"]
    if case["op"] == "query":
        q_lens, kv_lens = _query_sizes(case)
        w = case["window"]
        tokens = sum(min(nk, nq + w - 1) if w else nk for nq, nk in zip(q_lens, kv_lens))
        pairs = sum(_pairs(nq, nk, case["causal"], w) for nq, nk in zip(q_lens, kv_lens))
        rows, ints = sum(q_lens), 2 * case["batch"] + sum(-(-n // p) for n in kv_lens)
    else:
        members, prefix, mine = _prefix_sizes(case)
        used = [n if m else 0 for m, n in zip(members, prefix)]
        tokens = sum(used) + sum(mine)
        pairs = sum(m * n for m, n in zip(members, used)) + sum(mine)
        rows, ints = case["batch"], 2 * case["groups"] + case["batch"] + sum(-(-n // p) for n in used + mine)
    return {"bytes": tokens * row + rows * h * (4 * d + 4) + 4 * ints, "flops": 4 * pairs * h * d}
