"""The serving operators on the device side of the tiered cache, as measured cases.

Three operators that a serving step runs on the pages this library moves:

  append   norms of each query and key head, the position rotation, and the
           store of K and V into their slots of the paged device cache
           (``append_kv``);
  decode   attention of one new token per sequence over its pages, split over
           the cache's length and joined, with (optionally) the attention
           weight that each page received (``decode_attention``);
  evict    which pages of each sequence leave the cache: those with the least
           accumulated weight (``evict_pages``).

``own`` selects the library's calls; otherwise ``run`` computes the same from
elementary torch operations in 32 bits.  ``exact`` computes it in 64 bits, one
sequence (or token block) at a time, from the definitions.
"""
from __future__ import annotations

import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
DEV = "cuda"


# ---- cases ----------------------------------------------------------------------

def _append(name, tokens, q_heads, kv_heads, dim, page, dtype="bf16", cache="same", rot=0, rot_offset=0,
            interleaved=False, norm=0, padded=0):
    return {"name": name, "op": "append", "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim,
            "page": page, "dtype": dtype, "cache": cache, "rot": rot or dim, "rot_offset": rot_offset,
            "interleaved": interleaved, "norm": norm or dim, "padded": padded}


def _decode(name, batch, min_len, max_len, q_heads, kv_heads, dim, page, v_dim=0, dtype="bf16", cache="same",
            window=0, weights=False, holes=False, empty=False):
    return {"name": name, "op": "decode", "batch": batch, "min_len": min_len, "max_len": max_len,
            "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "page": page, "v_dim": v_dim or dim,
            "dtype": dtype, "cache": cache, "window": window, "weights": weights, "holes": holes, "empty": empty}


def _evict(name, batch, min_len, max_len, page, keep_percent, sink=4, recent=8):
    return {"name": name, "op": "evict", "batch": batch, "min_len": min_len, "max_len": max_len, "page": page,
            "keep_percent": keep_percent, "sink": sink, "recent": recent}


def listed():
    return [
        # one request decoding alone: 32 query heads on 8 kv heads of 128, the row of the 32-layer workload
        _append("append_1", 1, 32, 8, 128, 64),
        # a padded decode batch into an 8-bit cache, interleaved rotation of half of each head
        _append("append_300_e4m3", 300, 32, 8, 128, 16, dtype="fp16", cache="e4m3", rot=64, interleaved=True, padded=29),
        # one prefill chunk of a long prompt
        _append("append_8k", 8191, 32, 8, 128, 64),
        # prefill of a latent cache: the norm over the 512 latent elements, the rotation of the last 64
        _append("append_latent_4k", 4096, 16, 1, 576, 64, rot=64, rot_offset=512, norm=512),
        # one request decoding alone at 4K tokens: latency
        _decode("decode_1x4k", 1, 4097, 4097, 32, 8, 128, 64),
        # a multi-turn batch: ragged lengths, pages of 16, one sequence not started
        _decode("decode_64_ragged", 64, 33, 8192, 32, 8, 128, 16, empty=True),
        # long contexts at the 32-layer workload's row and page size
        _decode("decode_16x32k", 16, 32768, 32768, 32, 8, 128, 64),
        # an 8-bit cache whose pages are weighed for eviction
        _decode("decode_24_e4m3_weights", 24, 2000, 16384, 32, 8, 128, 16, dtype="fp16", cache="e4m3", weights=True),
        # the latent cache, one tensor-parallel rank's 16 heads
        _decode("decode_latent_16h", 32, 4096, 16384, 16, 0, 576, 64, v_dim=512),
        # the latent cache, all 128 heads on one GPU: compute
        _decode("decode_latent_128h", 32, 4096, 16384, 128, 0, 576, 64, v_dim=512),
        # a decode batch over its budget, pages of 16
        _evict("evict_32x2k", 32, 16384, 32768, 16, 50),
        # two very long sequences with one-token pages
        _evict("evict_2x100k", 2, 100000, 131071, 1, 75, sink=16, recent=256),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "decode", "decode", "latent", "evict"))
    dtype = rng.choice(("bf16", "fp16"))
    page = rng.choice((1, 5, 16, 64, 128))
    if op == "append":
        tokens = _log(rng, 1, 6000)
        if rng.random() < 0.25:
            c = _append("", tokens, rng.choice((8, 16, 32)), 1, 576, page, dtype, rot=64, rot_offset=512, norm=512,
                        interleaved=rng.random() < 0.5, padded=rng.randint(0, tokens // 4))
        else:
            kv = rng.choice((1, 2, 3, 4, 8))
            dim = rng.choice((64, 80, 96, 128, 192, 256))
            q_heads = max(kv, min(kv * rng.choice((1, 2, 4, 5, 7, 8)), 6144 // dim))
            c = _append("", tokens, q_heads, kv, dim, page, dtype, rng.choice(("same", "e4m3")),
                        rot=rng.choice((dim, dim // 2)), interleaved=rng.random() < 0.5,
                        padded=rng.randint(0, tokens // 4))
    elif op == "evict":
        longest = _log(rng, 2, 60000)
        batch = max(1, min(256, _log(rng, 1, 2 * 60000 // longest + 1)))
        c = _evict("", batch, max(1, longest * page // rng.randint(1, 8)), longest * page, page, rng.randint(5, 100),
                   sink=rng.randint(0, 8), recent=rng.randint(1, 16))
    else:
        longest = _log(rng, 1, 40000)
        batch = _log(rng, 1, max(1, min(256, 200000 // longest)))
        shortest = max(1, longest // rng.choice((1, 1, 3, 20)))
        more = {"weights": rng.random() < 0.4, "holes": rng.random() < 0.2, "empty": rng.random() < 0.3}
        if op == "latent":
            c = _decode("", batch, shortest, longest, rng.choice((8, 16, 20, 32, 64, 128)), 0, 576, page, 512, dtype,
                        **more)
        else:
            kv = rng.choice((1, 2, 4, 8))
            more["window"] = rng.choice((0, 0, 0, rng.randint(1, longest)))
            dim = rng.choice((64, 80, 96, 128, 192, 256))
            group = rng.choice((1, 2, 3, 4, 6, 8, 12, 16))
            c = _decode("", batch, shortest, longest, kv * group, kv, dim, page, 0, dtype,
                        rng.choice(("same", "e4m3")), **more)
    del c["name"]
    return c


# ---- sizes that follow from a case alone -------------------------------------------

def _lengths(case):
    """The sequences' lengths: spread evenly over the logarithm between the
    shortest and the longest, in mixed order, odd ones among them."""
    n, lo, hi = case["batch"], case["min_len"], case["max_len"]
    at = [(i * 0.6180339887498949 + 0.5) % 1.0 for i in range(n)]
    lens = [int(round(math.exp(math.log(lo) + (math.log(hi) - math.log(lo)) * x))) for x in at]
    lens[0] = hi
    if case.get("empty") and n > 1:
        lens[-1] = 0
    return lens


def _pages(case):
    p = case["page"]
    return [-(-n // p) for n in _lengths(case)]


def _elem(case):
    return 1 if case["cache"] == "e4m3" else 2


# ---- inputs ------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _table(counts, width, spare, g):
    """Page tables of sequences that share nothing, from a shuffled pool; -1
    behind each sequence's last page."""
    total = sum(counts)
    perm = torch.randperm(total + spare, generator=g, device=DEV)[:total].to(torch.int32)
    n = torch.tensor(counts, device=DEV)
    first = torch.cumsum(n, 0) - n
    col = torch.arange(width, device=DEV)
    inside = col[None, :] < n[:, None]
    at = (first[:, None] + col[None, :]).clamp_(max=max(0, total - 1))
    full = torch.full((len(counts), width), -1, dtype=torch.int32, device=DEV)
    return torch.where(inside, perm[at], full) if total else full


def _prepare_append(case, seed):
    g = _generator(seed)
    dt, n, d, p = DT[case["dtype"]], case["tokens"], case["dim"], case["page"]
    hq, hk, latent = case["q_heads"], case["kv_heads"], case["dim"] > 256
    heads = hq + hk * (1 if latent else 2)
    fused = torch.randn((n, heads * d), generator=g, device=DEV, dtype=torch.float32).to(dt)  # a fused projection's output
    q, k = fused[:, :hq * d].view(n, hq, d), fused[:, hq * d:(hq + hk) * d].view(n, hk, d)
    v = None if latent else fused[:, (hq + hk) * d:].view(n, hk, d)
    pages = -(-n // p) + 2
    cache = torch.float8_e4m3fn if case["cache"] == "e4m3" else dt
    slots = torch.randperm(pages * p, generator=g, device=DEV)[:n]
    if case["padded"]:  # rows that only fill up the batch: nothing of theirs is stored
        slots[n - case["padded"]:] = -1
    rows = 40000
    positions = torch.randint(0, rows, (n,), generator=g, device=DEV)
    freq = 10000.0 ** (-torch.arange(0, case["rot"], 2, device=DEV, dtype=torch.float64) / case["rot"])
    angle = torch.arange(rows, device=DEV, dtype=torch.float64)[:, None] * freq[None, :]
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float()
    weight = lambda m: (1 + 0.2 * torch.randn(m, generator=g, device=DEV)).to(dt)  # noqa: E731
    kw, qw = weight(case["norm"]), None if latent else weight(case["norm"])
    bufs = [torch.zeros((pages * p, hk * d), device=DEV, dtype=torch.float32).to(cache) for _ in range(1 if latent else 2)]
    s = {"q": q, "k": k, "v": v, "slots": slots, "positions": positions, "cos_sin": cos_sin, "q_weight": qw,
         "k_weight": kw, "q_out": torch.zeros((n, hq, d), device=DEV, dtype=dt), "bufs": bufs, "pages": pages,
         "k_scale": 0.02 if case["cache"] == "e4m3" else 1.0, "v_scale": 0.015 if case["cache"] == "e4m3" else 1.0}
    return s


def _prepare_decode(case, seed):
    g = _generator(seed)
    dt, d, p, b = DT[case["dtype"]], case["dim"], case["page"], case["batch"]
    latent = case["kv_heads"] == 0
    row = d if latent else case["kv_heads"] * d
    counts = _pages(case)
    width = max(1, max(counts))
    spare = max(1, sum(counts) // 16)
    table = _table(counts, width, spare, g)
    if case["holes"]:  # pages that are not on the device
        table = torch.where(torch.rand(table.shape, generator=g, device=DEV) < 0.1, -1, table)
    dp = sum(counts) + spare
    bufs = [torch.randn((dp * p, row), generator=g, device=DEV, dtype=dt) for _ in range(1 if latent else 2)]
    k_scale = v_scale = 1.0
    if case["cache"] == "e4m3":
        k_scale, v_scale = 0.0625, 0.03125
        bufs = [(x.float() / sc).to(torch.float8_e4m3fn) for x, sc in zip(bufs, (k_scale, v_scale))]
    q = (2 * torch.randn((b, case["q_heads"], d), generator=g, device=DEV)).to(dt)
    s = {"q": q, "table": table, "lens": torch.tensor(_lengths(case), dtype=torch.int32, device=DEV), "bufs": bufs,
         "pages": dp, "k_scale": k_scale, "v_scale": v_scale, "scale": 1.0 / math.sqrt(192.0 if latent else d),
         "out": torch.empty((b, case["q_heads"], case["v_dim"]), dtype=dt, device=DEV),
         "lse": torch.empty((b, case["q_heads"]), dtype=torch.float32, device=DEV), "weights": None}
    if case["weights"]:
        s["weights"] = torch.rand((b, width), generator=g, device=DEV)
    return s


def _prepare_evict(case, seed):
    g = _generator(seed)
    counts = _pages(case)
    width = max(counts) + 3
    table = _table(counts, width, 16, g)
    n = torch.tensor(counts, device=DEV)
    # accumulated softmax weight: most pages hold next to nothing, some of them exactly the same (none at all)
    w = torch.exp(3 * torch.randn((case["batch"], width), generator=g, device=DEV))
    w = torch.where(torch.rand(w.shape, generator=g, device=DEV) < 0.1, 0.0, w)
    keep = torch.div(n * case["keep_percent"], 100, rounding_mode="floor").to(torch.int32)
    like = torch.empty_like
    return {"table": table, "weights": w, "lens": torch.tensor(_lengths(case), dtype=torch.int32, device=DEV),
            "keep": keep, "victims": torch.full_like(table, -1), "counts": torch.zeros_like(keep),
            "out_table": torch.full_like(table, -1), "out_weights": torch.zeros_like(w), "out_lens": like(keep)}


def prepare(case, seed):
    s = {"append": _prepare_append, "decode": _prepare_decode, "evict": _prepare_evict}[case["op"]](case, seed)
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
    if case["op"] == "evict":
        return
    buf = s["bufs"][0]
    s["desc"] = hc.PoolDesc(1, len(s["bufs"]), case["page"], _elem(case), buf.shape[1], 1, hc.LAYER_FIRST, 0, 0, 0)
    s["kv"] = hc.DeviceKV(s["bufs"], s["pages"])
    if case["op"] == "decode":
        n = hc.decode_workspace(s["desc"], case["batch"], case["q_heads"], case["dim"], case["v_dim"],
                                s["table"].shape[1], case["weights"])
        s["workspace"] = torch.zeros(n, dtype=torch.uint8, device=DEV)


def _own(s):
    hc, case = s["hc"], s["case"]
    if case["op"] == "append":
        hc.append_kv(s["kv"], s["desc"], 0, s["q"], s["k"], s["v"], s["slots"], q_out=s["q_out"],
                     positions=s["positions"], cos_sin=s["cos_sin"], rot_offset=case["rot_offset"],
                     interleaved=case["interleaved"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                     k_scale=s["k_scale"], v_scale=s["v_scale"])
        return [s["q_out"], *s["bufs"]]
    if case["op"] == "decode":
        hc.decode_attention(s["kv"], s["desc"], 0, s["q"], s["table"], s["lens"], s["out"], s["workspace"],
                            scale=s["scale"], window=case["window"], weights=s["weights"], decay=0.875,
                            lse=s["lse"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        return [s["out"], s["lse"]] + ([s["weights"]] if case["weights"] else [])
    hc.evict_pages(case["page"], s["table"], s["lens"], s["weights"], s["keep"], s["victims"], s["counts"],
                   sink=case["sink"], recent=case["recent"], out_table=s["out_table"], out_lens=s["out_lens"],
                   out_weights=s["out_weights"])
    return [s["victims"], s["counts"], s["out_table"], s["out_lens"], s["out_weights"]]


# ---- the plain forms -------------------------------------------------------------------

def _norm(x, w):
    n = w.shape[0]
    y = x[..., :n]
    y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w.float()
    return torch.cat([y, x[..., n:]], -1) if n < x.shape[-1] else y


def _rotate(x, cs, offset, interleaved):
    half = cs.shape[-1] // 2
    cos, sin = cs[:, None, :half], cs[:, None, half:]
    r = x[..., offset:offset + 2 * half]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = r[..., :half], r[..., half:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([x[..., :offset], r, x[..., offset + 2 * half:]], -1)


def _to_cache(x, scale, dtype):
    if dtype == torch.float8_e4m3fn:
        x = (x / scale).clamp(-448.0, 448.0)
    return x.to(dtype)


def _plain_append(s):
    case = s["case"]
    cs = s["cos_sin"][s["positions"]]
    q, k = s["q"].float(), s["k"].float()
    q = _norm(q, s["q_weight"]) if s["q_weight"] is not None else q
    k = _norm(k, s["k_weight"])
    q, k = (_rotate(x, cs, case["rot_offset"], case["interleaved"]) for x in (q, k))
    s["q_out"].copy_(q)
    live = s["slots"] >= 0
    at = s["slots"][live]
    rows = [k] if s["v"] is None else [k, s["v"].float()]
    for buf, x, scale in zip(s["bufs"], rows, (s["k_scale"], s["v_scale"])):
        y = _to_cache(x.flatten(1)[live], scale, buf.dtype)
        small = buf.element_size() == 1
        (buf.view(torch.uint8) if small else buf)[at] = y.view(torch.uint8) if small else y
    return [s["q_out"], *s["bufs"]]


def _plain_decode(s):
    case = s["case"]
    b, p, d, dv = case["batch"], case["page"], case["dim"], case["v_dim"]
    latent = case["kv_heads"] == 0
    hk = 1 if latent else case["kv_heads"]
    table, lens = s["table"], s["lens"].long()
    width = table.shape[1]
    tok = torch.arange(width * p, device=DEV)
    seen = (tok[None, :] < lens[:, None]) & (table >= 0).repeat_interleave(p, 1)
    if case["window"]:
        seen &= tok[None, :] >= lens[:, None] - case["window"]
    at = table.clamp(min=0).long()
    rows = [(x.view(torch.uint8) if x.element_size() == 1 else x).view(s["pages"], p, hk, d)[at].view(x.dtype)
            .view(b, width * p, hk, d).transpose(1, 2) for x in s["bufs"]]
    k = rows[0].float()
    q = s["q"].float().view(b, hk, -1, d)
    x = torch.matmul(q, k.transpose(2, 3)) * (s["scale"] * s["k_scale"])
    x = torch.where(seen[:, None, None, :], x, -torch.inf)
    v = k[..., :dv] if latent else rows[1].float()
    del k
    v = torch.where(seen[:, None, :, None], v, 0.0)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -torch.inf, 0.0, top)
    x = torch.exp(x - top)
    z = x.sum(-1, keepdim=True)
    x = x / torch.where(z > 0, z, 1.0)
    s["out"].copy_((torch.matmul(x, v) * s["v_scale"]).view(b, -1, dv))
    s["lse"].copy_((top + torch.log(z)).view(b, -1))
    if not case["weights"]:
        return [s["out"], s["lse"]]
    w = x.sum((1, 2)).view(b, width, p).sum(2)
    live = torch.arange(width, device=DEV)[None, :] * p < lens[:, None]
    s["weights"].copy_(torch.where(live, 0.875 * s["weights"] + w, s["weights"]))
    return [s["out"], s["lse"], s["weights"]]


def _plain_evict(s):
    case = s["case"]
    p = case["page"]
    table, w, lens = s["table"], s["weights"], s["lens"]
    width = table.shape[1]
    col = torch.arange(width, device=DEV)[None, :]
    n = ((lens + (p - 1)) // p)[:, None]
    may = (col >= case["sink"]) & (col < n - case["recent"])
    gone = torch.minimum((n[:, 0] - s["keep"]).clamp(min=0), may.sum(1)).to(torch.int32)
    # rank among the pages that may go: by weight, the earliest first among equals
    order = torch.sort(w, dim=1, stable=True).indices
    late = torch.sort((~may.gather(1, order)).to(torch.uint8), dim=1, stable=True).indices
    rank = torch.empty_like(order).scatter_(1, order.gather(1, late), col.expand_as(order))
    out = may & (rank < gone[:, None])
    stay = (col < n) & ~out
    # destinations: pages that leave and pages that stay, each in their order
    victims, tables, weights = s["victims"], s["out_table"], s["out_weights"]
    row = torch.arange(case["batch"], device=DEV)[:, None].expand_as(table)
    to = torch.cumsum(out, 1) - 1
    victims[row[out], to[out]] = table[out]
    to = torch.cumsum(stay, 1) - 1
    left = n - gone[:, None]
    cleared = (col >= left) & (col < n)
    tables[cleared] = -1
    weights[cleared] = 0.0
    tables[row[stay], to[stay]] = table[stay]
    weights[row[stay], to[stay]] = w[stay]
    s["counts"].copy_(gone)
    s["out_lens"].copy_(lens - gone * p)
    return [victims, s["counts"], tables, s["out_lens"], weights]


def run(s):
    if own:
        return _own(s)
    op = s["case"]["op"]
    return _plain_append(s) if op == "append" else _plain_decode(s) if op == "decode" else _plain_evict(s)


# ---- 64 bits -----------------------------------------------------------------------------

def _exact_append(s, case):
    n, d, hk = case["tokens"], case["dim"], case["kv_heads"]
    half, off = case["rot"] // 2, case["rot_offset"]
    c = s["cos_sin"].double()[s["positions"]].view(n, 1, 2, half)
    first = torch.arange(half, device=DEV) * (2 if case["interleaved"] else 1) + off
    second = first + (1 if case["interleaved"] else half)

    def turned(x, w):
        y = x.double().clone()
        if w is not None:
            m = w.shape[0]
            y[..., :m] /= torch.sqrt(y[..., :m].pow(2).sum(-1, keepdim=True) / m + 1e-6)
            y[..., :m] *= w.double()
        a, b = y[..., first], y[..., second]
        y[..., first] = a * c[:, :, 0] - b * c[:, :, 1]
        y[..., second] = a * c[:, :, 1] + b * c[:, :, 0]
        return y

    out = [turned(s["q"], s["q_weight"])]
    stored = [(turned(s["k"], s["k_weight"]), s["k_scale"])]
    if s["v"] is not None:
        stored.append((s["v"].double(), s["v_scale"]))
    keep = n - case["padded"]
    for x, scale in stored:
        rows = torch.zeros((s["pages"] * case["page"], hk * d), dtype=torch.float64, device=DEV)
        rows[s["slots"][:keep]] = x[:keep].reshape(keep, hk * d) / scale
        out.append(rows.clamp(-448, 448) if case["cache"] == "e4m3" else rows)
    return out


def _exact_decode(s, case):
    p, d, dv, hq = case["page"], case["dim"], case["v_dim"], case["q_heads"]
    hk = max(1, case["kv_heads"])
    out = torch.zeros((case["batch"], hq, dv), dtype=torch.float64, device=DEV)
    lse = torch.full((case["batch"], hq), -torch.inf, dtype=torch.float64, device=DEV)
    weights = s["weights"].double() if case["weights"] else None
    for i, n in enumerate(_lengths(case)):
        pages = -(-n // p)
        t = torch.arange(max(0, n - case["window"]) if case["window"] else 0, n, device=DEV)
        page = s["table"][i].long()[t // p]
        t, page = t[page >= 0], page[page >= 0]
        share = torch.zeros(pages, dtype=torch.float64, device=DEV)
        if t.numel():
            k = s["bufs"][0][page * p + t % p].double().view(-1, hk, d) * s["k_scale"]
            v = k[..., :dv] if case["kv_heads"] == 0 else s["bufs"][1][page * p + t % p].double().view(-1, hk, d) * s["v_scale"]
            x = torch.einsum("kgd,tkd->kgt", s["q"][i].double().view(hk, -1, d), k) * s["scale"]
            z = torch.logsumexp(x, -1, keepdim=True)
            x = torch.exp(x - z)
            out[i] = torch.einsum("kgt,tkd->kgd", x, v).reshape(hq, dv)
            lse[i] = z.flatten()
            share.index_add_(0, t // p, x.sum((0, 1)))
        if weights is not None:
            weights[i, :pages] = 0.875 * weights[i, :pages] + share
    return [out, lse] + ([weights] if weights is not None else [])


def exact(case, seed):
    if case["op"] == "evict":
        return None  # whole numbers and copies
    s = prepare(case, seed)
    return _exact_append(s, case) if case["op"] == "append" else _exact_decode(s, case)


# ---- what a pass cannot do without ---------------------------------------------------------

def work(case):
    if case["op"] == "append":
        n, d = case["tokens"], case["dim"]
        live = n - case["padded"]
        lat = d > 256
        kv = case["kv_heads"] * d * (1 if lat else 2)
        read = n * (case["q_heads"] * d * 2 + 8 + 8 + case["rot"] * 4) + live * kv * 2
        wrote = n * case["q_heads"] * d * 2 + live * kv * _elem(case)
        return {"bytes": read + wrote, "flops": 6 * n * (case["q_heads"] + case["kv_heads"]) * d}
    lens, pages = _lengths(case), _pages(case)
    if case["op"] == "evict":
        n = sum(pages)
        return {"bytes": n * (4 + 4) * 2 + 20 * case["batch"], "flops": n}
    d, dv, hq = case["dim"], case["v_dim"], case["q_heads"]
    w = case["window"]
    tokens = sum(min(n, w) if w else n for n in lens)
    tokens = tokens * 0.9 if case["holes"] else tokens
    row = d if case["kv_heads"] == 0 else 2 * case["kv_heads"] * d
    size = tokens * row * _elem(case) + sum(pages) * (4 + (8 if case["weights"] else 0))
    size += case["batch"] * (hq * ((d + dv) * 2 + 4) + 4)
    return {"bytes": size, "flops": 2 * tokens * hq * (d + dv)}
