"""Attention of many queries over the device pages (cross attention, chunks of prompts,
shared prefixes, joins) against plain 64-bit forms, at the sizes and masks where it
can go wrong."""
import random

import pytest
import torch

import serving_reference as ref
import tiered_kv_cache_gb300 as hc

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
E4 = torch.float8_e4m3fn
INF = float("inf")


def desc(P, row, es, layers=1):
    return hc.PoolDesc(layers, 2, P, es, row, 1, hc.LAYER_FIRST, 0, 0, 0)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def raw(t):
    """Bits, for comparisons in which NaN equals itself."""
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Cache:
    """A cache filled with NaN in which only the tokens of the lists of lengths are
    written, and page tables whose other entries are out of range."""

    def __init__(self, lens, hk, d, P, dtype="bf16", e4=False, seed=1, holes=False, spare=3, k_size=1.0):
        g, rnd = gen(seed), random.Random(seed)
        dt = E4 if e4 else DT[dtype]
        counts = [[-(-n // P) for n in some] for some in lens]
        total = sum(map(sum, counts))
        self.pages = total + spare
        order = list(range(self.pages))
        rnd.shuffle(order)
        bad = [-1, self.pages, 2 ** 31 - 1, -2 ** 31, self.pages + 17]
        self.k_scale, self.v_scale = (0.0625, 0.03125) if e4 else (1.0, 1.0)
        self.hk, self.d, self.P = hk, d, P
        fill = torch.full((self.pages * P, hk * d * dt.itemsize), 0x7F if e4 else 0xFF, dtype=torch.uint8, device="cuda")
        self.bufs = [fill.clone().view(dt) for _ in range(2)]
        self.tables, self.rows = [], []
        at = 0
        for some, cnt in zip(lens, counts):
            width = max(1, max(cnt, default=1))
            table, rows = [], []
            for n, c in zip(some, cnt):
                t = order[at:at + c]
                at += c
                slots = [p * P + i for p in t for i in range(P)][:n]
                if slots:
                    where = torch.tensor(slots, device="cuda")
                    for buf, sc, size in zip(self.bufs, (self.k_scale, self.v_scale), (k_size, 1.0)):
                        x = size * torch.randn((n, hk * d), generator=g, device="cuda") / sc
                        raw(buf)[where] = raw(x.to(dt))
                if holes:
                    t = [p if rnd.random() < 0.7 else rnd.choice(bad) for p in t]
                # the cache rows of the tokens, -1 where the page is absent
                rows.append([t[i // P] * P + i % P if 0 <= t[i // P] < self.pages else -1 for i in range(n)])
                table.append(t + [rnd.choice(bad) for _ in range(width - c)])
            self.tables.append(i32(table))
            self.rows.append(rows)
        self.kv = hc.DeviceKV(self.bufs, self.pages)
        self.desc = desc(P, hk * d, dt.itemsize)

    def plain(self):
        return [b.view(-1, self.hk, self.d) if b.element_size() == 2 else b.float().view(-1, self.hk, self.d)
                for b in self.bufs]


def present(rows):
    return torch.tensor([r for r in rows if r >= 0], dtype=torch.long, device="cuda")


def seen(rows, nq, i, causal, window):
    """The cache rows that query i of nq attends to."""
    hi = len(rows) - nq + i + 1 if causal else len(rows)
    lo = max(0, hi - window) if window else 0
    return present(rows[lo:max(0, hi)])


def queries(n, hq, d, dtype, seed=2, sharp=2.0):
    return (sharp * torch.randn((n, hq, d), generator=gen(seed), device="cuda")).to(DT[dtype])


def workspace(n):
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


def run_query(c, q, q_lens, kv_lens, causal=False, window=0, scale=None, lead=0, tail=0, ws=None, **kw):
    """One call; returns out, lse.  lead and tail rows of q belong to no sequence."""
    starts = [lead]
    for n in q_lens:
        starts.append(starts[-1] + n)
    assert q.shape[0] == starts[-1] + tail
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 5.0, device="cuda")
    if ws is None:
        ws = workspace(hc.query_workspace(c.desc, len(q_lens), q.shape[0], q.shape[1], q.shape[2], c.tables[0].shape[1]))
    hc.query_attention(c.kv, c.desc, 0, q, i32(starts), c.tables[0], i32(kv_lens), out, ws, causal=causal, window=window,
                       scale=scale, lse=lse, k_scale=c.k_scale, v_scale=c.v_scale, **kw)
    assert not hc.decode_gave_up(ws)
    return out, lse


def check_query(c, q, q_lens, out, lse, causal=False, window=0, scale=None, lead=0, pick=None):
    """pick: the queries of a sequence that are compared (all by default)."""
    k, v = c.plain()
    at = lead
    p_type = torch.bfloat16 if c.bufs[0].dtype == torch.bfloat16 else torch.float16
    for b, nq in enumerate(q_lens):
        some = list(range(nq)) if pick is None else sorted({i for i in pick if i < nq} | ({nq - 1} if nq else set()))
        rows = [seen(c.rows[0][b], nq, i, causal, window) for i in some]
        want = ref.attend(q[[at + i for i in some]], k, v, rows, q.shape[2] ** -0.5 if scale is None else scale, c.k_scale,
                          c.v_scale)
        ref.check_decode(out[[at + i for i in some]], want, q.dtype, p_type, lse=lse[[at + i for i in some]])
        at += nq
    if lead:
        assert (out[:lead] == 7.0).all() and (lse[:lead] == 5.0).all()
    assert (out[at:] == 7.0).all() and (lse[at:] == 5.0).all(), "rows of no sequence were written"


QUERY = [
    # q_lens, kv_lens, hq, hk, d, P, dtype, e4m3, causal, window
    ([1], [1], 1, 1, 64, 16, "bf16", False, False, 0),
    ([1], [300], 16, 16, 64, 64, "fp16", False, False, 0),
    ([3, 1, 7], [5, 129, 0], 4, 2, 128, 16, "bf16", False, False, 0),
    ([130], [257], 2, 2, 128, 16, "bf16", False, False, 0),
    ([40], [384], 32, 4, 128, 64, "bf16", False, False, 0),
    ([65, 0, 31], [200, 33, 1000], 8, 1, 128, 5, "fp16", False, False, 0),
    ([9, 257], [1, 640], 3, 1, 80, 7, "bf16", False, False, 0),
    ([20, 150], [100, 150], 6, 2, 96, 16, "fp16", False, True, 0),
    ([33, 1, 128], [33, 90, 513], 4, 4, 64, 1, "bf16", False, True, 0),
    ([200], [456], 14, 2, 128, 16, "bf16", False, True, 70),
    ([100, 77], [100, 300], 4, 2, 256, 16, "bf16", False, True, 0),
    ([64, 5], [64, 1025], 4, 1, 192, 128, "fp16", False, True, 33),
    ([30], [130], 2, 1, 8, 16, "bf16", False, False, 0),
    ([30], [130], 2, 1, 24, 16, "fp16", False, True, 0),
    ([50], [70], 4, 2, 200, 3, "fp16", False, False, 0),
    ([3, 140, 20], [70, 300, 20], 8, 2, 128, 16, "fp16", True, True, 0),
    ([17, 64], [270, 64], 4, 4, 64, 5, "bf16", True, False, 0),
    ([90], [333], 6, 2, 256, 64, "bf16", True, True, 100),
    ([11], [200], 5, 1, 80, 16, "fp16", True, False, 0),
    ([40, 8], [10, 3], 4, 2, 64, 16, "bf16", False, True, 0),      # more queries than tokens: rows without any
    ([300, 2], [20, 0], 8, 2, 128, 16, "fp16", False, True, 0),
    ([1] * 40, [7 * i for i in range(40)], 4, 2, 128, 16, "bf16", False, False, 0),
]


@pytest.mark.parametrize("c", QUERY, ids=[f"{i}" for i in range(len(QUERY))])
def test_query(c):
    q_lens, kv_lens, hq, hk, d, P, dtype, e4, causal, window = c
    cache = Cache([kv_lens], hk, d, P, dtype, e4)
    q = queries(sum(q_lens) + 5, hq, d, dtype)
    before = hc.launch_count()
    out, lse = run_query(cache, q, q_lens, kv_lens, causal, window, lead=2, tail=3)
    assert hc.launch_count() > before
    check_query(cache, q, q_lens, out, lse, causal, window, lead=2)
    again, lse2 = run_query(cache, q, q_lens, kv_lens, causal, window, lead=2, tail=3)
    assert torch.equal(raw(out), raw(again)) and torch.equal(raw(lse), raw(lse2))


@pytest.mark.parametrize("hq,hk,d,P,dtype,e4,causal", [
    (4, 2, 128, 16, "bf16", False, False), (2, 1, 64, 5, "fp16", False, True), (4, 1, 256, 16, "bf16", False, True),
    (8, 2, 128, 1, "fp16", True, False)])
def test_query_absent_pages(hq, hk, d, P, dtype, e4, causal):
    kv_lens, q_lens = [300, 17, 700], [40, 3, 90]
    cache = Cache([kv_lens], hk, d, P, dtype, e4, seed=4, holes=True)
    q = queries(sum(q_lens), hq, d, dtype)
    out, lse = run_query(cache, q, q_lens, kv_lens, causal)
    check_query(cache, q, q_lens, out, lse, causal)


@pytest.mark.parametrize("hq,hk,d,dtype,e4,causal,window", [
    (8, 2, 128, "bf16", False, True, 0), (4, 4, 64, "fp16", False, False, 0), (4, 2, 256, "bf16", False, True, 500),
    (8, 1, 128, "fp16", True, True, 1000)])
def test_query_long(hq, hk, d, dtype, e4, causal, window):
    """Many blocks and units to a chunk; some queries compared."""
    kv_lens, q_lens = [6001, 2111], [1500, 2050 if causal else 1111]
    cache = Cache([kv_lens], hk, d, 16, dtype, e4, seed=6)
    q = queries(sum(q_lens), hq, d, dtype)
    out, lse = run_query(cache, q, q_lens, kv_lens, causal, window)
    check_query(cache, q, q_lens, out, lse, causal, window, pick=[0, 1, 63, 64, 127, 128, 700, 1023, 1499])


@pytest.mark.parametrize("hq,hk,d,P,dtype,e4", [
    (8, 8, 128, 16, "bf16", False), (16, 8, 64, 64, "fp16", False), (24, 8, 128, 5, "bf16", False),
    (8, 8, 64, 16, "bf16", True), (8, 4, 256, 32, "fp16", False), (8, 8, 128, 16, "fp16", True),
    (16, 8, 80, 128, "bf16", False)])
def test_query_few_rows_many_blocks(hq, hk, d, P, dtype, e4):
    """Units of one tile of rows, long enough that a chunk has many of their blocks, and of
    lengths that end within a box of rows."""
    kv_lens, q_lens = [9001, 17, 20000, 4100, 128], [1, 3, 5, 20, 2]
    cache = Cache([kv_lens], hk, d, P, dtype, e4, seed=8)
    q = queries(sum(q_lens), hq, d, dtype)
    for causal in (False, True):
        out, lse = run_query(cache, q, q_lens, kv_lens, causal)
        check_query(cache, q, q_lens, out, lse, causal, pick=[0, 4, 19])


@pytest.mark.parametrize("hq,hk,d,P,causal,dtype", [
    (4, 4, 64, 16, False, "bf16"), (6, 2, 128, 64, True, "fp16"), (16, 16, 128, 16, False, "bf16")])
def test_query_many_units(hq, hk, d, P, causal, dtype):
    """Whole units from the counter: more sequences than a warp has lanes, some without
    queries, some without tokens; the counter is back at zero for the next call."""
    rnd = random.Random(3)
    kv_lens = [rnd.choice((0, 1, 50, 128, 300, 513)) for _ in range(150)]
    q_lens = [rnd.choice((0, 1, 7, 40, 300)) for _ in range(150)]
    if causal:
        kv_lens = [max(k, n) if k else 0 for k, n in zip(kv_lens, q_lens)]
    cache = Cache([kv_lens], hk, d, P, dtype, seed=9)
    q = queries(sum(q_lens), hq, d, dtype)
    ws = workspace(hc.query_workspace(cache.desc, len(q_lens), q.shape[0], hq, d, cache.tables[0].shape[1]))
    out, lse = run_query(cache, q, q_lens, kv_lens, causal, ws=ws)
    check_query(cache, q, q_lens, out, lse, causal, pick=[0, 6, 150])
    again, lse2 = run_query(cache, q, q_lens, kv_lens, causal, ws=ws)
    assert torch.equal(raw(out), raw(again)) and torch.equal(raw(lse), raw(lse2))


PREFIX = [
    # members, prefix_lens, own_lens of all, hq, hk, d, P, dtype, e4m3
    ([1], [1], [0], 1, 1, 64, 16, "bf16", False),
    ([4], [2000], [1, 64, 0, 17], 32, 8, 128, 64, "bf16", False),
    ([3, 0, 2], [100, 50, 1], [5, 6, 7, 300, 0, 9, 0], 8, 2, 128, 16, "fp16", False),
    ([40, 1], [700, 0], [i % 19 for i in range(41)], 16, 2, 128, 5, "bf16", False),
    ([2, 70], [33, 257], [3 * i for i in range(75)], 4, 4, 64, 1, "fp16", False),
    ([5, 6], [640, 90], [40] * 12, 8, 2, 256, 16, "bf16", False),
    ([3], [130], [20, 1, 0], 12, 1, 80, 16, "fp16", False),
    ([9, 3], [300, 1025], [11, 0, 5, 64, 70, 1, 2, 3, 4, 100, 200, 300], 8, 2, 128, 16, "fp16", True),
    ([7], [77], [9] * 8, 6, 3, 96, 7, "bf16", True),
    ([6], [513], [130] * 6, 64, 2, 192, 16, "bf16", False),
]


def run_prefix(c, q, members, prefix, own, ws=None, lead=0, **kw):
    starts = [lead]
    for n in members:
        starts.append(starts[-1] + n)
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 5.0, device="cuda")
    if ws is None:
        ws = workspace(hc.prefix_workspace(c.desc, q.shape[0], len(members), q.shape[1], q.shape[2],
                                           c.tables[0].shape[1], c.tables[1].shape[1]))
    hc.prefix_attention(c.kv, c.desc, 0, q, i32(starts), c.tables[0], i32(prefix), c.tables[1], i32(own), out, ws,
                        lse=lse, k_scale=c.k_scale, v_scale=c.v_scale, **kw)
    assert not hc.decode_gave_up(ws)
    return out, lse


def check_prefix(c, q, members, out, lse, lead=0, pick=None):
    k, v = c.plain()
    owner = [-1] * lead + [g for g, m in enumerate(members) for _ in range(m)]
    owner += [-1] * (q.shape[0] - len(owner))
    rows = [present((c.rows[0][g] if g >= 0 else []) + c.rows[1][b]) for b, g in enumerate(owner)]
    some = list(range(q.shape[0])) if pick is None else pick
    want = ref.attend(q[some], k, v, [rows[i] for i in some], q.shape[2] ** -0.5, c.k_scale, c.v_scale, joins=5)
    p_type = torch.bfloat16 if c.bufs[0].dtype == torch.bfloat16 else torch.float16
    ref.check_decode(out[some], want, q.dtype, p_type, lse=lse[some])


@pytest.mark.parametrize("c", PREFIX, ids=[f"{i}" for i in range(len(PREFIX))])
@pytest.mark.parametrize("holes", [False, True])
def test_prefix(c, holes):
    members, prefix, own, hq, hk, d, P, dtype, e4 = c
    cache = Cache([prefix, own], hk, d, P, dtype, e4, holes=holes)
    q = queries(len(own), hq, d, dtype)
    out, lse = run_prefix(cache, q, members, prefix, own)
    check_prefix(cache, q, members, out, lse)
    again, lse2 = run_prefix(cache, q, members, prefix, own)
    assert torch.equal(raw(out), raw(again)) and torch.equal(raw(lse), raw(lse2))


def test_prefix_without_groups():
    """Without groups, with groups of no sequence, with empty prefixes: decode_attention's
    results, within the bounds of both."""
    own = [0, 3, 700, 65]
    cache = Cache([[1], own], 2, 128, 16)
    q = queries(4, 8, 128, "bf16")
    ws = workspace(hc.prefix_workspace(cache.desc, 4, 0, 8, 128, 1, cache.tables[1].shape[1]))
    out, lse = torch.full_like(q, 7.0), torch.full((4, 8), 5.0, device="cuda")
    hc.prefix_attention(cache.kv, cache.desc, 0, q, i32([0]), cache.tables[0][:0], i32([]), cache.tables[1], i32(own), out,
                        ws, lse=lse)
    check_prefix(cache, q, [], out, lse)
    for members, prefix, lead in (([0], [1], 2), ([4], [0], 0)):
        again, lse2 = run_prefix(cache, q, members, prefix, own, lead=lead)
        assert torch.equal(raw(out), raw(again)) and torch.equal(raw(lse), raw(lse2))
    want, want_lse = torch.zeros_like(q), torch.zeros((4, 8), device="cuda")
    ws = workspace(hc.decode_workspace(cache.desc, 4, 8, 128, 128, cache.tables[1].shape[1]))
    hc.decode_attention(cache.kv, cache.desc, 0, q, cache.tables[1], i32(own), want, ws, lse=want_lse)
    check_prefix(cache, q, [], want, want_lse)


@pytest.mark.parametrize("hq,hk,d,P,dtype,e4", [(8, 2, 128, 16, "bf16", False), (6, 2, 64, 5, "fp16", False),
                                                (4, 1, 256, 64, "bf16", True)])
def test_prefix_long_own(hq, hk, d, P, dtype, e4):
    """Own tokens of several parts, around their limits."""
    members, prefix = [2, 3], [5000, 300]
    own = [9000, 4096, 4097, 8192, 1, 0, 12289]
    cache = Cache([prefix, own], hk, d, P, dtype, e4, seed=12)
    q = queries(len(own), hq, d, dtype)
    out, lse = run_prefix(cache, q, members, prefix, own)
    check_prefix(cache, q, members, out, lse)


# ---- merge ----------------------------------------------------------------------------

@pytest.mark.parametrize("n,h,d,parts,dtype", [
    (1, 1, 8, 1, "bf16"), (1, 32, 128, 2, "bf16"), (7, 3, 80, 3, "fp16"), (33, 5, 64, 4, "bf16"), (100, 7, 256, 5, "fp16"),
    (1000, 4, 192, 8, "bf16"), (5, 1, 512, 6, "fp16"), (257, 2, 24, 7, "bf16")])
def test_merge(n, h, d, parts, dtype):
    dt, g = DT[dtype], gen(n)
    # heads outside tokens in some parts, rows apart in others
    outs = [torch.randn((h, n, d), generator=g, device="cuda").to(dt).transpose(0, 1) if i % 2 else
            torch.randn((n, h, d + 8), generator=g, device="cuda").to(dt)[:, :, :d] for i in range(parts)]
    lses = [30 * torch.randn((n, h + 3), generator=g, device="cuda")[:, :h] for _ in range(parts)]
    for i, (x, z) in enumerate(zip(outs, lses)):
        none = torch.rand((n, h), generator=g, device="cuda") < 0.3
        z[none] = -INF
        x[none] = float("nan")                    # not read
    if parts > 1:
        for z in lses:
            z[n // 2] = -INF
    want_z = torch.logsumexp(torch.stack(lses).double(), 0)
    w = [torch.exp(z.double() - torch.where(want_z == -INF, 0.0, want_z)) for z in lses]
    terms = [torch.where((f > 0)[..., None], f[..., None] * x.double(), 0.0) for f, x in zip(w, outs)]
    want, spread = sum(terms), sum(t.abs() for t in terms)
    out, lse = torch.full((n, h, d), 7.0, dtype=dt, device="cuda"), torch.full((n, h), 5.0, device="cuda")
    hc.merge_attention(outs, lses, out, lse=lse)
    # a weight: the distance of two log-sums and its product with log2 e, two roundings of
    # up to |distance| (beyond 100 the weight is under 2^-144), 2^-22 of the exponential,
    # the same again in the sum, then products and sums of `parts`
    rel = 2 * (2 * 100 * 1.45 * ref.U32 + 2.0 ** -22) + (2 * parts + 4) * ref.U32
    tol = spread * rel + want.abs() * ref.UNIT[dt] * (1 + rel) + ref.TINY[dt] + 2.0 ** -120
    assert ((out.double() - want).abs() <= tol).all()
    none = want_z == -INF
    assert (lse[none] == -INF).all() and (out[none] == 0).all()
    assert ((lse.double() - want_z).abs() <= rel + 4 * want_z.abs() * ref.U32 + 2.0 ** -21)[~none].all()
    # in place of a part with its strides, without lse: the same bits
    twin = outs[-1].clone(memory_format=torch.preserve_format)
    hc.merge_attention(outs[:-1] + [twin], lses, twin)
    assert torch.equal(raw(twin.contiguous()), raw(out))


def test_merge_of_parts_is_the_whole():
    """Queries over a prefix in two parts and their own tokens, joined, against one call."""
    P, hq, hk, d = 16, 8, 2, 128
    kv, nq = 700, 50
    cache = Cache([[kv]], hk, d, P)
    q = queries(nq, hq, d, "bf16")
    whole, z = run_query(cache, q, [nq], [kv], causal=True)
    ws = workspace(hc.query_workspace(cache.desc, 1, nq, hq, d, cache.tables[0].shape[1]))
    outs, lses = [], []
    cut = [0, 256, 640, kv]
    for i in range(3):
        o, s = torch.zeros_like(q), torch.zeros((nq, hq), device="cuda")
        hc.query_attention(cache.kv, cache.desc, 0, q, i32([0, nq]), cache.tables[0][:, cut[i] // P:].contiguous(),
                           i32([cut[i + 1] - cut[i]]), o, ws, causal=i == 2, lse=s)
        outs.append(o)
        lses.append(s)
    out, lse = torch.zeros_like(q), torch.zeros((nq, hq), device="cuda")
    hc.merge_attention(outs, lses, out, lse=lse)
    check_query(cache, q, [nq], whole, z, causal=True)
    k, v = cache.plain()
    rows = [seen(cache.rows[0][0], nq, i, True, 0) for i in range(nq)]
    for i, (want, zz, _, bd) in enumerate(ref.attend(q, k, v, rows, d ** -0.5, joins=3)):
        # each part's out was rounded once, the whole once more
        tol = bd["spread"] * (2 * ref.UNIT[q.dtype] * 1.01 + bd["de"][:, None] + 2 * bd["n"] * ref.U32) + \
            want.abs() * ref.UNIT[q.dtype] * 1.01
        assert ((out[i].double() - want).abs() <= tol).all()
        assert ((lse[i].double() - zz).abs() <= bd["dl"] + 4 * zz.abs() * ref.U32 + 2.0 ** -20).all()
