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


# ---- what the calls allow beyond the usual one -------------------------------------------

@pytest.mark.parametrize("d,e4,dtype", [(128, False, "bf16"), (64, True, "bf16"), (256, False, "fp16")])
def test_query_strides(d, e4, dtype):
    """Heads outside tokens, rows apart, a slice of a wider table, one token, one head."""
    kv_lens, q_lens, hq, hk = [700, 130], [60, 9], 4, 2
    cache = Cache([kv_lens], hk, d, 16, dtype, e4, seed=3)
    n = sum(q_lens)
    q = queries(n, hq, d, dtype)
    want, want_z = run_query(cache, q, q_lens, kv_lens, True)
    check_query(cache, q, q_lens, want, want_z, True)
    q2 = q.transpose(0, 1).contiguous().transpose(0, 1)                  # [heads][tokens] in memory
    wide = torch.zeros((n, hq, d + 24), dtype=q.dtype, device="cuda")
    wide[:, :, :d] = q
    table = torch.full((2, cache.tables[0].shape[1] + 5), -7, dtype=torch.int32, device="cuda")
    table[:, 2:-3] = cache.tables[0]
    ws = workspace(hc.query_workspace(cache.desc, 2, n, hq, d, cache.tables[0].shape[1]))
    for x in (q2, wide[:, :, :d]):
        out = torch.full((hq, n, d), 7.0, dtype=q.dtype, device="cuda").transpose(0, 1)
        lse = torch.full((n, hq + 3), 5.0, device="cuda")
        hc.query_attention(cache.kv, cache.desc, 0, x, i32([0, 60, 69]), table[:, 2:-3], i32(kv_lens), out, ws, causal=True,
                           lse=lse[:, :hq], k_scale=cache.k_scale, v_scale=cache.v_scale)
        assert same(out.contiguous(), want) and same(lse[:, :hq].contiguous(), want_z)
        assert (lse[:, hq:] == 5.0).all()
    # one query head of one token, whatever its strides
    one = q[:1, :1].as_strided((1, 1, d), (3, 1, 1))
    small = Cache([[300]], 1, d, 16, dtype, e4, seed=5)
    out, lse = run_query(small, one, [1], [300])
    check_query(small, one, [1], out, lse)


@pytest.mark.parametrize("dtype,e4", [("bf16", False), ("fp16", False), ("fp16", True), ("bf16", True)])
@pytest.mark.parametrize("k_size,order", [(1.0, 0), (6.0, 0), (6.0, 1), (6.0, -1)])
def test_query_references(dtype, e4, k_size, order):
    """Scores that leave the reference far behind, in falling and rising order of the
    tokens, so that every block moves it."""
    kv, nq, hq, d = 900, 140, 2, 128
    cache = Cache([[kv]], 1, d, 16, dtype, e4, seed=7, k_size=k_size)
    q = queries(nq, hq, d, dtype, sharp=4.0)
    q[:] = q[:1, :1]                              # all alike, so that one order of the keys serves them
    if order:
        k, v = cache.bufs
        at = present(cache.rows[0][0])
        s = k.float()[at] @ q[0, 0].float()
        raw(k)[at] = raw(k)[at][s.argsort(descending=order < 0)]
    for causal in (False, True):
        out, lse = run_query(cache, q, [nq], [kv], causal)
        check_query(cache, q, [nq], out, lse, causal)


def same(a, b):
    return a.shape == b.shape and bool((raw(a) == raw(b)).all())


def test_query_infinities():
    """A key of +-infinity: its weight is none, or everything is NaN, for the queries that
    see it alone; a NaN key or value is seen by its kv head alone.  The rows of a warp move
    their references together, so a query before the key can be rounded otherwise than
    without it: it is held to the bounds against 64 bits."""
    kv, nq, hq, d = 300, 100, 4, 64
    cache = Cache([[kv]], 2, d, 16, seed=2)
    q = queries(nq, hq, d, "bf16").abs()          # positive: scores with +inf are +inf
    k, v = cache.bufs
    row = cache.rows[0][0]
    clean, z = run_query(cache, q, [nq], [kv], causal=True)
    check_query(cache, q, [nq], clean, z, causal=True)
    first = [seen(cache.rows[0][0], nq, i, True, 0) for i in range(50)]
    want = ref.attend(q[:50], *cache.plain(), first, d ** -0.5)
    for x in (float("inf"), -float("inf"), float("nan")):
        k[row[250], d:] = x                       # of kv head 1, seen by queries from 50 on
        out, lse = run_query(cache, q, [nq], [kv], causal=True)
        assert same(out[:, :2].contiguous(), clean[:, :2].contiguous()) and same(lse[:, :2].contiguous(), z[:, :2].contiguous())
        ref.check_decode(out[:50], want, q.dtype, torch.bfloat16, lse=lse[:50])
        if x == -float("inf"):                    # weight 0: as if the token were absent
            gone = [torch.tensor([r for r in seen(row, nq, i, True, 0).tolist() if r != row[250]], device="cuda")
                    for i in range(50, nq)]
            k[row[250], d:] = 0
            less = ref.attend(q[50:, 2:], *[t[:, 1:] for t in cache.plain()], gone, d ** -0.5)
            ref.check_decode(out[50:, 2:], less, q.dtype, torch.bfloat16, lse=lse[50:, 2:])
        else:
            assert out[50:, 2:].isnan().all() and lse[50:, 2:].isnan().all()


@pytest.mark.parametrize("d,P,dtype,e4", [(128, 16, "bf16", False), (128, 64, "fp16", False), (256, 128, "bf16", False),
                                          (64, 5, "fp16", False), (80, 32, "bf16", False), (128, 16, "fp16", True)])
def test_anything_before_the_windows(d, P, dtype, e4):
    """Tokens that no query's window reaches, K and V, hold NaN: in the box, block and page of
    the first one that counts too."""
    kv, nq, window = 500, 20, 100
    cache = Cache([[kv]], 2, d, P, dtype, e4, seed=4)
    q = queries(nq, 4, d, dtype)
    want, z = run_query(cache, q, [nq], [kv], causal=True, window=window)
    check_query(cache, q, [nq], want, z, causal=True, window=window)
    for buf in cache.bufs:
        raw(buf)[present(cache.rows[0][0][:kv - nq - window + 1])] = 0x7F if e4 else -1
    out, lse = run_query(cache, q, [nq], [kv], causal=True, window=window)
    assert same(out, want) and same(lse, z)


def test_bad_starts_and_lengths():
    """What the host cannot see: starts that descend or leave the rows, lengths below 0 and
    beyond the table.  Nothing outside the rows is written."""
    cache = Cache([[200, 200, 200]], 2, 64, 16)
    q = queries(20, 4, 64, "bf16")
    ws = workspace(hc.query_workspace(cache.desc, 3, 20, 4, 64, cache.tables[0].shape[1]))
    guard = torch.full((24, 4, 64), 7.0, dtype=q.dtype, device="cuda")
    for starts, lens in (([-5, 4, 9, 30], [200, 200, 200]), ([2 ** 31 - 1, 3, -2 ** 31, 5], [200, 200, 200]),
                         ([0, 10, 5, 20], [200, -1, 200]), ([0, 5, 10, 15], [-2 ** 31, 2 ** 31 - 1, 0])):
        out = guard.clone()
        for causal in (False, True):
            hc.query_attention(cache.kv, cache.desc, 0, q, i32(starts), cache.tables[0], i32(lens), out[2:22], ws,
                               causal=causal)
            assert not hc.decode_gave_up(ws)
            assert (out[:2] == 7.0).all() and (out[22:] == 7.0).all()
    out = guard.clone()
    hc.query_attention(cache.kv, cache.desc, 0, q, i32([0, 5, 10, 15]), cache.tables[0], i32([-9, 2 ** 31 - 1, 0]), out[:20], ws)
    assert (out[:5] == 0).all() and (out[10:15] == 0).all() and (out[15:] == 7.0).all()


def test_far_pages():
    """Pages whose elements lie beyond 2^32 of the buffer's first, by boxes and row by row."""
    for P, d in ((64, 128), (3, 128)):
        pages = 5_700_000_000 // (P * d)
        bufs = [torch.empty((pages * P, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        kv = 5 * P + 2
        table = i32([[pages - 1 - 7 * i for i in range(6)]])
        rows = torch.tensor([table[0, t // P].item() * P + t % P for t in range(kv)], device="cuda")
        for i, b in enumerate(bufs):
            b[(table[0].long()[:, None] * P + torch.arange(P, device="cuda")).flatten()] = float("nan")
            b[rows] = torch.randn((kv, d), generator=gen(i), device="cuda").bfloat16()
        q = queries(30, 4, d, "bf16")
        dd = desc(P, d, 2)
        ws = workspace(hc.query_workspace(dd, 1, 30, 4, d, 6))
        out, lse = torch.zeros_like(q), torch.zeros((30, 4), device="cuda")
        hc.query_attention(hc.DeviceKV(bufs, pages), dd, 0, q, i32([0, 30]), table, i32([kv]), out, ws, lse=lse)
        assert not hc.decode_gave_up(ws)
        k, v = (b[rows].view(kv, 1, d) for b in bufs)
        want = ref.attend(q, k, v, [torch.arange(kv, device="cuda")] * 30, d ** -0.5)
        ref.check_decode(out, want, q.dtype, torch.bfloat16, lse=lse)
        del bufs, k, v
        torch.cuda.empty_cache()


def test_one_workspace_for_many_shapes():
    """Calls of different shapes one after another over one workspace."""
    cache = Cache([[900, 40, 3000]], 2, 128, 16, seed=1)
    shapes = [([700, 1, 300], False), ([1, 1, 1], False), ([300, 40, 1], True), ([2000, 40, 2500], False)]
    n = max(hc.query_workspace(cache.desc, 3, sum(l), 8, 128, cache.tables[0].shape[1]) for l, _ in shapes)
    ws = workspace(n)
    first = []
    for _ in range(2):
        got = []
        for lens, causal in shapes:
            q = queries(sum(lens), 8, 128, "bf16", seed=sum(lens))
            got.append((q, lens, causal) + run_query(cache, q, lens, [900, 40, 3000], causal, ws=ws))
        if first:
            for a, b in zip(first, got):
                assert same(a[3], b[3]) and same(a[4], b[4])
        first = got
    for q, lens, causal, out, lse in first:
        check_query(cache, q, lens, out, lse, causal, pick=[0, 1, 39, 200])


def test_workspace_shared_with_decode():
    """One workspace for decode, query and prefix attention, one call after another: what
    each counts in is zero for the others, whatever their parts hold."""
    cache = Cache([[900] * 60, [200] * 60], 4, 128, 16, seed=3)
    hq, d, n = 8, 128, 60
    q = queries(n, hq, d, "bf16")
    many = queries(n * 300, hq, d, "bf16", seed=4)          # more units than whole ones need
    ws = workspace(max(hc.decode_workspace(cache.desc, n, hq, d, d, cache.tables[0].shape[1], True),
                       hc.query_workspace(cache.desc, n, n * 300, hq, d, cache.tables[0].shape[1]),
                       hc.prefix_workspace(cache.desc, n, 1, hq, d, cache.tables[0].shape[1], cache.tables[1].shape[1])))

    def calls(w):
        out, lse = torch.zeros_like(q), torch.zeros((n, hq), device="cuda")
        weight = torch.zeros(cache.tables[0].shape, device="cuda")
        hc.decode_attention(cache.kv, cache.desc, 0, q, cache.tables[0], i32([900] * n), out, w[0], lse=lse, weights=weight)
        big, big_lse = run_query(cache, many, [300] * n, [900] * n, ws=w[1])
        both, both_lse = torch.zeros_like(q), torch.zeros((n, hq), device="cuda")
        hc.prefix_attention(cache.kv, cache.desc, 0, q, i32([0, n]), cache.tables[0][:1], i32([900]), cache.tables[1],
                            i32([200] * n), both, w[2], lse=both_lse)
        return out, lse, weight, big, big_lse, both, both_lse

    want = calls([workspace(ws.numel()) for _ in range(3)])
    check_query(cache, many, [300] * n, want[3], want[4], pick=[0, 33])
    for _ in range(2):
        assert all(same(a, b) for a, b in zip(calls([ws] * 3), want))


@pytest.mark.parametrize("scale", [0.0, -0.2, 1e-30, 3.0])
@pytest.mark.parametrize("d,e4", [(64, False), (128, True), (256, False)])
def test_scales(scale, d, e4):
    cache = Cache([[300, 40]], 2, d, 16, "bf16", e4, seed=5)
    q = queries(70, 4, d, "bf16", sharp=0.5)
    out, lse = run_query(cache, q, [60, 10], [300, 40], True, scale=scale)
    check_query(cache, q, [60, 10], out, lse, True, scale=scale)


@pytest.mark.parametrize("hq,hk,d,causal", [(160, 1, 64, True), (300, 2, 128, False), (129, 1, 256, True)])
def test_many_heads_a_kv_head(hq, hk, d, causal):
    """More query heads on a kv head than a tile has rows."""
    cache = Cache([[200, 140]], hk, d, 16, seed=6)
    q = queries(13, hq, d, "bf16")
    out, lse = run_query(cache, q, [3, 10], [200, 140], causal)
    check_query(cache, q, [3, 10], out, lse, causal)


def test_largest_batch():
    """65,535 sequences of one query, most without tokens."""
    n, hq, d, P = 65535, 2, 64, 16
    cache = Cache([[33, 5, 16, 0]], 1, d, P, seed=7)
    width = cache.tables[0].shape[1]
    table, lens = torch.full((n, width), -1, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    at = [0, 31, 32, 4095, 4096, 40000, 65534]
    for j, i in enumerate(at):
        table[i], lens[i] = cache.tables[0][j % 4], [33, 5, 16, 0][j % 4]
    q = queries(n, hq, d, "bf16")
    out, lse = torch.full_like(q, 7.0), torch.full((n, hq), 5.0, device="cuda")
    ws = workspace(hc.query_workspace(cache.desc, n, n, hq, d, width))
    starts = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    for _ in range(2):
        hc.query_attention(cache.kv, cache.desc, 0, q, starts, table, lens, out, ws, lse=lse)
        assert not hc.decode_gave_up(ws)
    want = ref.attend(q[at], *cache.plain(), [present(cache.rows[0][j % 4]) for j in range(len(at))], d ** -0.5)
    ref.check_decode(out[at], want, q.dtype, torch.bfloat16, lse=lse[at])
    none = torch.ones(n, dtype=torch.bool, device="cuda")
    none[at] = False
    assert (out[none] == 0).all() and (lse[none] == -INF).all()
    # the same as sequences with tokens of their own, in no group
    wp = workspace(hc.prefix_workspace(cache.desc, n, 0, hq, d, width, width))
    out2, lse2 = torch.full_like(q, 7.0), torch.full((n, hq), 5.0, device="cuda")
    hc.prefix_attention(cache.kv, cache.desc, 0, q, i32([0]), table[:0], i32([]), table, lens, out2, wp, lse=lse2)
    ref.check_decode(out2[at], want, q.dtype, torch.bfloat16, lse=lse2[at])
    assert (out2[none] == 0).all() and (lse2[none] == -INF).all()


def test_captured_calls():
    """All three in a CUDA graph, replayed with other starts, lengths, tables and values."""
    hq, hk, d, P = 8, 2, 128, 16
    own, prefix = [40, 0, 300], [600]
    cache = Cache([prefix, own], hk, d, P, seed=6)
    q = queries(3, hq, d, "bf16")
    starts, lens, shared = i32([0, 3]), i32(own), i32(prefix)
    t0, t1 = cache.tables[0].clone(), cache.tables[1].clone()
    ws = workspace(hc.prefix_workspace(cache.desc, 3, 1, hq, d, t0.shape[1], t1.shape[1]))
    ws2 = workspace(hc.query_workspace(cache.desc, 1, 3, hq, d, t0.shape[1]))
    outs = [torch.zeros_like(q) for _ in range(3)]
    lses = [torch.zeros((3, hq), device="cuda") for _ in range(3)]

    def calls():
        hc.prefix_attention(cache.kv, cache.desc, 0, q, starts, t0, shared, t1, lens, outs[0], ws, lse=lses[0])
        hc.query_attention(cache.kv, cache.desc, 0, q, starts, t0, shared, outs[1], ws2, lse=lses[1])
        hc.merge_attention(outs[:2], lses[:2], outs[2], lse=lses[2])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for i, (s, n, l) in enumerate((([0, 3], [600], own), ([1, 2], [77], [1, 299, 0]), ([0, 0], [600], [40, 0, 300]),
                                   ([0, 3], [0], [0, 0, 0]))):
        starts.copy_(i32(s))
        shared.copy_(i32(n))
        lens.copy_(i32(l))
        q.copy_(queries(3, hq, d, "bf16", seed=20 + i))
        for x in outs[:2]:
            x.fill_(3.0)
        for z in lses[:2]:
            z.fill_(-INF)
        graph.replay()
        got = [x.clone() for x in outs + lses]
        for x in outs[:2]:
            x.fill_(3.0)
        for z in lses[:2]:
            z.fill_(-INF)
        calls()
        for a, b in zip(got, outs + lses):
            assert same(a, b)


def test_streams_at_once():
    """Calls on two streams, each with a workspace of its own."""
    cache = Cache([[2000, 700]], 2, 128, 16, seed=2)
    lens = [2000, 700]
    streams = [torch.cuda.Stream() for _ in range(2)]
    q = [queries(900, 8, 128, "bf16", seed=i) for i in range(2)]
    ws = [workspace(hc.query_workspace(cache.desc, 2, 900, 8, 128, cache.tables[0].shape[1])) for _ in range(2)]
    outs = [[torch.zeros_like(q[0]) for _ in range(6)] for _ in range(2)]
    starts, kl = i32([0, 300, 900]), i32(lens)
    torch.cuda.synchronize()
    for r in range(6):
        for i, st in enumerate(streams):
            hc.query_attention(cache.kv, cache.desc, 0, q[i], starts, cache.tables[0], kl, outs[i][r], ws[i], causal=i == 0,
                               stream=st)
    torch.cuda.synchronize()
    for i in range(2):
        want, z = run_query(cache, q[i], [300, 600], lens, i == 0)
        check_query(cache, q[i], [300, 600], want, z, i == 0, pick=[0, 299, 400])
        for x in outs[i]:
            assert same(x, want)


def test_grad_is_refused():
    cache = Cache([[100]], 2, 64, 16)
    q = queries(4, 4, 64, "bf16")
    ws = workspace(hc.query_workspace(cache.desc, 1, 4, 4, 64, cache.tables[0].shape[1]))
    out = torch.zeros_like(q).requires_grad_()
    with pytest.raises(ValueError, match="requires grad"):
        hc.query_attention(cache.kv, cache.desc, 0, q, i32([0, 4]), cache.tables[0], i32([100]), out, ws)
    with pytest.raises(ValueError, match="requires grad"):
        hc.merge_attention([q], [torch.zeros((4, 4), device="cuda")], out)
    with torch.no_grad():
        hc.query_attention(cache.kv, cache.desc, 0, q, i32([0, 4]), cache.tables[0], i32([100]), out, ws)


def test_serving_run():
    """A prompt whose prefix is in L2: the prefix is loaded, the rest appended and attended
    to in chunks; then samples that share the prompt are decoded, their own tokens
    appended; a two-level tree by queries and merge gives the same."""
    hq, hk, d, P, dt = 8, 2, 128, 16, torch.bfloat16
    prompt, cached, samples, steps = 300, 160, 3, 4
    g = gen(11)
    pages = 64
    bufs = [torch.full((pages * P, hk * d), float("nan"), dtype=dt, device="cuda") for _ in range(2)]
    kv = hc.DeviceKV(bufs, pages)
    k_all = torch.randn((prompt + samples * steps, hk, d), generator=g, device="cuda").to(dt)
    v_all = torch.randn((prompt + samples * steps, hk, d), generator=g, device="cuda").to(dt)
    with hc.Pool(1, 2, P, hk * d, 32, "page_first") as pool:
        # the prefix was computed before, backed up, and comes back into other pages
        first = list(range(40, 40 + cached // P))
        slots = torch.tensor([first[t // P] * P + t % P for t in range(cached)], device="cuda")
        hc.append_kv(kv, pool, 0, None, k_all[:cached], v_all[:cached], slots)
        torch.cuda.synchronize()
        pool.backup(kv, first, list(range(len(first))))
        torch.cuda.synchronize()
        for b in bufs:
            b.fill_(float("nan"))
        mine = [3, 9, 1, 30, 22, 5, 6, 17, 8, 11, 2, 33, 21, 50, 51, 52, 53, 54, 55]
        pool.load(kv, mine[:len(first)], list(range(len(first))))
        torch.cuda.synchronize()
        table = i32([mine])
        q = torch.randn((prompt - cached, hq, d), generator=g, device="cuda").to(dt)
        out, lse = torch.zeros_like(q), torch.zeros((prompt - cached, hq), device="cuda")
        ws = workspace(hc.query_workspace(pool, 1, 140, hq, d, len(mine)))
        for a, z in ((cached, 230), (230, prompt)):
            slots = torch.tensor([mine[t // P] * P + t % P for t in range(a, z)], device="cuda")
            hc.append_kv(kv, pool, 0, None, k_all[a:z], v_all[a:z], slots)
            part = slice(a - cached, z - cached)
            hc.query_attention(kv, pool, 0, q[part], i32([0, z - a]), table, i32([z]), out[part], ws, causal=True, lse=lse[part])
        want = ref.attend(q, k_all, v_all, [torch.arange(cached + i + 1, device="cuda") for i in range(prompt - cached)], d ** -0.5)
        ref.check_decode(out, want, dt, dt, lse=lse)
        # samples: each step stores one token of each, then attends
        own = i32([[40 + s] for s in range(samples)])
        wp = workspace(hc.prefix_workspace(pool, samples, 1, hq, d, len(mine), 1))
        for step in range(steps):
            rows = prompt + torch.arange(samples, device="cuda") * steps + step
            hc.append_kv(kv, pool, 0, None, k_all[rows], v_all[rows], (own[:, 0] * P + step).long())
            x = torch.randn((samples, hq, d), generator=g, device="cuda").to(dt)
            o, z = torch.zeros_like(x), torch.zeros((samples, hq), device="cuda")
            hc.prefix_attention(kv, pool, 0, x, i32([0, samples]), table, i32([prompt]), own, i32([step + 1] * samples), o, wp,
                                lse=z)
            seen_rows = [torch.cat([torch.arange(prompt, device="cuda"), prompt + s * steps + torch.arange(step + 1, device="cuda")])
                         for s in range(samples)]
            want = ref.attend(x, k_all, v_all, seen_rows, d ** -0.5, joins=2)
            ref.check_decode(o, want, dt, dt, lse=z)
        # the same from two levels, joined
        parts, sums = [torch.zeros_like(x) for _ in range(2)], [torch.zeros((samples, hq), device="cuda") for _ in range(2)]
        hc.query_attention(kv, pool, 0, x, i32([0, samples]), table, i32([prompt]), parts[0], ws, lse=sums[0])
        wd = workspace(hc.decode_workspace(pool, samples, hq, d, d, 1))
        hc.decode_attention(kv, pool, 0, x, own, i32([steps] * samples), parts[1], wd, lse=sums[1])
        both, z2 = torch.zeros_like(x), torch.zeros((samples, hq), device="cuda")
        hc.merge_attention(parts, sums, both, lse=z2)
        for i, (w, zz, _, bd) in enumerate(want):
            tol = bd["spread"] * (2 * ref.UNIT[dt] * 1.01 + bd["de"][:, None] + 2 * bd["n"] * ref.U32) + w.abs() * ref.UNIT[dt] * 1.01
            assert ((both[i].double() - w).abs() <= tol).all()
            assert ((z2[i].double() - zz).abs() <= bd["dl"] + 4 * zz.abs() * ref.U32 + 2.0 ** -20).all()
        for w in (ws, wp, wd):
            assert not hc.decode_gave_up(w)
