"""Query and prefix attention at the limits of what the calls accept, against plain 64-bit forms."""
import pytest
import torch

import serving_reference as ref
import tiered_kv_cache_gb300 as hc
from test_gpu_queries import Cache, DT, check_prefix, desc, gen, i32, present, queries, run_prefix, workspace

pytestmark = pytest.mark.gpu


def far_apart(P, d, width, at, lens):
    """A small cache, and tables of `width` pages of which those of the lists `at` are there:
    (kv, descriptor, table, rows of each sequence's tokens, k, v)."""
    pages = sum(map(len, at))
    bufs = [torch.randn((pages * P, d), generator=gen(i), device="cuda").bfloat16() for i in range(2)]
    table = torch.full((len(at), width), -1, dtype=torch.int32, device="cuda")
    rows, page = [], 0
    for b, some in enumerate(at):
        mine = []
        for x in some:
            table[b, x] = page
            mine += [page * P + t for t in range(P) if x * P + t < lens[b]]
            page += 1
        rows.append(torch.tensor(mine, dtype=torch.long, device="cuda"))
    return hc.DeviceKV(bufs, pages), desc(P, d, 2), table, rows, *[b.view(-1, 1, d) for b in bufs]


def test_prefix_own_tokens_of_the_longest_table():
    """As many own tokens as a table can have, most on absent pages, between sequences of a few."""
    P, d, hq, width = 1000, 64, 2, 2_147_482
    lens = [1500, width * P, 700, 2 ** 31 - 1, 0, 3]
    at = [[0, 1], [0, 4, 1_000_000, width - 1], [0], [5, width - 1], [], [0]]
    kv, dd, table, rows, k, v = far_apart(P, d, width, at, [min(n, width * P) for n in lens])
    q = queries(len(lens), hq, d, "bf16")
    ws = workspace(hc.prefix_workspace(dd, len(lens), 0, hq, d, 1, width))
    out, lse = torch.full_like(q, 7.0), torch.full((len(lens), hq), 5.0, device="cuda")
    hc.prefix_attention(kv, dd, 0, q, i32([0]), table[:0], i32([]), table, i32(lens), out, ws, lse=lse)
    assert not hc.decode_gave_up(ws)
    want = ref.attend(q, k, v, rows, d ** -0.5, joins=5)
    ref.check_decode(out, want, q.dtype, torch.bfloat16, lse=lse)


@pytest.mark.parametrize("causal", [False, True])
def test_query_unit_of_seconds(causal):
    """One sequence whose tokens keep its CTA busy for longer than any wait may last, among so many
    that CTAs take whole units."""
    P, d, hq, n, long = 1024, 64, 1, 700, 600_000_000
    width = -(-long // P)
    kv, dd, table, rows, k, v = far_apart(P, d, width, [[0, 3, 300_000, width - 2]], [long])
    lens = [10] * n
    lens[5] = long
    q = queries(n, hq, d, "bf16")
    ws = workspace(hc.query_workspace(dd, n, n, hq, d, width))
    out, lse = torch.full_like(q, 7.0), torch.full((n, hq), 5.0, device="cuda")
    hc.query_attention(kv, dd, 0, q, torch.arange(n + 1, dtype=torch.int32, device="cuda"), table.expand(n, -1), i32(lens), out,
                       ws, causal=causal, lse=lse)
    assert not hc.decode_gave_up(ws)
    want = ref.attend(q, k, v, [rows[0] if x == long else rows[0][:10] for x in lens], d ** -0.5)
    ref.check_decode(out, want, q.dtype, torch.bfloat16, lse=lse)


@pytest.mark.parametrize("dtype,big", [("bf16", 3.38e38), ("fp16", 65504.0)])
@pytest.mark.parametrize("parts", [1, 2, 3, 4, 5, 8])
def test_merge_of_the_largest_values(parts, dtype, big):
    """A weighted mean of elements near the type's largest lies among them."""
    n, h, d, dt = 33, 3, 72, DT[dtype]
    outs = [((1.0 - 0.3 * torch.rand((n, h, d), generator=gen(i), device="cuda")) * big).to(dt) for i in range(parts)]
    lses = [(0.0 if i % 2 else 3.0) * torch.randn((n, h), generator=gen(9 + i), device="cuda") for i in range(parts)]
    z = torch.stack(lses).double()
    w = torch.softmax(z, 0)[..., None]
    want = (w * torch.stack(outs).double()).sum(0)
    out, lse = torch.zeros((n, h, d), dtype=dt, device="cuda"), torch.zeros((n, h), device="cuda")
    hc.merge_attention(outs, lses, out, lse=lse)
    # weights as in test_merge, of log-sums up to 20 apart; then their sums and the rounding
    rel = 2 * (2 * 20 * 1.45 * ref.U32 + 2.0 ** -22) + (2 * parts + 4) * ref.U32
    assert ((out.double() - want).abs() <= want.abs() * (rel + ref.UNIT[dt] * (1 + rel))).all()
    assert ((lse.double() - torch.logsumexp(z, 0)).abs() <= rel + 4 * 20 * ref.U32 + 2.0 ** -21).all()


@pytest.mark.parametrize("own", [[0, 1, 40, 700], [9000, 0, 4097, 3]])
def test_prefix_of_the_largest_values(own):
    """Values near bf16's largest in the prefix and in every part of the sequences' own tokens."""
    prefix, members = [500, 90], [2, 1]
    cache = Cache([prefix, own], 2, 128, 16, seed=15)
    v = cache.bufs[1]
    big = (1.0 - 0.3 * torch.rand(v.shape, generator=gen(3), device="cuda")) * 3.38e38
    v.copy_(torch.where(v.isnan(), v, big.bfloat16()))
    q = queries(4, 8, 128, "bf16", sharp=0.3)
    out, lse = run_prefix(cache, q, members, prefix, own)
    check_prefix(cache, q, members, out, lse)


@pytest.mark.parametrize("starts,sure", [
    ([-5, 4, 9, 30], range(20)), ([0, 10, 5, 20], [*range(5), *range(10, 20)]), ([4, 4, 3, 4], [*range(3), *range(4, 20)]),
    ([2 ** 31 - 1, 3, -2 ** 31, 5], range(5, 20)), ([-2 ** 31, -1, 2 ** 31 - 1, 0], []), ([25, 24, 23, 22], range(20)),
])
@pytest.mark.parametrize("bad", [False, True])
def test_prefix_bad_starts_and_lengths(starts, sure, bad):
    """What the host cannot see: starts that descend or leave the rows, lengths below 0 and beyond
    the tables.  Nothing outside the rows is written, and rows in one group at most are right.  (Where
    starts descend, rows may lie in two groups or behind the last start.)"""
    n, hq, d, P = 20, 4, 64, 16
    prefix, own = [96, 96, 96], [(0, 16, 48, 33)[i % 4] for i in range(n)]
    cache = Cache([prefix, own], 2, d, P, seed=16)
    q = queries(n, hq, d, "bf16")
    lens, own_lens = list(prefix), list(own)
    if bad:
        lens[0], lens[2] = -1, 2 ** 31 - 1
        prefix[0] = 0
        for i in range(0, n, 4):                  # nothing, and a table's 3 pages
            own_lens[i] = -2 ** 31
            own_lens[i + 2] = 2 ** 31 - 1
    out = torch.full((n + 4, hq, d), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full((n + 4, hq), 5.0, device="cuda")
    ws = workspace(hc.prefix_workspace(cache.desc, n, 3, hq, d, cache.tables[0].shape[1], cache.tables[1].shape[1]))
    hc.prefix_attention(cache.kv, cache.desc, 0, q, i32(starts), cache.tables[0], i32(lens), cache.tables[1], i32(own_lens),
                        out[2:-2], ws, lse=lse[2:-2])
    assert not hc.decode_gave_up(ws)
    for x, v in ((out, 7.0), (lse, 5.0)):
        assert (x[:2] == v).all() and (x[-2:] == v).all()
    at = [min(max(s, 0), n) for s in starts]
    owner = [-1] * n
    for g in range(3):
        for b in range(at[g], max(at[g], at[g + 1])):
            owner[b] = g
    k, v = cache.plain()
    sure = list(sure)
    rows = [present((cache.rows[0][owner[b]][:prefix[owner[b]]] if owner[b] >= 0 else []) + cache.rows[1][b]) for b in sure]
    want = ref.attend(q[sure], k, v, rows, d ** -0.5, joins=5)
    ref.check_decode(out[2:-2][sure], want, q.dtype, torch.bfloat16, lse=lse[2:-2][sure])


def test_prefix_without_a_table():
    """No groups, and a prefix table without columns."""
    own = [0, 33, 200]
    cache = Cache([[], own], 2, 128, 16, seed=17)
    q = queries(3, 8, 128, "bf16")
    ws = workspace(hc.prefix_workspace(cache.desc, 3, 0, 8, 128, 0, cache.tables[1].shape[1]))
    out, lse = torch.full_like(q, 7.0), torch.full((3, 8), 5.0, device="cuda")
    none = torch.zeros((0, 0), dtype=torch.int32, device="cuda")
    hc.prefix_attention(cache.kv, cache.desc, 0, q, i32([0]), none, i32([]), cache.tables[1],
                        i32(own), out, ws, lse=lse)
    want = ref.attend(q, *cache.plain(), [present(r) for r in cache.rows[1]], 128 ** -0.5, joins=5)
    ref.check_decode(out, want, q.dtype, torch.bfloat16, lse=lse)
