"""The operators on the device pages (append, decode attention, eviction) against
plain 64-bit forms, at the sizes and masks where they can go wrong."""
import random

import numpy as np
import pytest
import torch

import serving_reference as ref
import tiered_kv_cache_gb300 as hc

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
E4 = torch.float8_e4m3fn


def desc(P, row, es, buffers=2, layers=1):
    return hc.PoolDesc(layers, buffers, P, es, row, 1, hc.LAYER_FIRST, 0, 0, 0)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def raw(t):
    """Bits, for comparisons in which NaN equals itself."""
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


# ---- append ---------------------------------------------------------------------

APPEND = [
    # n, hq, hk, d, P, dtype, e4m3, norm_q, norm_k, rot, off, interleaved, latent
    (1, 32, 8, 128, 64, "bf16", False, 128, 128, 128, 0, False, False),
    (1, 1, 1, 8, 1, "fp16", False, 8, 0, 0, 0, False, False),
    (7, 4, 2, 64, 16, "bf16", False, 0, 0, 64, 0, False, False),
    (33, 6, 3, 80, 5, "fp16", False, 80, 80, 40, 0, False, False),
    (50, 5, 1, 80, 16, "bf16", True, 80, 80, 40, 4, False, False),
    (129, 8, 8, 96, 16, "bf16", True, 96, 96, 48, 10, True, False),
    (64, 3, 1, 256, 64, "fp16", True, 256, 256, 256, 0, False, False),
    (19, 2, 2, 192, 7, "bf16", False, 64, 128, 100, 30, True, False),
    (40, 16, 1, 576, 64, "bf16", False, 0, 512, 64, 512, False, True),
    (3, 128, 1, 576, 64, "fp16", False, 576, 512, 64, 512, True, True),
    (11, 2, 1, 768, 4, "bf16", False, 768, 768, 768, 0, False, True),
    (1000, 14, 2, 128, 16, "fp16", False, 128, 128, 64, 64, False, False),
    (9, 4, 2, 128, 16, "bf16", True, 128, 128, 128, 0, True, False),
    (9, 5, 2, 256, 16, "fp16", False, 0, 256, 64, 192, True, False),
    (10, 6, 2, 256, 16, "bf16", False, 256, 64, 64, 64, False, False),
    (5, 3, 1, 64, 8, "fp16", True, 64, 0, 64, 0, True, False),
    (5, 2, 1, 64, 8, "bf16", False, 64, 64, 6, 2, False, False),
    (13, 9, 1, 128, 4, "bf16", False, 64, 128, 64, 0, False, False),
    (13, 2, 1, 128, 4, "fp16", False, 8, 120, 128, 0, False, False),
    (4000, 1, 1, 64, 4, "bf16", False, 64, 64, 0, 0, False, False),
    (6, 3, 1, 384, 4, "fp16", False, 384, 384, 384, 0, False, True),
]


def append_inputs(c, seed):
    n, hq, hk, d, P, dt, e4, nq, nk, rot, off, il, latent = c
    dt, g = DT[dt], gen(seed)
    per = hq + hk * (1 if latent else 2)
    fused = (2 * torch.randn((n, per, d), generator=g, device="cuda")).to(dt)
    q, k = fused[:, :hq], fused[:, hq:hq + hk]
    v = None if latent else fused[:, hq + hk:]
    pages = -(-n // P) + 2
    slots = torch.randperm(pages * P, generator=g, device="cuda")[:n]
    pos = torch.randint(0, 5000, (n,), generator=g, device="cuda")
    cs = None
    if rot:
        ang = torch.arange(5000, device="cuda", dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
        cs = torch.cat([ang.cos(), ang.sin()], 1).float()
    w = lambda m: (1 + 0.3 * torch.randn(m, generator=g, device="cuda")).to(dt) if m else None  # noqa: E731
    cache = E4 if e4 else dt
    bufs = [torch.full((pages * P, hk * d), 0x5A, dtype=torch.uint8, device="cuda").repeat(1, 1 if e4 else 2)
            .view(cache) for _ in range(1 if latent else 2)]
    return q, k, v, slots, pos, cs, w(nq), w(nk), bufs, pages


def check_append(c, q, k, v, slots, pos, cs, qw, kw, bufs, q_out, old, ks, vs, skip=None):
    n, hq, hk, d, P, dt, e4, nq, nk, rot, off, il, latent = c
    dt = DT[dt]
    skip = torch.zeros(n, dtype=torch.bool, device="cuda") if skip is None else skip
    rows = cs[pos.clamp(0, 4999)] if cs is not None else None
    y, err = ref.norm_rotate(q.double(), qw, rows, off, il, 1e-6)
    ok = (q_out.double() - y).abs() <= err + (y.abs() + err) * ref.UNIT[dt] + ref.TINY[dt]
    assert ok[~skip].all(), "q_out"
    live = (slots >= 0) & (slots < old[0].shape[0]) & ~skip
    at = slots[live]
    cache = bufs[0].dtype
    rest = torch.ones(old[0].shape[0], dtype=torch.bool, device="cuda")
    rest[at] = False
    stored = [ref.norm_rotate(k.double(), kw, rows, off, il, 1e-6) + (ks,)]
    if v is not None:
        stored.append((v.double(), torch.zeros_like(v, dtype=torch.float64), vs))
    for buf, before, (y, err, sc) in zip(bufs, old, stored):
        y, err = y[live].reshape(-1, hk * d) / sc, err[live].reshape(-1, hk * d) / sc
        if cache == E4:
            err = err + y.abs() * ref.U32
            y = y.clamp(-448, 448)
        got = raw(buf)[at].view(cache).double()
        assert ((got - y).abs() <= err + (y.abs() + err) * ref.UNIT[cache] + ref.TINY[cache]).all(), "cache"
        assert torch.equal(raw(buf)[rest], raw(before)[rest]), "rows that no token has were written"


@pytest.mark.parametrize("c", APPEND, ids=[f"{i}" for i in range(len(APPEND))])
def test_append(c):
    q, k, v, slots, pos, cs, qw, kw, bufs, pages = append_inputs(c, 3)
    old = [b.clone() for b in bufs]
    ks, vs = (0.03, 0.05) if c[6] else (1.0, 1.0)
    q_out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
    kv = hc.DeviceKV(bufs, pages)
    dd = desc(c[4], c[2] * c[3], bufs[0].element_size(), len(bufs))
    before = hc.launch_count()
    hc.append_kv(kv, dd, 0, q, k, v, slots, q_out=q_out, positions=pos if cs is not None else None, cos_sin=cs,
                 rot_offset=c[10], interleaved=c[11], q_weight=qw, k_weight=kw, k_scale=ks, v_scale=vs)
    assert hc.launch_count() == before + 1
    check_append(c, q, k, v, slots, pos, cs, qw, kw, bufs, q_out, old, ks, vs)
    # in place (q is a view of the fused tensor): the same bits
    keep = q_out.clone()
    hc.append_kv(kv, dd, 0, q, None, None, None, positions=pos if cs is not None else None, cos_sin=cs,
                 rot_offset=c[10], interleaved=c[11], q_weight=qw)
    assert torch.equal(raw(q), raw(keep))


def test_append_tables_at_any_row():
    """A table that starts between 16-byte boundaries, and token rows that are not
    next to one another."""
    c = (31, 4, 2, 128, 8, "bf16", False, 128, 128, 126, 2, False, False)
    q, k, v, slots, pos, cs, qw, kw, bufs, pages = append_inputs(c, 6)
    wide = torch.zeros((5001, 126), device="cuda")
    wide[1:] = cs
    wide[0] = float("nan")
    old = [b.clone() for b in bufs]
    q_out = torch.zeros((31, 4, 128), dtype=q.dtype, device="cuda")
    hc.append_kv(hc.DeviceKV(bufs, pages), desc(8, 256, 2), 0, q, k, v, slots, q_out=q_out, positions=pos,
                 cos_sin=wide[1:], rot_offset=2, q_weight=qw, k_weight=kw)
    check_append(c, q, k, v, slots, pos, cs, qw, kw, bufs, q_out, old, 1.0, 1.0)


def test_append_skips_rows():
    """Slots and positions outside their ranges: nothing is stored there, and
    rows whose position is outside are left as they were."""
    c = (24, 4, 2, 64, 8, "bf16", False, 64, 64, 64, 0, False, False)
    q, k, v, slots, pos, cs, qw, kw, bufs, pages = append_inputs(c, 5)
    slots[2], slots[3], slots[4], slots[5] = -1, pages * 8, 2 ** 62, -2 ** 63
    pos[7], pos[8], pos[9] = -1, 5000, 2 ** 61
    old = [b.clone() for b in bufs]
    q_out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    hc.append_kv(hc.DeviceKV(bufs, pages), desc(8, 128, 2), 0, q, k, v, slots, q_out=q_out, positions=pos, cos_sin=cs,
                 q_weight=qw, k_weight=kw)
    skip = (pos < 0) | (pos >= 5000)
    check_append(c, q, k, v, slots, pos, cs, qw, kw, bufs, q_out, old, 1.0, 1.0, skip)
    assert (q_out[skip] == 7.0).all()


LONG_APPEND = [
    # several tokens to a warp, and warps that begin and end within one
    (3001, 5, 3, 64, 16, "bf16", False, 64, 64, 64, 0, False, False),
    (4099, 1, 1, 64, 16, "fp16", True, 0, 64, 64, 0, True, False),
    (2500, 9, 2, 128, 16, "fp16", False, 128, 128, 128, 0, False, False),
    (1999, 4, 5, 128, 7, "bf16", True, 128, 64, 64, 64, False, False),
    (2311, 6, 1, 128, 16, "bf16", False, 0, 0, 0, 0, False, False),
    (1777, 3, 2, 256, 16, "bf16", False, 256, 256, 256, 0, False, False),
    (1501, 5, 1, 256, 16, "fp16", True, 128, 256, 128, 64, True, False),
    (1409, 7, 1, 576, 16, "bf16", False, 0, 512, 64, 512, False, True),
    (911, 17, 1, 576, 64, "fp16", True, 576, 512, 64, 448, True, True),
    (1205, 2, 1, 576, 64, "bf16", False, 512, 512, 0, 0, False, True),
]


@pytest.mark.parametrize("c", LONG_APPEND, ids=[f"{i}" for i in range(len(LONG_APPEND))])
def test_append_many_tokens(c):
    """Runs of tokens through each shape, some of whose slots or positions are outside."""
    q, k, v, slots, pos, cs, qw, kw, bufs, pages = append_inputs(c, 11)
    n, hq, hk, d, P = c[:5]
    slots[::5] = -1
    slots[3::17] = pages * P
    skip = torch.zeros(n, dtype=torch.bool, device="cuda")
    if cs is not None:
        skip[2::7] = True
        skip[40:43] = True
        pos[2::7] = -1
        pos[40:43] = 5000
    old = [b.clone() for b in bufs]
    ks, vs = (0.03, 0.05) if c[6] else (1.0, 1.0)
    q_out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    hc.append_kv(hc.DeviceKV(bufs, pages), desc(P, hk * d, bufs[0].element_size(), len(bufs)), 0, q, k, v, slots,
                 q_out=q_out, positions=pos if cs is not None else None, cos_sin=cs, rot_offset=c[10],
                 interleaved=c[11], q_weight=qw, k_weight=kw, k_scale=ks, v_scale=vs)
    check_append(c, q, k, v, slots, pos, cs, qw, kw, bufs, q_out, old, ks, vs, skip)
    assert (q_out[skip] == 7.0).all()
    hc.append_kv(hc.DeviceKV(bufs, pages), desc(P, hk * d, bufs[0].element_size(), len(bufs)), 0, q, None, None, None,
                 positions=pos if cs is not None else None, cos_sin=cs, rot_offset=c[10], interleaved=c[11],
                 q_weight=qw)
    assert torch.equal(raw(q)[~skip], raw(q_out)[~skip])


def test_append_heads_outer_and_extremes():
    """Heads outside tokens, e4m3 saturation, infinities and NaN."""
    g = gen(9)
    k = torch.randn((2, 5, 64), generator=g, device="cuda").to(torch.float16).transpose(0, 1)
    k = k.clone(memory_format=torch.preserve_format)
    v = torch.full((5, 2, 64), 60000.0, dtype=torch.float16, device="cuda")
    v[1], v[2, 0], v[3, 1] = -60000.0, float("inf"), float("nan")
    bufs = [torch.zeros((16, 128), dtype=torch.uint8, device="cuda").view(E4) for _ in range(2)]
    slots = torch.arange(5, device="cuda") * 3
    hc.append_kv(hc.DeviceKV(bufs, 4), desc(4, 128, 1), 0, None, k, v, slots, k_scale=0.5, v_scale=2.0)
    got = bufs[1].float().view(16, 2, 64)[slots]
    assert (got[0] == 448).all() and (got[1] == -448).all() and (got[2, 0] == 448).all()
    assert got[3, 1].isnan().all() and (got[3, 0] == 448).all()
    want = (k.float() / 0.5).to(E4).float().reshape(5, 128)
    assert torch.equal(bufs[0].float()[slots], want)


# ---- decode ---------------------------------------------------------------------

def decode_inputs(lens, hq, hk, d, P, dtype="bf16", e4=False, latent=False, seed=1, holes=False, sharp=2.0, width=0,
                  spare=3):
    """Caches filled with NaN, in which only the tokens of the sequences are
    written, and page tables whose other entries are out of range."""
    g, dt = gen(seed), DT[dtype]
    rnd = random.Random(seed)
    counts = [-(-n // P) for n in lens]
    width = max(width, max(counts), 1)
    Dp = sum(counts) + spare
    order = list(range(Dp))
    rnd.shuffle(order)
    bad = [-1, Dp, 2 ** 31 - 1, -2 ** 31, Dp + 17]
    table, at = [], 0
    for c in counts:
        row = order[at:at + c]
        at += c
        if holes:
            row = [p if rnd.random() < 0.7 else rnd.choice(bad) for p in row]
        table.append(row + [rnd.choice(bad) for _ in range(width - c)])
    row_e = d if latent else hk * d
    es = 1 if e4 else 2
    bufs = []
    for _ in range(1 if latent else 2):
        b = torch.full((Dp * P, row_e * es), 0x7F if e4 else 0xFF, dtype=torch.uint8, device="cuda")
        b = b.view(E4 if e4 else dt)
        for i, n in enumerate(lens):
            for j, p in enumerate(table[i][:counts[i]]):
                m = min(P, n - j * P)
                if 0 <= p < Dp:
                    x = torch.randn((m, row_e), generator=g, device="cuda")
                    if e4:
                        b.view(torch.uint8)[p * P:p * P + m] = (8 * x).to(E4).view(torch.uint8)
                    else:
                        b[p * P:p * P + m] = x.to(dt)
        bufs.append(b)
    q = (sharp * torch.randn((len(lens), hq, d), generator=g, device="cuda")).to(dt)
    clean = [[p if 0 <= p < Dp else -1 for p in r] for r in table]
    return {"q": q, "bufs": bufs, "table": torch.tensor(table, dtype=torch.int32, device="cuda"), "clean": clean,
            "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"), "Dp": Dp, "width": width, "dt": dt,
            "ks": 0.125 if e4 else 1.0, "vs": 0.25 if e4 else 1.0, "desc": desc(P, row_e, es, len(bufs)),
            "kv": hc.DeviceKV(bufs, Dp)}


def workspace(s, hq, d, dv, weights):
    n = hc.decode_workspace(s["desc"], s["q"].shape[0], hq, d, dv, s["width"], weights)
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


def run_decode(lens, hq, hk, d, P, dtype="bf16", e4=False, latent=False, window=0, weights=True, holes=False,
               sharp=2.0, seed=1, scale=None, width=0):
    s = decode_inputs(lens, hq, hk, d, P, dtype, e4, latent, seed, holes, sharp, width)
    dv = 512 if latent else d
    scale = d ** -0.5 if scale is None else scale
    out = torch.full((len(lens), hq, dv), 3.0, dtype=s["dt"], device="cuda")
    lse = torch.full((len(lens), hq), 3.0, device="cuda")
    w = torch.rand((len(lens), s["width"]), generator=gen(8), device="cuda") if weights else None
    before = w.clone() if weights else None
    ws = workspace(s, hq, d, dv, weights)
    hc.decode_attention(s["kv"], s["desc"], 0, s["q"], s["table"], s["lens"], out, ws, scale=scale, window=window,
                        weights=w, decay=0.5, lse=lse, k_scale=s["ks"], v_scale=s["vs"])
    k = s["bufs"][0].view(s["Dp"] * P, -1, d)
    v = k[..., :512] if latent else s["bufs"][1].view(s["Dp"] * P, -1, d)
    want = ref.decode(s["q"], k, v, s["clean"], [max(0, n) for n in lens], P, scale, window, s["ks"], s["vs"])
    ref.check_decode(out, want, s["dt"], torch.float16 if e4 else s["dt"], lse, w, before, 0.5)
    return s, out


DECODE = [
    # lens, hq, hk, d, P, dtype, e4m3
    ([1], 1, 1, 64, 1, "bf16", False),
    ([1, 0, 2], 4, 2, 64, 16, "fp16", False),
    ([15, 16, 17, 31, 32, 33], 8, 2, 64, 16, "bf16", False),
    ([4097], 32, 8, 128, 64, "bf16", False),
    ([63, 64, 65, 129, 1000, 0, 5], 32, 8, 128, 64, "fp16", False),
    ([300, 7, 2500], 6, 2, 96, 5, "bf16", False),
    ([700, 13], 5, 1, 80, 16, "fp16", False),
    ([257, 1024], 3, 3, 72, 1, "bf16", False),
    ([900, 30], 16, 1, 256, 128, "bf16", False),
    ([513, 100], 24, 1, 192, 300, "fp16", False),
    ([513, 100], 40, 2, 128, 16, "bf16", False),
    ([1, 0, 1500, 31], 8, 2, 128, 16, "fp16", True),
    ([4097, 255], 32, 8, 128, 64, "bf16", True),
    ([300, 7, 1100], 12, 2, 96, 5, "bf16", True),
    ([900, 30], 16, 1, 256, 1, "fp16", True),
    ([513, 100], 20, 1, 192, 300, "bf16", True),
    ([77, 2000], 7, 1, 16, 16, "bf16", True),
    ([77, 2000], 7, 7, 8, 16, "bf16", False),
    ([33000, 5, 9000], 8, 2, 128, 16, "bf16", False),
    ([3 + 37 * i % 400 for i in range(70)], 8, 2, 64, 16, "fp16", False),
]


@pytest.mark.parametrize("c", DECODE, ids=[f"{i}" for i in range(len(DECODE))])
def test_decode(c):
    run_decode(*c)


@pytest.mark.parametrize("c", [
    ([1], 16, 64), ([0, 1, 63, 64, 65], 16, 64), ([129, 4000, 127, 0, 128], 128, 64), ([1000, 17], 20, 5),
    ([300, 9], 64, 1), ([513, 2049], 8, 300), ([20000], 33, 16), ([400 + 3 * i for i in range(40)], 16, 16),
], ids=[f"{i}" for i in range(8)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_decode_latent(c, dtype):
    run_decode(c[0], c[1], 1, 576, c[2], dtype, latent=True, scale=192 ** -0.5)


@pytest.mark.parametrize("latent", [False, True])
def test_decode_many_sequences(latent):
    """More sequences than a CTA has threads, most of them short or empty."""
    lens = [(7 * i) % 41 if i % 5 else 0 for i in range(700)]
    lens[333] = 900
    run_decode(lens, 4, 2, 576 if latent else 64, 16, "bf16", latent=latent)


@pytest.mark.parametrize("latent", [False, True])
@pytest.mark.parametrize("n", [16, 17, 100, 2400, 4864, 4880, 20000])
def test_decode_one_sequence(latent, n):
    """One sequence dealt to ever more CTAs: fewer tiles than CTAs, as many, more."""
    run_decode([n], 8, 1, 576 if latent else 128, 64, "fp16", latent=latent)


@pytest.mark.parametrize("latent,e4", [(False, False), (False, True), (True, False)])
@pytest.mark.parametrize("window", [1, 16, 100, 1023])
def test_decode_window_and_absent_pages(latent, e4, window):
    """A window and absent pages, among them sequences of which nothing is left."""
    run_decode([1, 100, 1000, 0, 2040, 17], 8, 2, 576 if latent else 64, 16, "bf16", e4, latent, window=window,
               holes=True, seed=window)


@pytest.mark.parametrize("latent,e4", [(False, False), (False, True), (True, False)])
def test_decode_sharp_scores_and_negative_scale(latent, e4):
    d = 576 if latent else 128
    run_decode([700, 64, 2], 8, 2, d, 16, "fp16", e4, latent, sharp=40.0)
    run_decode([700, 64, 2], 8, 2, d, 16, "bf16", e4, latent, scale=-0.1)


def plain_call(s, out, ws, **kw):
    hc.decode_attention(s["kv"], s["desc"], 0, s["q"], s["table"], s["lens"], out, ws, k_scale=s["ks"],
                        v_scale=s["vs"], **kw)


@pytest.mark.parametrize("latent", [False, True])
def test_decode_lengths_outside_the_table(latent):
    """Negative lengths count as 0, lengths behind the table as its end."""
    s = decode_inputs([320, 320, 100], 4, 2, 576 if latent else 64, 16, latent=latent)
    dv = 512 if latent else 64
    ws = workspace(s, 4, s["q"].shape[2], dv, False)
    a, b = (torch.empty((3, 4, dv), dtype=s["dt"], device="cuda") for _ in range(2))
    s["lens"][0], s["lens"][1] = -5, 320
    plain_call(s, a, ws)
    s["lens"][0], s["lens"][1] = -2 ** 31, 2 ** 31 - 1
    plain_call(s, b, ws)
    assert torch.equal(a, b) and (a[0] == 0).all() and (a[1] != 0).any()


@pytest.mark.parametrize("latent", [False, True])
def test_decode_strides(latent):
    """q and out as views of wider tensors, tables, lse and weights with longer
    rows, one layer of several: the same bits as contiguous arguments, and
    nothing else written."""
    d, hq, P = (576, 6, 16) if latent else (64, 6, 16)
    dv = 512 if latent else d
    s = decode_inputs([100, 33, 650], hq, 2, d, P, latent=latent)
    ws = workspace(s, hq, d, dv, True)
    out = torch.empty((3, hq, dv), dtype=s["dt"], device="cuda")
    lse = torch.empty((3, hq), device="cuda")
    w = torch.zeros((3, s["width"]), device="cuda")
    plain_call(s, out, ws, weights=w, lse=lse)
    wide_q = torch.full((3, hq + 4, d + 16), float("nan"), dtype=s["dt"], device="cuda")
    wide_q[:, 2:2 + hq, 8:8 + d] = s["q"]
    wide_o = torch.full((hq, 3, dv + 24), 5.0, dtype=s["dt"], device="cuda")
    wide_t = torch.full((3, s["width"] + 7), -9, dtype=torch.int32, device="cuda")
    wide_t[:, 3:3 + s["width"]] = s["table"]
    wide_l = torch.full((3, hq + 3), 5.0, device="cuda")
    wide_w = torch.full((3, s["width"] + 5), 5.0, device="cuda")
    wide_w[:, 1:1 + s["width"]] = 0
    layers = 3
    bufs = []
    for b in s["bufs"]:
        bufs += [torch.full_like(b, float("nan")), b, torch.full_like(b, float("nan"))]
    dd = hc.PoolDesc(layers, len(s["bufs"]), P, 2, s["desc"].row_elems, 1, hc.PAGE_FIRST, 0, 0, 0)
    hc.decode_attention(hc.DeviceKV(bufs, s["Dp"]), dd, 1, wide_q[:, 2:2 + hq, 8:8 + d], wide_t[:, 3:3 + s["width"]],
                        s["lens"], wide_o.transpose(0, 1)[:, :, 16:16 + dv], ws, weights=wide_w[:, 1:1 + s["width"]],
                        lse=wide_l[:, 2:2 + hq])
    assert torch.equal(wide_o.transpose(0, 1)[:, :, 16:16 + dv], out)
    assert (wide_o[..., :16] == 5).all() and (wide_o[..., 16 + dv:] == 5).all()
    assert torch.equal(wide_l[:, 2:2 + hq], lse) and (wide_l[:, :2] == 5).all() and (wide_l[:, 2 + hq:] == 5).all()
    assert torch.equal(wide_w[:, 1:1 + s["width"]], w) and (wide_w[:, 0] == 5).all()
    # a broadcast query
    one = s["q"][:1, :1].expand(3, hq, d)
    a, b = torch.empty_like(out), torch.empty_like(out)
    s["q"] = one
    plain_call(s, a, ws)
    s["q"] = one.contiguous()
    plain_call(s, b, ws)
    assert torch.equal(a, b)


@pytest.mark.parametrize("latent", [False, True])
def test_decode_far_pages(latent):
    """Pages whose byte and element offsets pass 32 bits."""
    d = 576 if latent else 128
    row, P, hk = (576, 64, 1) if latent else (1024, 64, 8)
    dp = (5 << 30) // row // P
    buf = torch.empty((dp * P, row), dtype=torch.bfloat16, device="cuda")
    pages = [dp - 1, 0, dp - 2, dp // 2, dp - 3]
    rows = torch.cat([torch.arange(p * P, (p + 1) * P, device="cuda") for p in pages])
    vals = torch.randn((rows.numel(), row), generator=gen(4), device="cuda").to(torch.bfloat16)
    buf[rows] = vals
    small = torch.cat([vals])
    q = torch.randn((1, 8, d), generator=gen(5), device="cuda").to(torch.bfloat16)
    dv = 512 if latent else d
    outs = []
    for b, n, t in ((buf, dp, pages), (small, len(pages), list(range(len(pages))))):
        bufs = [b] if latent else [b, b]
        dd = desc(P, row, 2, len(bufs))
        out = torch.empty((1, 8, dv), dtype=torch.bfloat16, device="cuda")
        ws = torch.zeros(hc.decode_workspace(dd, 1, 8, d, dv, len(pages)), dtype=torch.uint8, device="cuda")
        hc.decode_attention(hc.DeviceKV(bufs, n), dd, 0, q, torch.tensor([t], dtype=torch.int32, device="cuda"),
                            torch.tensor([P * 5 - 3], dtype=torch.int32, device="cuda"), out, ws)
        outs.append(out)
    assert torch.equal(*outs)
    if not latent:        # the append finds the same rows
        slots = rows[torch.randperm(rows.numel(), generator=gen(6), device="cuda")[:50]]
        k = torch.randn((50, 8, 128), generator=gen(7), device="cuda").to(torch.bfloat16)
        hc.append_kv(hc.DeviceKV([buf, buf], dp), desc(P, row, 2), 0, None, k, k, slots)
        assert torch.equal(buf[slots], k.reshape(50, row))


@pytest.mark.parametrize("latent", [False, True])
def test_decode_repeats_streams_and_one_workspace(latent):
    """The same bits each time, on any stream, with a workspace that calls of
    other shapes used in between."""
    d, dv = (576, 512) if latent else (128, 128)
    big = decode_inputs([5000, 70, 0, 3000], 16, 4, d, 16, latent=latent, seed=2)
    small = decode_inputs([90, 4] * 9, 16, 4, d, 16, latent=latent, seed=3, width=400)
    n = max(workspace(x, 16, d, dv, True).numel() for x in (big, small))
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    first = {}
    streams = [None, torch.cuda.Stream(), torch.cuda.Stream()]
    for turn in range(6):
        stream = streams[turn % 3]
        for name, x in (("big", big), ("small", small)):
            out = torch.empty((x["q"].shape[0], 16, dv), dtype=x["dt"], device="cuda")
            w = torch.zeros((x["q"].shape[0], x["width"]), device="cuda")
            torch.cuda.synchronize()
            plain_call(x, out, ws, weights=w, stream=stream)
            torch.cuda.synchronize()
            if name in first:
                assert torch.equal(first[name][0], out) and torch.equal(first[name][1], w)
            first[name] = (out, w)


@pytest.mark.parametrize("latent", [False, True])
def test_decode_graphs(latent):
    """Captured once, replayed with other lengths and pages; two graphs with a
    workspace each replayed together."""
    d, dv = (576, 512) if latent else (128, 128)
    lens = [2000, 64, 900]
    sets = [decode_inputs(lens, 8, 2, d, 16, latent=latent, seed=i) for i in (11, 12)]
    graphs, outs, ws, wts = [], [], [], []
    for s in sets:
        o = torch.empty((3, 8, dv), dtype=s["dt"], device="cuda")
        k = workspace(s, 8, d, dv, True)
        w = torch.zeros((3, s["width"]), device="cuda")
        plain_call(s, o, k, weights=w)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            plain_call(s, o, k, weights=w, stream=torch.cuda.current_stream())
        graphs.append(g)
        outs.append(o)
        ws.append(k)
        wts.append(w)
    streams = [torch.cuda.Stream() for _ in sets]
    for shorter in (0, 3, 61):
        want = []
        for s, w in zip(sets, wts):
            s["lens"].copy_(torch.tensor([n - shorter for n in lens], dtype=torch.int32))
            w.zero_()
            o, w2 = torch.empty((3, 8, dv), dtype=s["dt"], device="cuda"), torch.zeros_like(w)
            plain_call(s, o, workspace(s, 8, d, dv, True), weights=w2)
            want.append((o, w2))
        torch.cuda.synchronize()
        for _ in range(20):
            for w in wts:
                w.zero_()
            torch.cuda.synchronize()
            for g, st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    g.replay()
            torch.cuda.synchronize()
            for o, w, (a, b) in zip(outs, wts, want):
                assert torch.equal(o, a) and torch.equal(w, b)


def test_first_calls_in_a_capture():
    """Every operator's first call in a process, captured into a graph."""
    import subprocess
    import sys
    code = """
import torch, tiered_kv_cache_gb300 as hc, test_gpu_serving as t
c = t.APPEND[0]
q, k, v, slots, pos, cs, qw, kw, bufs, pages = t.append_inputs(c, 3)
s = [t.decode_inputs([300, 40], 4, 2, 128, 16), t.decode_inputs([300, 40], 4, 2, 576, 16, latent=True)]
dv = [128, 512]
outs = [torch.zeros((2, 4, n), dtype=x['dt'], device='cuda') for x, n in zip(s, dv)]
ws = [t.workspace(x, 4, x['q'].shape[2], n, True) for x, n in zip(s, dv)]
w = [torch.zeros((2, x['width']), device='cuda') for x in s]
table = torch.arange(12, dtype=torch.int32, device='cuda').view(2, 6)
wt = torch.rand((2, 6), device='cuda')
lens, keep = (torch.full((2,), n, dtype=torch.int32, device='cuda') for n in (96, 3))
vic, cnt = torch.full((2, 6), -1, dtype=torch.int32, device='cuda'), torch.zeros(2, dtype=torch.int32, device='cuda')
ot, ow, ol = torch.zeros_like(table), torch.zeros_like(wt), torch.zeros_like(lens)
q_out = torch.zeros_like(q)
torch.cuda.synchronize()
def go(stream):
    hc.append_kv(hc.DeviceKV(bufs, pages), t.desc(64, 1024, 2), 0, q, k, v, slots, q_out=q_out, positions=pos,
                 cos_sin=cs, q_weight=qw, k_weight=kw, stream=stream)
    for x, o, y, z in zip(s, outs, ws, w):
        t.plain_call(x, o, y, weights=z, decay=0.0, stream=stream)
    hc.evict_pages(16, table, lens, wt, keep, vic, cnt, out_table=ot, out_weights=ow, out_lens=ol, stream=stream)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    go(torch.cuda.current_stream())
everything = [q_out, *bufs, *outs, *w, vic, cnt, ot, ow, ol]
for x in everything: x.zero_()
g.replay()
torch.cuda.synchronize()
first = [x.clone() for x in everything]
for x in everything: x.zero_()
go(None)
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(first, everything))
assert outs[0].any() and outs[1].any() and cnt.tolist() == [3, 3]
assert not any(hc.decode_gave_up(x) for x in ws)
print('ok')
"""
    import os
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([os.path.dirname(here), here]))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def test_decode_random_corpus():
    """Random shapes over the documented ranges."""
    rnd = random.Random(20)
    for i in range(60):
        latent = rnd.random() < 0.25
        e4 = not latent and rnd.random() < 0.4
        unit = 16 if e4 else 8
        d = 576 if latent else unit * rnd.randint(1, 256 // unit)
        hk = 1 if latent else rnd.randint(1, 4)
        group = rnd.choice((1, 2, 3, 4, 7, 8, 9, 16, 17, 33))
        P = rnd.choice((1, 2, 3, 16, 37, 64, 128))
        lens = [int(2 ** rnd.uniform(0, 11)) - 1 for _ in range(rnd.randint(1, 12))]
        run_decode(lens, hk * group, hk, d, P, rnd.choice(("bf16", "fp16")), e4, latent,
                   window=rnd.choice((0, 0, rnd.randint(1, 2000))), weights=rnd.random() < 0.5,
                   holes=rnd.random() < 0.3, seed=i, scale=192 ** -0.5 if latent else None)


# ---- eviction -------------------------------------------------------------------

def run_evict(table, w, lens, keep, P, sink, recent, cap, in_place, pad=0):
    t = torch.tensor(table, dtype=torch.int32, device="cuda")
    wt = torch.tensor(w, dtype=torch.float32, device="cuda")
    b, width = t.shape
    if pad:
        t = torch.cat([t, torch.full((b, pad), 77, dtype=torch.int32, device="cuda")], 1)[:, :width]
        wt = torch.cat([wt, torch.full((b, pad), 77.0, device="cuda")], 1)[:, :width]
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    kp = torch.tensor(keep, dtype=torch.int32, device="cuda")
    vic = torch.full((b, max(1, cap)), -7, dtype=torch.int32, device="cuda")[:, :cap]
    cnt = torch.full((b,), -7, dtype=torch.int32, device="cuda")
    if in_place:
        before = t.clone(), wt.clone()
        ot, ow, ol = t, wt, ln
        hc.evict_pages(P, t, ln, wt, kp, vic, cnt, sink=sink, recent=recent)
    else:
        ot, ow, ol = torch.full_like(t, 55), torch.full_like(wt, 55.0), torch.full_like(ln, 55)
        before = ot.clone(), ow.clone()
        hc.evict_pages(P, t, ln, wt, kp, vic, cnt, sink=sink, recent=recent, out_table=ot, out_weights=ow, out_lens=ol)
    exact = [[float(np.float32(x)) for x in r] for r in w]
    for i, (v, tt, ww, n) in enumerate(ref.evict(table, exact, lens, keep, P, sink, recent, cap)):
        assert cnt[i].item() == len(v) and ol[i].item() == n
        assert vic[i, :len(v)].tolist() == v and (vic[i, len(v):] == -7).all()
        m = len(tt)
        assert ot[i, :m].tolist() == tt and torch.equal(ot[i, m:], before[0][i, m:])
        assert torch.equal(raw(ow)[i, :m], raw(torch.tensor(ww, dtype=torch.float32, device="cuda")))
        assert torch.equal(raw(ow)[i, m:], raw(before[1])[i, m:])


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_small_and_special(in_place):
    w = [[3.0, 1.0, 2.0, 1.0, 0.0, -0.0, 0.0, 5.0],
         [NAN, INF, -INF, -1.0, 1e-45, -1e-45, 0.0, NAN],
         [1.0] * 8, [0.0] * 8, [NAN] * 8, [2.0] * 8, [2.0] * 8, [1.0, 2.0] * 4]
    table = [[10 * i + j for j in range(8)] for i in range(8)]
    table[5][3] = -1
    lens = [32, 30, 29, 0, 31, -4, 1, 1 << 30]
    for keep in ([4] * 8, [0] * 8, [-3] * 8, [100] * 8, [1, 2, 3, 4, 5, 6, 7, 7]):
        for sink, recent, cap in ((0, 1, 8), (2, 1, 8), (0, 3, 8), (0, 1, 2), (0, 1, 0), (7, 1, 8), (0, 100, 8), (50, 1, 8)):
            run_evict(table, w, lens, keep, 4, sink, recent, cap, in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n,b,kinds", [(1, 3, 2), (31, 2, 3), (1023, 2, 5), (1024, 2, 0), (1025, 3, 0), (2049, 300, 4),
                                       (4096, 2, 7), (4097, 2, 7), (5000, 2, 0), (40000, 2, 9), (131072, 3, 0),
                                       (196608, 1, 50), (196609, 1, 50), (300001, 1, 3), (393216, 1, 20), (393217, 1, 20)])
def test_evict_sizes(n, b, kinds, in_place):
    """kinds > 0: that many different weights only, so that most are equal."""
    rng = np.random.default_rng(n + b)
    w = rng.integers(0, kinds, (b, n)).astype(np.float32) if kinds else rng.standard_normal((b, n)).astype(np.float32)
    lens = [int(x) for x in rng.integers(0, 3 * n + 1, b)]
    lens[0] = 3 * n - 1
    keep = [int(x) for x in rng.integers(0, n + 1, b)]
    run_evict(rng.integers(-1, 10 ** 6, (b, n)).tolist(), w.tolist(), lens, keep, 3, int(rng.integers(0, 5)),
              int(rng.integers(1, 5)), n if b < 3 else max(1, n // 3), in_place, pad=5)


# ---- together --------------------------------------------------------------------

@pytest.mark.parametrize("latent", [False, True])
def test_serving_step_through_both_tiers(latent):
    """Prefill and decode steps through append and attention, pages evicted by
    their weight and backed up to the host, loaded back into other pages behind
    a per-layer wait, and attended to again: each against the plain forms."""
    L, P, B, steps = 2, 8, 3, 5
    hq, hk, d = (8, 1, 576) if latent else (8, 2, 64)
    dv, row = (512, 576) if latent else (64, 128)
    nb = 1 if latent else 2
    dp, width = 80, 24
    g = gen(21)
    bf = torch.bfloat16
    bufs = [torch.full((dp * P, row), float("nan"), dtype=bf, device="cuda") for _ in range(nb * L)]
    kv = hc.DeviceKV(bufs, dp)
    free = list(range(dp))
    random.Random(3).shuffle(free)
    lens = [100, 37, 9]
    table = [[-1] * width for _ in range(B)]
    cs = torch.randn((400, 64), generator=g, device="cuda")
    kw = (1 + 0.1 * torch.randn(512 if latent else d, generator=g, device="cuda")).to(bf)
    off = 512 if latent else 0
    comp, xfer = torch.cuda.Stream(), torch.cuda.Stream()
    with hc.Pool(L, nb, P, row, 64, "page_first") as pool:
        ws = torch.zeros(hc.decode_workspace(pool, B, hq, d, dv, width, True), dtype=torch.uint8, device="cuda")

        def slot(i, t):
            if table[i][t // P] < 0:
                table[i][t // P] = free.pop()
            return table[i][t // P] * P + t % P

        def append(layer, slots, positions):
            n = len(slots)
            k = torch.randn((n, hk, d), generator=g, device="cuda").to(bf)
            v = None if latent else torch.randn((n, hk, d), generator=g, device="cuda").to(bf)
            q = torch.randn((n, hq, d), generator=g, device="cuda").to(bf)
            raw_q = q.clone()
            sl, po = (torch.tensor(x, device="cuda") for x in (slots, positions))
            hc.append_kv(kv, pool, layer, q, k, v, sl, positions=po, cos_sin=cs, rot_offset=off, k_weight=kw,
                         stream=torch.cuda.current_stream())
            y, err = ref.norm_rotate(k.double(), kw, cs[po], off, False, 1e-6)
            got = bufs[layer][sl].double().view(n, hk, d)
            assert ((got - y).abs() <= err + (y.abs() + err) * 2.0 ** -8).all()
            y, err = ref.norm_rotate(raw_q.double(), None, cs[po], off, False, 1e-6)
            assert ((q.double() - y).abs() <= err + (y.abs() + err) * 2.0 ** -8).all()
            return q

        def attend(layer, q, weights):
            t = torch.tensor(table, dtype=torch.int32, device="cuda")
            n = torch.tensor(lens, dtype=torch.int32, device="cuda")
            out = torch.empty((B, hq, dv), dtype=bf, device="cuda")
            before = weights.clone()
            hc.decode_attention(kv, pool, layer, q, t, n, out, ws, weights=weights, decay=0.75,
                                stream=torch.cuda.current_stream())
            k = bufs[layer].view(dp * P, hk, d)
            v = k[..., :512] if latent else bufs[L + layer].view(dp * P, hk, d)
            want = ref.decode(q, k, v, table, lens, P, d ** -0.5)
            ref.check_decode(out, want, bf, bf, None, weights, before, 0.75)
            return out

        with torch.cuda.stream(comp):
            weights = torch.zeros((B, width), device="cuda")
            for layer in range(L):
                append(layer, [slot(i, t) for i in range(B) for t in range(lens[i])],
                       [t for i in range(B) for t in range(lens[i])])
            for _ in range(steps):
                at = [slot(i, lens[i]) for i in range(B)]
                pos = list(lens)
                lens = [n + 1 for n in lens]
                for layer in range(L):
                    attend(layer, append(layer, at, pos), weights)
            # the least attended pages of each sequence leave for the host
            t = torch.tensor(table, dtype=torch.int32, device="cuda")
            n = torch.tensor(lens, dtype=torch.int32, device="cuda")
            keep = torch.tensor([5, 3, 10], dtype=torch.int32, device="cuda")
            vic = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
            cnt = torch.empty(B, dtype=torch.int32, device="cuda")
            exp = ref.evict(table, weights.tolist(), lens, [5, 3, 10], P, 1, 1, width)
            hc.evict_pages(P, t, n, weights, keep, vic, cnt, sink=1, recent=1, stream=comp)
            comp.synchronize()
            victims = [vic[i, :c].tolist() for i, c in enumerate(cnt.tolist())]
            assert victims == [e[0] for e in exp] and cnt.tolist()[0] > 0 and cnt.tolist()[2] == 0
            old_table, old_lens = [list(r) for r in table], list(lens)
            gone = [p for r in victims for p in r]
            pool.backup(kv, gone, list(range(len(gone))), stream=comp)
            q = torch.randn((B, hq, d), generator=g, device="cuda").to(bf)
            whole = attend(1, q, torch.zeros((B, width), device="cuda"))
            table = [r[1] + [-1] * (width - len(r[1])) for r in exp]
            assert t.tolist() == table and n.tolist() == [e[3] for e in exp]
            lens = [e[3] for e in exp]
            attend(0, q, weights)                       # what stays
        comp.synchronize()
        # back into other pages, attention behind the layer's wait
        new = [free.pop() for _ in gone]
        for b in bufs:
            b.view(dp, P, row)[gone] = float("nan")
        torch.cuda.synchronize()
        pool.load_pipelined(kv, new, list(range(len(gone))), stream=xfer)
        pool.wait_layer(1, comp)
        moved = dict(zip(gone, new))
        table = [[moved.get(p, p) for p in r] for r in old_table]
        lens = old_lens
        with torch.cuda.stream(comp):
            again = attend(1, q, torch.zeros((B, width), device="cuda"))
        torch.cuda.synchronize()
        assert torch.equal(whole, again)


# ---- one side of an append -------------------------------------------------------

@pytest.mark.parametrize("d", [96, 128, 576])
def test_append_one_side_with_both_weights(d):
    """Queries alone, or keys and values alone, with the other kind's weight given
    all the same: what a call with both writes."""
    c = (37, 5, 1, d, 16, "bf16", False, d, d, 64, 0, False, d == 576)
    q, k, v, slots, pos, cs, qw, kw, bufs, pages = append_inputs(c, 17)
    q_out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
    kv, dd = hc.DeviceKV(bufs, pages), desc(16, d, 2, len(bufs))
    args = dict(positions=pos, cos_sin=cs, q_weight=qw, k_weight=kw)
    hc.append_kv(kv, dd, 0, q, k, v, slots, q_out=q_out, **args)
    want, stored = q_out.clone(), [raw(b).clone() for b in bufs]
    q_out.zero_()
    hc.append_kv(kv, dd, 0, q, None, None, None, q_out=q_out, **args)
    assert torch.equal(q_out, want) and all(torch.equal(raw(b), s) for b, s in zip(bufs, stored))
    for b in bufs:
        b.view(torch.uint8)[:] = 0x5A
    hc.append_kv(kv, dd, 0, None, k, v, slots, **args)
    assert all(torch.equal(raw(b), s) for b, s in zip(bufs, stored))


# ---- the largest batches ---------------------------------------------------------

@pytest.mark.parametrize("latent", [False, True])
@pytest.mark.parametrize("batch", [32767, 32768, 40000, 65535])
def test_decode_mostly_empty_large_batches(latent, batch):
    """Tens of thousands of sequences, all but a few empty, on a workspace that a
    call of another shape has filled."""
    d, dv = (576, 512) if latent else (64, 64)
    full = {0: 5, batch // 2: 130, batch - 1: 40}
    lens = [full.get(i, 0) for i in (0, batch // 2, batch - 1)]
    s = decode_inputs(lens, 2, 2, d, 16, latent=latent, seed=batch)
    small = torch.empty((3, 2, dv), dtype=s["dt"], device="cuda")
    plain_call(s, small, workspace(s, 2, d, dv, False))
    q = torch.zeros((batch, 2, d), dtype=s["dt"], device="cuda")
    table = torch.full((batch, s["width"]), -1, dtype=torch.int32, device="cuda")
    n = torch.zeros(batch, dtype=torch.int32, device="cuda")
    at = list(full)
    q[at], table[at], n[at] = s["q"], s["table"], s["lens"]
    other = decode_inputs([3000, 900], 64, 2 if not latent else 1, d, 16, latent=latent, seed=1, width=400)
    size = max(hc.decode_workspace(s["desc"], batch, 2, d, dv, s["width"], True),
               hc.decode_workspace(other["desc"], 2, 64, d, dv, other["width"], True))
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    plain_call(other, torch.empty((2, 64, dv), dtype=s["dt"], device="cuda"), ws,
               weights=torch.zeros((2, other["width"]), device="cuda"))
    out = torch.full((batch, 2, dv), 3.0, dtype=s["dt"], device="cuda")
    lse = torch.full((batch, 2), 3.0, device="cuda")
    s["q"], s["table"], s["lens"] = q, table, n
    plain_call(s, out, ws, lse=lse)
    empty = n == 0
    assert (out[empty] == 0).all() and (lse[empty] == -torch.inf).all()
    assert (lse[at] > -torch.inf).all()
    # the few others as in a batch of their own, up to how they are cut: the
    # exponentials' rounding, the sums' and the final one
    bound = 2.0 ** -6 * max(b[b == b].abs().max().item() for b in s["bufs"])
    assert ((out[at].float() - small.float()).abs() <= bound).all()


# ---- the workspace's error word --------------------------------------------------

def test_decode_status_and_clear():
    """The error word (behind one counter per CTA), set by hand: reported until it
    is cleared, left alone by calls in between, which are right all the same."""
    s = decode_inputs([700, 90], 16, 1, 576, 16, latent=True)
    ws = workspace(s, 16, 576, 512, False)
    a, b, c = (torch.zeros((2, 16, 512), dtype=s["dt"], device="cuda") for _ in range(3))
    plain_call(s, a, ws)
    assert not hc.decode_gave_up(ws)
    ws.view(torch.int32)[152] = 1
    assert hc.decode_gave_up(ws)
    plain_call(s, b, ws)
    assert hc.decode_gave_up(ws) and hc.decode_gave_up(ws, clear=True) and not hc.decode_gave_up(ws)
    plain_call(s, c, ws)
    assert not hc.decode_gave_up(ws) and torch.equal(a, b) and torch.equal(a, c) and a.any()


def test_decode_status_waits_for_every_stream():
    """Work still to run on a stream that does not block the default one."""
    ws = torch.zeros(1024, dtype=torch.uint8, device="cuda")
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(200_000_000)            # about a tenth of a second
        ws.view(torch.int32)[152] = 1
    assert hc.decode_gave_up(ws, clear=True)
    with torch.cuda.stream(st):
        assert ws.view(torch.int32)[152].item() == 0


# ---- eviction: the ends of the ranges --------------------------------------------

@pytest.mark.parametrize("in_place", [False, True])
def test_evict_protects_everything(in_place):
    """sink and recent at and near the largest 32-bit number."""
    big = 2 ** 31 - 1
    w = [[float((5 * i + j) % 7) for j in range(12)] for i in range(4)]
    table = [[20 * i + j for j in range(12)] for i in range(4)]
    for sink, recent in ((0, big), (4, big), (big, 1), (big, big), (5, big - 3), (big - 1, 2), (1 << 30, 1 << 30)):
        run_evict(table, w, [48, 4, 8, 0], [0, 0, -1, 2], 4, sink, recent, 12, in_place)
    rows = [[float((3 * j) % 11) for j in range(5000)]] * 2
    run_evict([list(range(5000))] * 2, rows, [5000, 2], [1, 0], 1, 4, big, 5000, in_place)


def evict_present(table, weights, lens, keep, page, sink, recent, cap):
    """serving_reference.evict where absent pages (negative entries) stay."""
    res = []
    for t, w, n_t, k in zip(table, weights, lens, keep):
        n = min(len(t), -(-n_t // page)) if n_t > 0 else 0
        may = [p for p in range(sink, max(sink, n - recent)) if t[p] >= 0]
        count = min(max(0, n - max(0, k)), len(may), cap)
        gone = set(sorted(may, key=lambda p: (w[p] != w[p], w[p] if w[p] == w[p] else 0.0, p))[:count])
        stay = [p for p in range(n) if p not in gone]
        res.append(([t[p] for p in sorted(gone)], [t[p] for p in stay] + [-1] * count,
                    [w[p] for p in stay] + [0.0] * count, n_t - count * page))
    return res


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n,b,share", [(1, 2, 0.5), (9, 6, 0.5), (40, 5, 0.9), (1025, 3, 0.3), (4096, 2, 1.0),
                                       (5000, 3, 0.5), (40000, 2, 0.99), (196609, 1, 0.2), (393217, 1, 0.5)])
def test_evict_absent_pages(monkeypatch, n, b, share, in_place):
    """Pages that are not on the device never leave, whatever their weight: not
    where fewer are present than asked for, nor where none is."""
    monkeypatch.setattr(ref, "evict", evict_present)
    rng = np.random.default_rng(n)
    table = rng.integers(0, 10 ** 6, (b, n))
    table[rng.random((b, n)) < share] = -1
    table[0, 0] = -2 ** 31
    w = rng.integers(0, 6, (b, n)).astype(np.float32)
    w[table < 0] *= rng.integers(0, 2)            # an absent page receives no attention, as a rule
    lens = [3 * n - 1] + [int(x) for x in rng.integers(0, 3 * n + 1, b - 1)]
    for keep in (0, n // 3, n - 1):
        run_evict(table.tolist(), w.tolist(), lens, [keep] * b, 3, 2, 1, n, in_place, pad=3)
        run_evict(table.tolist(), w.tolist(), lens, [keep] * b, 3, 0, 1, max(1, n // 5), in_place)


# ---- exponentials at the ends of the products' types ------------------------------

def level_caches(lens, level, value, d, hk, dtype, e4, latent, ks=1.0, vs=1.0):
    """Caches whose token t of sequence i has the score level(i, t) (log2, with a
    query of ones at one element) and value(i, t) in every element of V, pages
    of 16 in order; and the arguments of a call over them."""
    P, at = 16, 570 if latent else 0
    counts = [-(-n // P) for n in lens]
    dp, width = sum(counts), max(counts)
    row = d if latent else hk * d
    cache = E4 if e4 else dtype
    k, v = (torch.zeros((dp * P, hk, d), dtype=torch.float64, device="cuda") for _ in range(2))
    table, first = [], 0
    for i, n in enumerate(lens):
        t = torch.arange(n)
        lv, val = ([float(f(i, int(x))) for x in t] for f in (level, value))
        rows = slice(first * P, first * P + n)
        k[rows, :, at] = torch.tensor(lv, dtype=torch.float64, device="cuda")[:, None]
        (k[..., :512] if latent else v)[rows] = torch.tensor(val, dtype=torch.float64, device="cuda")[:, None, None]
        table.append(list(range(first, first + counts[i])) + [-1] * (width - counts[i]))
        first += counts[i]
    bufs = [x.reshape(-1, row).float().to(cache) for x in ((k,) if latent else (k, v))]
    for b, x in zip(bufs, (k, v)):
        assert torch.equal(b.double(), x.reshape(-1, row)), "not representable"
    q = torch.zeros((len(lens), 2 * hk, d), dtype=dtype, device="cuda")
    q[..., at] = 1
    dd = desc(P, row, 1 if e4 else 2, len(bufs))
    s = {"q": q, "desc": dd, "kv": hc.DeviceKV(bufs, dp), "width": width, "ks": ks, "vs": vs, "dt": dtype,
         "table": torch.tensor(table, dtype=torch.int32, device="cuda"),
         "lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    dv = 512 if latent else d
    out = torch.empty((len(lens), 2 * hk, dv), dtype=dtype, device="cuda")
    lse = torch.empty((len(lens), 2 * hk), device="cuda")
    plain_call(s, out, workspace(s, 2 * hk, d, dv, False), scale=float(np.log(2.0)) / ks, lse=lse)
    want, z = [], []
    for i, n in enumerate(lens):
        p = np.exp2(np.array([level(i, t) for t in range(n)], dtype=np.float64))
        want.append(float((p * [value(i, t) for t in range(n)]).sum() / p.sum()) * vs)
        z.append(float(np.log(p.sum())))
    return out.double(), lse.double(), want, z


@pytest.mark.parametrize("kind", ["fp16", "e4m3 fp16", "e4m3 bf16", "latent fp16"])
@pytest.mark.parametrize("low", [-18, -22, -24, -26, -28, -30])
def test_decode_small_weights_beside_a_large_one(kind, low):
    """The first token takes nearly all the weight and has no value; the others,
    2^low of it each, have a large one and decide the result."""
    dt = torch.bfloat16 if "bf16" in kind else torch.float16
    e4, latent = "e4m3" in kind, "latent" in kind
    big = 448.0 if e4 else 57344.0
    lens = [16, 17, 64, 200, 1000]
    out, lse, want, z = level_caches(lens, lambda i, t: low if t else 0, lambda i, t: big if t else 0.0,
                                     576 if latent else 64, 1 if latent else 2, dt, e4, latent, vs=128.0 if e4 else 1.0)
    for i, n in enumerate(lens):
        # exponentials: argument and function 2^-18 (powers of two, so that fp16's places
        # take nothing more from 2^-30 of the largest on; 2^-33 for each is left); sums of
        # n; the last rounding
        tol = abs(want[i]) * (2.0 ** -17 + 2 * n * 2.0 ** -24 + ref.UNIT[dt] + 2.0 ** -11) + \
            n * 2.0 ** -33 * 57344.0 + ref.TINY[dt]
        assert (out[i] - want[i]).abs().max().item() <= tol, (n, out[i].flatten()[0].item(), want[i])
        assert (lse[i] - z[i]).abs().max().item() <= 2.0 ** -17 + n * 2.0 ** -24


@pytest.mark.parametrize("latent", [False, True])
@pytest.mark.parametrize("power", [-100, 0, 85, 100, 115])
def test_decode_rising_scores_with_large_values(latent, power):
    """bf16 values near both ends of their range, under scores that rise by 39 (log2)
    between tiles of the same piece: exponentials that used the type's whole range
    would overflow their sums."""
    tile, n, b = (64, 1024, 60) if latent else (16, 256, 300)
    value = 2.0 ** power
    out, lse, want, z = level_caches([n] * b, lambda i, t: 39 * (t // tile % 2), lambda i, t: value,
                                     576 if latent else 64, 1 if latent else 2, torch.bfloat16, False, latent)
    # 2^-8 of each exponential, sums of n, the last rounding
    assert ((out / value - 1).abs() <= 2.0 ** -8 + 2 * n * 2.0 ** -24 + 2.0 ** -17 + 2.0 ** -8).all()
    assert ((lse - z[0]).abs() <= 2.0 ** -17 + n * 2.0 ** -24 + 4 * z[0] * 2.0 ** -24).all()


# ---- the binding's checks on the device --------------------------------------------

def test_caches_of_another_type_are_refused():
    s = decode_inputs([40], 4, 2, 64, 16, "bf16")
    ws = workspace(s, 4, 64, 64, False)
    out, before = torch.zeros((1, 4, 64), dtype=torch.float16, device="cuda"), hc.launch_count()
    slots = torch.zeros(1, dtype=torch.int64, device="cuda")
    s["q"] = s["q"].to(torch.float16)
    with pytest.raises(ValueError, match="expected torch.float16"):
        plain_call(s, out, ws)
    with pytest.raises(ValueError, match="expected torch.float16"):
        hc.append_kv(s["kv"], s["desc"], 0, None, s["q"][:, :2], s["q"][:, :2], slots)
    assert hc.launch_count() == before


def test_tensors_that_autograd_records_are_not_written():
    s = decode_inputs([40], 4, 2, 64, 16, "bf16")
    ws = workspace(s, 4, 64, 64, True)
    out = torch.zeros((1, 4, 64), dtype=s["dt"], device="cuda")
    w, lse = torch.zeros((1, s["width"]), device="cuda"), torch.zeros((1, 4), device="cuda")
    k = torch.ones((1, 2, 64), dtype=s["dt"], device="cuda")
    slots = torch.full((1,), -1, dtype=torch.int64, device="cuda")
    i32 = lambda *x: torch.zeros(x, dtype=torch.int32, device="cuda")  # noqa: E731
    calls = {
        "q": lambda x: hc.append_kv(s["kv"], s["desc"], 0, x, k, k, slots),
        "q_out": lambda x: hc.append_kv(s["kv"], s["desc"], 0, s["q"], k, k, slots, q_out=x),
        "out": lambda x: plain_call(s, x, ws),
        "lse": lambda x: plain_call(s, out, ws, lse=x),
        "weights": lambda x: plain_call(s, out, ws, weights=x),
        "weights ": lambda x: hc.evict_pages(16, s["table"], s["lens"], x, i32(1), i32(1, 2), i32(1)),
        "out_weights": lambda x: hc.evict_pages(16, s["table"], s["lens"], w, i32(1), i32(1, 2), i32(1), out_weights=x),
    }
    like = {"q": s["q"], "q_out": out, "out": out, "lse": lse, "weights": w, "weights ": w, "out_weights": w}
    for name, call in calls.items():
        t = torch.zeros_like(like[name]).requires_grad_()
        before = hc.launch_count()
        for x in (t, t * 1):                      # a leaf, and a tensor that was computed
            with pytest.raises(ValueError, match=f"{name.strip()}: written"):
                call(x)
        assert hc.launch_count() == before
        with torch.no_grad():
            call(t)
        assert hc.launch_count() > before
    # inputs that are only read may
    plain_call({**s, "q": s["q"].clone().requires_grad_()}, out, ws)
    torch.cuda.synchronize()


def test_calls_follow_the_current_stream():
    """Without a stream each operator runs on torch's current one, behind inputs that
    are still being made there, and is captured with it; with 0 on the default one."""
    s = decode_inputs([300, 40], 4, 2, 64, 16)
    ws = workspace(s, 4, 64, 64, True)
    q, lens, weight = s["q"].clone(), s["lens"].clone(), torch.rand((2, s["width"]), device="cuda")
    k = torch.randn((2, 2, 64), generator=gen(3), device="cuda").to(s["dt"])
    slots = torch.tensor([3, 700], device="cuda")
    kw = torch.ones(64, dtype=s["dt"], device="cuda")
    keep = torch.full((2,), 2, dtype=torch.int32, device="cuda")
    kv = hc.DeviceKV([torch.zeros_like(b) for b in s["bufs"]], s["Dp"])

    def step(late, stream=None):
        bufs = kv._tensors
        new = {"q": torch.zeros_like(q), "k": torch.zeros_like(k), "lens": torch.zeros_like(lens)}
        out = torch.zeros((2, 4, 64), dtype=s["dt"], device="cuda")
        w, t, n = torch.zeros_like(weight), s["table"].clone(), torch.zeros_like(lens)
        vic, cnt = torch.full_like(t, -1), torch.zeros_like(lens)
        for b, x in zip(bufs, s["bufs"]):
            b.copy_(x)
        torch.cuda.synchronize()
        if late:
            torch.cuda._sleep(50_000_000)
        new["q"].copy_(q), new["k"].copy_(k), new["lens"].copy_(lens), n.copy_(lens)
        hc.append_kv(kv, s["desc"], 0, new["q"], new["k"], new["k"], slots, q_weight=kw, stream=stream)
        hc.decode_attention(kv, s["desc"], 0, new["q"], s["table"], new["lens"], out, ws, weights=w, stream=stream)
        w.add_(weight)
        hc.evict_pages(16, t, n, w, keep, vic, cnt, stream=stream)
        return [new["q"], out, w, t, n, vic, cnt]
    want = step(False)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = step(True)
        torch.cuda.current_stream().synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and want[-1].tolist() == [17, 1]
    got = step(False, stream=0)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out = torch.zeros_like(want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        hc.decode_attention(kv, s["desc"], 0, want[0], s["table"], lens, out, ws)
    assert not out.any()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[1])


@pytest.mark.parametrize("latent", [False, True])
def test_single_rows_with_odd_strides(latent):
    """One sequence, one head, one token, as views whose unused strides are odd."""
    d, dv = (576, 512) if latent else (64, 64)
    s = decode_inputs([90], 1, 1, d, 16, latent=latent)
    ws = workspace(s, 1, d, dv, True)
    odd = lambda t, *st: torch.as_strided(t, t.shape, (*st, 1))  # noqa: E731
    a, b = (torch.zeros((1, 1, dv), dtype=s["dt"], device="cuda") for _ in range(2))
    w, lse = [torch.zeros((1, s["width"]), device="cuda") for _ in range(2)], torch.zeros((1, 1), device="cuda")
    q, table = s["q"], s["table"]
    plain_call(s, a, ws, weights=w[0])
    s["q"], s["table"] = odd(q, 13, 7), odd(table, 1)
    plain_call(s, odd(b, 3, 5), ws, weights=odd(w[1], 3), lse=odd(lse, 9))
    assert torch.equal(a, b) and torch.equal(*w) and a.any()
    k = torch.randn((1, 1, d), generator=gen(2), device="cuda").to(s["dt"])
    for x in (k, odd(k, 11, 3)):
        for buf in s["bufs"]:
            buf[5] = 0
        got = torch.zeros((1, 1, d), dtype=s["dt"], device="cuda")
        hc.append_kv(s["kv"], s["desc"], 0, odd(q, 9, 1), x, None if latent else x,
                     torch.tensor([5], device="cuda"), q_out=odd(got, 1, 1))
        assert torch.equal(got, q) and all(torch.equal(buf[5], k.view(-1)) for buf in s["bufs"])
    n = [torch.tensor([90], dtype=torch.int32, device="cuda") for _ in range(4)]
    vic = [torch.full((1, 4), -1, dtype=torch.int32, device="cuda") for _ in range(2)]
    keep, cnt = torch.full((1,), 3, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    t = [table.clone(), table.clone()]
    hc.evict_pages(16, t[0], n[0], w[0], keep, vic[0], cnt)
    hc.evict_pages(16, odd(t[1], 2), n[1], odd(w[1], 1), keep, odd(vic[1], 1), cnt)
    assert torch.equal(*t) and torch.equal(*w) and torch.equal(*vic) and cnt.item() == 3


@pytest.mark.parametrize("c", [(40, 16, 1, 576, 64, "bf16", True, 0, 512, 64, 512, False, True),
                               (700, 3, 1, 576, 16, "fp16", True, 576, 512, 64, 512, True, True),
                               (9, 2, 1, 384, 4, "bf16", True, 384, 384, 96, 10, False, True)], ids=["0", "1", "2"])
def test_append_latent_e4m3(c):
    """Latent rows in e4m3: stored like those of K."""
    test_append(c)


# ---- how far off on the whole ------------------------------------------------------

@pytest.mark.parametrize("kind", ["bf16", "fp16", "e4m3 fp16", "latent bf16", "latent fp16"])
def test_decode_error_as_a_root_mean_square(kind):
    """Thousands of tokens of about the same weight, where a bound on each element's worst
    case is as large as the element: a tile of V left out, or counted twice, would
    pass it.  Rounding the exponentials p shifts an output, sum p v, by errors that are
    independent and uniform over half a step either way, u p / sqrt 3 at most as a root
    mean square: u / sqrt 3 sqrt(sum p^2 v^2) together, where sqrt(sum p^2 v^2) is the
    outputs' own root mean square (v of mean zero).  The last rounding adds as much of
    the output's type.  A token left out of 4,096 alone would be 2^-6."""
    dt = torch.bfloat16 if "bf16" in kind else torch.float16
    e4, latent = "e4m3" in kind, "latent" in kind
    lens, P = [4096, 1000, 2777], 16
    hq, hk, d = (16, 1, 576) if latent else (8, 2, 128)
    s = decode_inputs(lens, hq, hk, d, P, "bf16" if "bf16" in kind else "fp16", e4, latent, seed=31, sharp=0.5)
    dv = 512 if latent else d
    out = torch.empty((3, hq, dv), dtype=dt, device="cuda")
    w = torch.zeros((3, s["width"]), device="cuda")
    plain_call(s, out, workspace(s, hq, d, dv, True), weights=w, scale=d ** -0.5)
    k = s["bufs"][0].view(s["Dp"] * P, -1, d)
    v = k[..., :512] if latent else s["bufs"][1].view(s["Dp"] * P, -1, d)
    want = ref.decode(s["q"], k, v, s["clean"], lens, P, d ** -0.5, 0, s["ks"], s["vs"])
    p_unit = ref.UNIT[torch.float16 if e4 else dt]
    for i, (o, z, share, _) in enumerate(want):
        rms = lambda x: x.double().pow(2).mean().sqrt().item()  # noqa: E731
        # sqrt 3 above that, for chance
        off = rms(out[i].double() - o) / rms(o)
        assert off <= (p_unit ** 2 + ref.UNIT[dt] ** 2) ** 0.5, (i, off)
        # scores: d / 16 <= 36 sums in 32 bits, each off by at most a step (2^-23) of less
        # than 4; arguments under 16 by 2^-21, the function by 2^-22
        pages = share.numel()
        assert rms(w[i, :pages].double() - share) / rms(share) <= 2.0 ** -15


# ---- random shapes -----------------------------------------------------------------

def test_append_random_corpus():
    """Random shapes over the documented ranges, some slots and positions outside."""
    rnd = random.Random(41)
    for i in range(120):
        e4, latent, il = rnd.random() < 0.4, rnd.random() < 0.25, rnd.random() < 0.5
        unit = 16 if e4 else 8
        d = rnd.choice((64, 128, 256, 576, unit * rnd.randint(1, 768 // unit), unit * rnd.randint(1, 256 // unit)))
        hk = 1 if latent else rnd.randint(1, 5)
        norms = [rnd.choice((0, d, 8 * rnd.randint(0, d // 8), d // 128 * 64)) for _ in range(2)]
        rot = rnd.choice((0, d, 64 if d >= 64 else 2, 2 * rnd.randint(0, d // 2), d // 4 // 2 * 2))
        off = rnd.choice((0, d - rot, 2 * rnd.randint(0, (d - rot) // 2), (d - rot) // 64 * 64))
        n = int(2 ** rnd.uniform(0, 11))
        c = (n, rnd.randint(1, 17), hk, d, rnd.choice((1, 5, 16, 64)), rnd.choice(("bf16", "fp16")), e4, *norms, rot,
             off, il, latent)
        q, k, v, slots, pos, cs, qw, kw, bufs, pages = append_inputs(c, i)
        skip = torch.zeros(n, dtype=torch.bool, device="cuda")
        if rnd.random() < 0.5:
            slots[::3] = rnd.choice((-1, pages * c[4], 2 ** 40))
            if cs is not None:
                skip[1::4] = True
                pos[1::4] = rnd.choice((-1, 5000, -2 ** 50))
        old = [b.clone() for b in bufs]
        ks, vs = (0.03, 0.05) if e4 else (1.0, 1.0)
        q_out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
        hc.append_kv(hc.DeviceKV(bufs, pages), desc(c[4], hk * d, bufs[0].element_size(), len(bufs)), 0, q, k, v, slots,
                     q_out=q_out, positions=pos if cs is not None else None, cos_sin=cs, rot_offset=off, interleaved=il,
                     q_weight=qw, k_weight=kw, k_scale=ks, v_scale=vs)
        try:
            check_append(c, q, k, v, slots, pos, cs, qw, kw, bufs, q_out, old, ks, vs, skip)
            assert (q_out[skip] == 7.0).all()
        except AssertionError as e:
            raise AssertionError(f"{i}: {c}: {e}") from None


def test_evict_random_corpus(monkeypatch):
    """Random tables, weights, budgets and protected pages, absent pages among them."""
    monkeypatch.setattr(ref, "evict", evict_present)
    rng = np.random.default_rng(7)
    for i in range(80):
        n, b, P = int(2 ** rng.uniform(0, 13.5)), int(rng.integers(1, 7)), int(rng.choice((1, 4, 16, 100)))
        w = rng.standard_normal((b, n)).astype(np.float32) if i % 2 else rng.integers(0, 4, (b, n)).astype(np.float32)
        table = rng.integers(0, 10 ** 6, (b, n))
        table[rng.random((b, n)) < rng.choice((0.0, 0.0, 0.3, 1.0))] = -1
        lens = [int(x) for x in rng.integers(-1, n * P + 2 * P, b)]
        keep = [int(x) for x in rng.integers(-1, n + 2, b)]
        run_evict(table.tolist(), w.tolist(), lens, keep, P, int(rng.choice((0, 1, 4, n, 2 ** 31 - 1))),
                  int(rng.choice((1, 2, 8, n + 1, 2 ** 31 - 1), p=(0.4, 0.2, 0.2, 0.1, 0.1))),
                  int(rng.choice((0, 1, n, 2 * n))), bool(rng.integers(0, 2)), pad=int(rng.integers(0, 3)))


# ---- at once, and shared pages -----------------------------------------------------

@pytest.mark.parametrize("latent", [False, True])
def test_decode_from_threads_at_once(latent):
    """Calls from several host threads on a stream and a workspace each, over one
    cache: the bits of a call alone."""
    import threading
    d, dv = (576, 512) if latent else (128, 128)
    s = decode_inputs([3000, 40, 700, 0, 1111], 16, 4, d, 16, latent=latent, seed=9)
    want, w0 = torch.empty((5, 16, dv), dtype=s["dt"], device="cuda"), torch.zeros((5, s["width"]), device="cuda")
    plain_call(s, want, workspace(s, 16, d, dv, True), weights=w0)
    torch.cuda.synchronize()
    bad = []

    def work():
        st, ws = torch.cuda.Stream(), workspace(s, 16, d, dv, True)
        with torch.cuda.stream(st):
            for _ in range(30):
                out, w = torch.zeros_like(want), torch.zeros_like(w0)
                st.synchronize()
                plain_call(s, out, ws, weights=w)
                st.synchronize()
                if not (torch.equal(out, want) and torch.equal(w, w0)):
                    bad.append(1)
    threads = [threading.Thread(target=work) for _ in range(4)]
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


@pytest.mark.parametrize("latent", [False, True])
def test_decode_pages_of_several_sequences(latent):
    """Sequences that share a prefix's pages, one page twice in a sequence, a table that
    all sequences share (stride 0): as over copies of the pages."""
    d, dv, P = (576, 512, 16) if latent else (64, 64, 16)
    s = decode_inputs([160], 4, 2, d, P, latent=latent, spare=0)
    base = s["table"][0].clone()
    tables = [base.tolist(), base.tolist()[:4] + base.tolist()[7:] + [-1] * 3, [int(base[2])] * 10]
    lens = [160, 100, 150]
    q = torch.randn((3, 4, d), generator=gen(3), device="cuda").to(s["dt"])
    total = sum(-(-n // P) for n in lens)
    copies, at, apart = [torch.zeros((total * P, b.shape[1]), dtype=b.dtype, device="cuda") for b in s["bufs"]], 0, []
    for t, n in zip(tables, lens):
        row = []
        for p in t[:-(-n // P)]:
            for c, b in zip(copies, s["bufs"]):
                c[at * P:at * P + P] = b[p * P:p * P + P]
            row.append(at)
            at += 1
        apart.append(row + [-1] * (10 - len(row)))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = torch.zeros(hc.decode_workspace(s["desc"], 3, 4, d, dv, 10, True), dtype=torch.uint8, device="cuda")

    def call(kv, table):
        out, w = torch.zeros((3, 4, dv), dtype=s["dt"], device="cuda"), torch.zeros((3, 10), device="cuda")
        hc.decode_attention(kv, s["desc"], 0, q, table, i32(lens), out, ws, weights=w)
        return out, w
    for a, b in zip(call(s["kv"], i32(tables)), call(hc.DeviceKV(copies, total), i32(apart))):
        assert torch.equal(a, b) and a.any()
    one = i32([tables[0]])
    for a, b in zip(call(s["kv"], one.expand(3, 10)), call(s["kv"], one.repeat(3, 1))):
        assert torch.equal(a, b)
