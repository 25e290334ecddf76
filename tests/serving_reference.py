"""Plain 64-bit forms of the operators on the device pages, one sequence at a
time, and the error bounds their results are held to.

Bounds count roundings: u(t) = eps(t) / 2 relative for each rounding to type t
(2^-8 bf16, 2^-11 fp16, 2^-24 fp32, 2^-4 e4m3), half the smallest subnormal
absolute."""
from __future__ import annotations

import torch

U32 = 2.0 ** -24
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float8_e4m3fn: 2.0 ** -4}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float8_e4m3fn: 2.0 ** -10}


def norm_rotate(x, weight, cs, rot_offset, interleaved, eps):
    """x [n, h, d] float64 -> (result, bound before the final rounding)."""
    y = x.clone()
    m = 0 if weight is None else weight.numel()
    if m:
        ms = y[..., :m].pow(2).mean(-1, keepdim=True) + eps
        y[..., :m] = y[..., :m] / ms.sqrt() * weight.double()
    # the sum of m squares: m + 1 roundings of the square, half of that in the
    # root, then the root itself (2), the quotient by m, eps, and two products
    rel = (m / 2 + 8) * U32
    err = y.abs() * rel
    if cs is not None:
        rot = cs.shape[1]
        half = rot // 2
        j = torch.arange(half, device=x.device)
        a = rot_offset + (2 * j if interleaved else j)
        b = rot_offset + (2 * j + 1 if interleaved else j + half)
        co, si = cs[:, None, :half].double(), cs[:, None, half:].double()
        ya, yb = y[..., a].clone(), y[..., b].clone()
        y[..., a] = ya * co - yb * si
        y[..., b] = yb * co + ya * si
        both = ya.abs() + yb.abs()
        err[..., a] = both * (rel + 2 * U32)
        err[..., b] = both * (rel + 2 * U32)
    return y, err


def decode(q, k, v, table, lens, page, scale, window=0, k_scale=1.0, v_scale=1.0):
    """q [b, hq, d], k and v [slots, hk, d(v)] (values without their scales),
    table (a list of lists, None or out of range = absent is given as -1).
    Returns per sequence (out, lse, share per page, bounds) in float64."""
    res = []
    hk = k.shape[1]
    for i, n in enumerate(lens):
        pages = -(-n // page)
        t = torch.arange(max(0, n - window) if window else 0, n, device=q.device)
        pg = torch.tensor(table[i][:pages] or [-1], device=q.device)[t // page] if n else t
        t, pg = t[pg >= 0], pg[pg >= 0]
        hq, d = q.shape[1], q.shape[2]
        if t.numel() == 0:
            res.append((torch.zeros(hq, v.shape[-1], dtype=torch.float64, device=q.device),
                        torch.full((hq,), -torch.inf, dtype=torch.float64, device=q.device),
                        torch.zeros(pages, dtype=torch.float64, device=q.device), None))
            continue
        rows = pg * page + t % page
        kk, vv = k[rows].double() * k_scale, v[rows].double() * v_scale
        qq = q[i].double().view(hk, hq // hk, d)
        x = torch.einsum("kgd,tkd->kgt", qq, kk) * scale
        # |s| error: d products summed in 32 bits (a tensor core's sum may
        # truncate: a whole step, 2 U32, an addition), the scale's and the
        # product's rounding; for an e4m3 cache q goes to fp16 scaled to its
        # largest element, off by at most 2^-25 of that
        mass = torch.einsum("kgd,tkd->kgt", qq.abs(), kk.abs()) * abs(scale)
        big = qq.abs().amax(-1)[..., None] * kk.abs().sum(-1).T[:, None, :] * abs(scale)
        ds = (mass * (2 * d + 4) * U32 + big * 2.0 ** -25 + 2 * x.abs() * U32).amax(-1)
        z = torch.logsumexp(x, -1, keepdim=True)
        p = torch.exp(x - z)
        out = torch.einsum("kgt,tkd->kgd", p, vv)
        spread = torch.einsum("kgt,tkd->kgd", p, vv.abs())
        share = torch.zeros(pages, dtype=torch.float64, device=q.device)
        share.index_add_(0, t // page, p.sum((0, 1)))
        # an exponential: twice the error of s (its own and the maximum's), the
        # argument's rounding (|x - max| U32 <= 2^-19 at 32 apart, below which
        # the term itself is under 2^-46), 2^-21 of the exponential itself
        de = 2 * ds + 2.0 ** -19
        n_t = t.numel()
        dl = de + n_t * U32                               # the sum
        res.append((out.reshape(hq, -1), z.flatten(), share,
                    {"spread": spread.reshape(hq, -1), "de": (de + dl).flatten(), "dl": dl.flatten(),
                     "n": n_t, "vmax": vv.abs().max().item()}))
    return res


def check_decode(got, want, dtype, p_type, lse=None, weights=None, before=None, decay=1.0):
    """got [b, hq, dv]; p_type: the type the exponentials are rounded to."""
    worst = 0.0
    for i, (out, z, share, bd) in enumerate(want):
        g = got[i].double()
        if bd is None:
            assert torch.equal(g, torch.zeros_like(g)), f"sequence {i}: no tokens, but out is not zero"
            if lse is not None:
                assert (lse[i] == -torch.inf).all(), f"sequence {i}: lse of no tokens"
        else:
            # the exponentials' rounding, the sum over tokens in 32 bits, the
            # final rounding; fp16 exponentials under 2^-14 lose 2^-25 each,
            # against a sum of at least 1
            rel = UNIT[p_type] + (bd["de"][:, None] + 2 * bd["n"] * U32)
            tol = bd["spread"] * rel + out.abs() * UNIT[dtype] * (1 + rel) + TINY[dtype]
            tol = tol + (bd["n"] * 2.0 ** -25 * bd["vmax"] if p_type == torch.float16 else 0.0) + 1e-30
            off = ((g - out).abs() / tol).max().item()
            assert off <= 1.0, f"sequence {i}: out is {off:.3g} of its bound off"
            worst = max(worst, off)
            if lse is not None:
                off = ((lse[i].double() - z).abs() / (bd["dl"] + 4 * z.abs() * U32 + 2.0 ** -21)).max().item()
                assert off <= 1.0, f"sequence {i}: lse is {off:.3g} of its bound off"
        if weights is not None:
            w = weights[i].double()
            pages = share.numel()
            b0 = before[i].double()
            exp = decay * b0[:pages] + share
            rel = (bd["de"].max().item() + 2.0 ** -20) if bd is not None else 0.0
            count = 4 + got.shape[1] + 512
            tol = share * (rel + count * U32) + exp.abs() * 4 * U32 + 1e-30
            off = ((w[:pages] - exp).abs() / tol).max().item() if pages else 0.0
            assert off <= 1.0, f"sequence {i}: weights are {off:.3g} of their bound off"
            assert torch.equal(weights[i][pages:], before[i][pages:]), f"sequence {i}: weights behind its pages changed"
    return worst


def evict(table, weights, lens, keep, page, sink, recent, cap):
    """Lists in, lists out: (victims, table, weights, length) per sequence;
    the table and weights are the first n entries after the call."""
    res = []
    for t, w, n_t, k in zip(table, weights, lens, keep):
        n = min(len(t), -(-n_t // page)) if n_t > 0 else 0
        may = list(range(sink, max(sink, n - recent)))
        count = min(max(0, n - max(0, k)), len(may), cap)
        order = sorted(may, key=lambda p: (w[p] != w[p], w[p] if w[p] == w[p] else 0.0, p))
        gone = set(order[:count])
        stay = [p for p in range(n) if p not in gone]
        res.append(([t[p] for p in sorted(gone)], [t[p] for p in stay] + [-1] * count,
                    [w[p] for p in stay] + [0.0] * count, n_t - count * page))
    return res
