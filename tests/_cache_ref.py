"""The operators of a cache in 4 bits and of its pages (idx_cache_append_mxfp4, idx_window_attention_mxfp4,
idx_cache_fork, idx_cache_resize, idx_cache_compact) in 64 bits and plain loops, on the CPU, with the error
bounds their formats give."""
import math

import numpy as np
import torch

from _serve_ref import U32, unit

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


# ---------------------------------------------------------------- the format

def quantise(x):
    """(codes [..., D / 2], scales [..., D / 32]) uint8 of x [..., D], an element at a time in 64 bits."""
    x = x.double().numpy()
    flat = x.reshape(-1, 32)
    codes, scales = np.zeros(flat.shape, dtype=np.uint8), np.zeros(len(flat), dtype=np.uint8)
    for i, block in enumerate(flat):
        if not np.isfinite(block).all():
            scales[i] = 255
            continue
        top = np.abs(block).max()
        e = max(math.frexp(top)[1] - 1 - 2, -127) if top > 0 else 0
        scales[i] = e + 127
        for j, v in enumerate(block):
            a = abs(math.ldexp(v, -e))
            # the nearest value, the even code of two that are as near
            best = min(range(8), key=lambda c: (abs(GRID[c] - a), c % 2))
            codes[i, j] = best + 8 * (math.copysign(1.0, v) < 0)
    codes = codes.reshape(x.shape)
    packed = codes[..., 0::2] | codes[..., 1::2] << 4
    return torch.from_numpy(packed.copy()), torch.from_numpy(scales.reshape(*x.shape[:-1], -1).copy())


def values(codes, sf):
    """[..., D] in 64 bits; NaN under a scale of 255."""
    lut = torch.tensor(list(GRID) + [-g for g in GRID], dtype=torch.float64)
    x = torch.stack([lut[(codes & 15).long()], lut[(codes >> 4).long()]], -1).flatten(-2)
    scale = torch.where(sf == 255, math.nan, torch.pow(2.0, sf.double() - 127))
    return x * scale.repeat_interleave(32, -1)


def starts(new, T=None):
    return torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32)


def append(k, v, cache, table, lens, q_start):
    """cache: (k_codes, k_sf, v_codes, v_sf); the same after the append."""
    out = [c.clone() for c in cache]
    page = out[0].shape[2]
    rows = [quantise(k), quantise(v)]
    for b in range(len(lens)):
        first, end = int(q_start[b]), int(q_start[b + 1])
        for t in range(first, end):
            p = int(lens[b]) - end + t
            where = int(table[b, p // page])
            if where < 0:
                continue
            for i in range(2):
                out[2 * i][where, :, p % page] = rows[i][0][t]
                out[2 * i + 1][where, :, p % page] = rows[i][1][t]
    return out


# ----------------------------------------------------------------- attention

def attention(q, cache, table, lens, q_start, window=0, sink=0, scale=None):
    """Per row o, lse, the mean and the sum of |v| (for the bound), and the largest sum |q_d k_d| that a row meets;
    rows of tokens outside every request are NaN in `o`'s place of `big`."""
    T, Hq, D = q.shape
    page, Hkv = cache[0].shape[2], cache[0].shape[1]
    G = Hq // Hkv
    scale = D ** -0.5 if scale is None else scale
    q = q.double()
    o = torch.zeros(T, Hq, D, dtype=torch.float64)
    absv, sumv = torch.zeros_like(o), torch.zeros_like(o)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    big = torch.zeros(T, Hq, dtype=torch.float64)
    inside = torch.zeros(T, dtype=torch.bool)
    for b in range(len(lens)):
        n, first, end = int(lens[b]), int(q_start[b]), int(q_start[b + 1])
        for t in range(first, end):
            inside[t] = True
            p = n - end + t
            j = torch.arange(max(0, min(n, p + 1)))
            if window:
                j = j[(j < sink) | (j > p - window)]
            if len(j) == 0:
                continue
            ids = table[b].long()[j // page]
            k = values(cache[0][ids, :, j % page], cache[1][ids, :, j % page])
            v = values(cache[2][ids, :, j % page], cache[3][ids, :, j % page])
            for h in range(Hq):
                kh, vh = k[:, h // G], v[:, h // G]
                z = scale * (kh @ q[t, h])
                # a slot with a NaN scale, in K or V, is a NaN logit
                z = torch.where(torch.isnan(kh).any(1) | torch.isnan(vh).any(1), math.nan, z)
                lse[t, h] = torch.logsumexp(z, 0)
                w = torch.exp(z - lse[t, h])
                o[t, h] = w @ vh
                absv[t, h] = w @ vh.abs()
                sumv[t, h] = vh.abs().sum(0)
                big[t, h] = abs(scale) * (kh.abs() @ q[t, h].abs()).max()
    return o, lse, absv, sumv, big, inside


def check_attention(got, ref, dtype, keys, D):
    """Codes and queries are exact in the products (bf16 queries to 2^-38 of a row's largest).  A logit's D products and
    sums lose at most 2 (D + 8) units of sum |q k| scale and its scaling 8 units of itself: dz, an absolute error
    of the exponent, so a relative one of the weight, to which the exponential (2^-22) and a sum over at most
    `keys` weights (a unit each) add.  Weights enter the second product rounded by at most a half step of the
    tensors' type, and by 2^-32 of the row's largest where they are small; o is rounded to that type."""
    o, lse, absv, sumv, big, inside = ref
    u = unit(dtype)
    go, gl = got[0].double()[inside], got[1].double()[inside]
    o, lse, absv, sumv, big = (x[inside] for x in (o, lse, absv, sumv, big))
    nan = torch.isnan(lse)
    assert torch.isnan(gl[nan]).all() and torch.isnan(go[nan]).all(), "rows that see a NaN"
    empty = lse == -math.inf
    assert (gl[empty] == -math.inf).all() and (go[empty] == 0).all(), "rows that see nothing"
    full = ~nan & ~empty
    # what the type does not hold is infinite in it: from its largest number on, half a step and the error below apart
    most = torch.finfo(dtype).max
    over = full[..., None] & (o.abs() > most * (1 - 2.0 ** -6))
    assert (torch.isinf(go[over]) | (go[over].abs() >= most * (1 - 2.0 ** -5))).all(), "values past the type's range"
    assert (torch.sign(go[over]) == torch.sign(o[over])).all()
    assert torch.isfinite(gl[full]).all() and torch.isfinite(go[full[..., None] & ~over]).all(), "rows that are finite"
    dz = 2 * (D + 8) * U32 * big + 8 * U32 * big + 2.0 ** -20 + keys * U32
    tol = dz + 4 * U32 * lse.abs()
    err = (gl - lse).abs()
    assert (err <= tol)[full].all(), f"lse: {float((err / tol)[full].max())} of the bound"
    tol = (u + 2 * dz)[..., None] * absv * 1.01 + 2.0 ** -32 * sumv + u * o.abs() + 2.0 ** -24
    err = torch.where(over, 0.0, (go - o).abs())
    assert (err <= tol)[full].all(), f"out: {float((err / tol)[full].max())} of the bound"


# --------------------------------------------------------------------- pages

def pages_of(n, page):
    return -(-n // page)


def held(table, lens, page):
    return [r[:pages_of(n, page)] for r, n in zip(table.tolist(), lens.tolist())]


def counts(rows, pages):
    c = [0] * pages
    for r in rows:
        for p in r:
            c[p] += 1
    return torch.tensor(c, dtype=torch.int32)


def laid_out(rows, like, before=None):
    t = torch.full_like(like, -1) if before is None else before.clone()
    for i, r in enumerate(rows):
        t[i, :len(r)] = torch.tensor(r, dtype=torch.int32)
    return t


def fork(table, lens, parent, page):
    """(rows of pages, lengths)"""
    rows = held(table, lens, page)
    return ([list(rows[p]) if p >= 0 else [] for p in parent.tolist()],
            torch.tensor([int(lens[p]) if p >= 0 else 0 for p in parent.tolist()], dtype=torch.int32))


def resize(caches, table, lens, new_lens, page, pages):
    """(caches, rows of pages, lengths, whether the pages sufficed): row by row, as the definition says it."""
    old, new = lens.tolist(), new_lens.tolist()
    rows = [r[:pages_of(min(n, m), page)] for r, n, m in zip(held(table, lens, page), old, new)]
    count = counts(rows, pages).tolist()
    free = [p for p in range(pages) if count[p] == 0]
    out, served, enough = [c.clone() for c in caches], list(old), True
    for i, (n, m) in enumerate(zip(old, new)):
        if m <= n:
            served[i] = m
            continue
        copy = n % page != 0 and count[rows[i][-1]] > 1
        want = pages_of(m, page) - pages_of(n, page) + copy
        if want and (want > len(free) or not enough):
            enough = False
            continue
        if copy:
            to = free.pop(0)
            for c, o in zip(caches, out):
                o[to] = c[rows[i][-1]]
            rows[i][-1] = to
        while len(rows[i]) < pages_of(m, page):
            rows[i].append(free.pop(0))
        served[i] = m
    return out, rows, torch.tensor(served, dtype=torch.int32), enough


def compact(caches, refs, table, lens, page):
    """(caches, counts, rows of pages, live)"""
    c = refs.tolist()
    live = sum(n > 0 for n in c)
    holes = [p for p in range(live) if c[p] <= 0]
    to = dict(zip([p for p in range(live, len(c)) if c[p] > 0], holes))
    out, refs_out = [x.clone() for x in caches], torch.zeros_like(refs)
    for p, n in enumerate(c):
        if n > 0:
            refs_out[to.get(p, p)] = n
            for x, y in zip(caches, out):
                y[to.get(p, p)] = x[p]
    return out, refs_out, [[to.get(p, p) for p in r] for r in held(table, lens, page)], live
