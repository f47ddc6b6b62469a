"""The serving operators (idx_add_rmsnorm_quant, idx_prefix_attention, idx_cache_evict) in
64 bits and plain loops, on the CPU, with the error bounds their formats give.

Rounding to a type with unit roundoff u = eps / 2 (bf16 2^-8, fp16 2^-11, fp32 2^-24,
e4m3 2^-4) is off by at most u times the value."""
import math

import numpy as np
import torch

U32 = 2.0 ** -24


def unit(dtype):
    return torch.finfo(dtype).eps / 2


# ------------------------------------------------------------------ norm

def norm(x, weight, residual=None, eps=1e-6, group=0):
    """(y in 64 bits, scale in 64 bits, h in 64 bits)"""
    h = x.double() + (residual.double() if residual is not None else 0.0)
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + eps) * weight.double()
    parts = y.reshape(y.shape[0], -1, group or y.shape[1])
    scale = torch.clamp(parts.abs().amax(2) / 448.0, min=2.0 ** -100)
    return y, (scale if group else scale[:, 0]), h


def check_norm(out, scale, x, weight, residual=None, residual_out=None, eps=1e-6, group=0):
    """The norm's fp32 steps: a sum of N squares (at most 32 in sequence per thread, then
    a tree and 32 partial sums: under 80 roundings, halved by the square root), rsqrt
    (2 units), and a handful of products: 64 units cover them.  Codes add half an e4m3
    step: 2^-4 of the value, or 2^-10 of the scale for subnormal codes."""
    y, want, h = norm(x, weight, residual, eps, group)
    rel = 64 * U32
    got = scale.double()
    assert (got > 0).all()
    assert ((got - want).abs() <= rel * want).all(), "scale"
    N = y.shape[1]
    spread = got.reshape(y.shape[0], -1).repeat_interleave(group or N, 1)
    err = (out.float().double() * spread - y).abs()
    assert (err <= (2.0 ** -4 + 2 * rel) * y.abs() + (2.0 ** -10 + rel) * spread).all(), "codes"
    if residual_out is not None:
        u = unit(x.dtype)
        assert ((residual_out.double() - h).abs() <= (u + 2 * U32) * h.abs()).all(), "residual"


# ------------------------------------------------------------- attention

def gather(cache, table, n):
    """[n, Hkv, D] of the slots 0 .. n - 1 that a table row names."""
    page = cache.shape[2]
    s = torch.arange(n)
    return cache[table.long()[s // page], :, s % page]


def attention(q, k_cache, v_cache, table, lens, prefix_table=None, prefix_len=0, scale=None, weights=None):
    """Per row o and lse, the mean of |v| under the weights (for the bound), the largest
    sum |q_d k_d| a row meets, and the private weights with what they gathered."""
    B, Q, Hq, D = q.shape
    Hkv = k_cache.shape[1]
    G = Hq // Hkv
    scale = D ** -0.5 if scale is None else scale
    q = q.double()
    o = torch.zeros(B, Q, Hq, D, dtype=torch.float64)
    absv = torch.zeros_like(o)
    lse = torch.full((B, Q, Hq), -math.inf, dtype=torch.float64)
    big = torch.zeros(B, Q, Hq, dtype=torch.float64)
    w = None if weights is None else weights.double().clone()
    kp = gather(k_cache, prefix_table, prefix_len).double() if prefix_len else None
    vp = gather(v_cache, prefix_table, prefix_len).double() if prefix_len else None
    for b in range(B):
        n = int(lens[b])
        ks, vs = gather(k_cache, table[b], n).double(), gather(v_cache, table[b], n).double()
        if w is not None:
            w[b, :, max(0, n - Q):n] = 0.0
        for t in range(Q):
            m = max(0, n - (Q - 1 - t))
            k = torch.cat([kp, ks[:m]]) if prefix_len else ks[:m]
            v = torch.cat([vp, vs[:m]]) if prefix_len else vs[:m]
            if k.shape[0] == 0:
                continue
            for h in range(Hq):
                z = scale * (k[:, h // G] @ q[b, t, h])
                lse[b, t, h] = torch.logsumexp(z, 0)
                p = torch.exp(z - lse[b, t, h])
                o[b, t, h] = p @ v[:, h // G]
                absv[b, t, h] = p @ v[:, h // G].abs()
                big[b, t, h] = abs(scale) * (k[:, h // G].abs() @ q[b, t, h].abs()).max()
                if w is not None:
                    w[b, h // G, :m] += p[prefix_len:]
    return o, lse, absv, big, w


def check_attention(got, ref, dtype, keys, D, old=None, lens=None):
    """A logit's D products and sums lose at most (D + 4) units of sum |q k| scale: dz,
    an absolute error of the exponent, so a relative one of the weight, to which the
    exponential (2^-22) and a sum over at most `keys` weights (a unit each) add.  o also
    rounds every weight to the tensors' type (u of the mean |v|) and itself (u |o|)."""
    o, lse, absv, big, w = ref
    dz = (D + 4) * U32 * big * 2 + 2.0 ** -20 + keys * U32
    u = unit(dtype)
    go, gl = got[0].double(), got[1].double()
    empty = lse == -math.inf
    assert (gl[empty] == -math.inf).all() and (go[empty] == 0).all()
    assert torch.isfinite(gl[~empty]).all()
    tol_l = dz + 4 * U32 * lse.abs()
    assert ((gl - lse).abs()[~empty] <= tol_l[~empty]).all(), float((gl - lse).abs()[~empty].max())
    tol = (u + 2 * dz)[..., None] * absv * 1.01 + u * o.abs() + 2.0 ** -24
    err = (go - o).abs()
    assert (err <= tol).all(), f"out: {float((err / tol).max())} of the bound"
    if w is not None:
        gw = got[2].double()
        for b in range(w.shape[0]):
            n = int(lens[b])
            rel = 2 * float(dz[b].max()) + float((4 * U32 * lse[b].abs())[~empty[b]].max() if (~empty[b]).any() else 0)
            e = (gw[b, :, :n] - w[b, :, :n]).abs()
            assert (e <= (rel + 300 * U32) * w[b, :, :n] + 2.0 ** -126).all(), "weights"


# ----------------------------------------------------------------- evict

def evict(k_cache, v_cache, table, lens, weights, positions, next_pos, budget, recent, sink):
    """New (k, v, lens, weights, positions): lists and one copied row at a time.  Entries
    past the new length are -1 positions and 0 weights."""
    k, v = k_cache.clone(), v_cache.clone()
    page = k.shape[2]
    B, Hkv = weights.shape[:2]
    w_out, p_out = torch.zeros_like(weights), torch.full_like(positions, -1)
    new_lens = []
    for b in range(B):
        n = int(lens[b])
        new = min(n, budget)
        new_lens.append(new)
        for h in range(Hkv):
            w, p = weights[b, h, :n].numpy(), positions[b, h, :n].numpy()
            safe = (p < sink) | (p >= int(next_pos[b]) - recent)
            order = np.lexsort((np.arange(n), np.where(safe, 0.0, -w.astype(np.float64)), ~safe))
            kept = set(order[:new].tolist())
            holes = [j for j in range(new) if j not in kept]
            srcs = sorted(j for j in kept if j >= new)
            at = list(range(new))
            for i, j in zip(holes, srcs):
                at[i] = j
                dst, src = int(table[b, i // page]), int(table[b, j // page])
                k[dst, h, i % page] = k_cache[src, h, j % page]
                v[dst, h, i % page] = v_cache[src, h, j % page]
            w_out[b, h, :new] = weights[b, h, at]
            p_out[b, h, :new] = positions[b, h, at]
    return k, v, torch.tensor(new_lens, dtype=torch.int32), w_out, p_out
