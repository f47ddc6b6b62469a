"""Cases of the serving operators around the indexer: the norm that makes its 8-bit rows, the attention
of a decode batch over a shared prefix and private paged caches, and the eviction that keeps those caches
within a budget.  `run` is one call; the plain forms are elementary torch operations."""
import math

import numpy as np
import torch

own = False
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_idx = None


def _package():
    global _idx
    if _idx is None:
        import sparse_attention_indexer_tiles_gb300 as pkg
        _idx = pkg
    return _idx


# ------------------------------------------------------------------ cases

def _norm(rows, cols, residual, group, dt, name=None):
    return {"op": "norm", "rows": rows, "cols": cols, "residual": residual, "group": group, "dt": dt,
            **({"name": name} if name else {})}


def _attn(batch, tokens, group, kv_heads, dim, prefix, lo, hi, weights, page, dt, name=None):
    return {"op": "attn", "batch": batch, "tokens": tokens, "group": group, "kv_heads": kv_heads,
            "dim": dim, "prefix": prefix, "lo": lo, "hi": hi, "weights": weights, "page": page,
            "dt": dt, **({"name": name} if name else {})}


def _evict(batch, kv_heads, dim, lo, hi, budget, recent, sink, page, dt, name=None):
    return {"op": "evict", "batch": batch, "kv_heads": kv_heads, "dim": dim, "lo": lo, "hi": hi,
            "budget": budget, "recent": recent, "sink": sink, "page": page, "dt": dt,
            **({"name": name} if name else {})}


def listed():
    return [
        # one decoded token's hidden row before its projections (scales per 128 columns)
        _norm(1, 4096, True, 128, "bf16", "norm one token"),
        # the index keys of a 65536-token prefill: k and k_scale as the scorer reads them
        _norm(65536, 128, False, 0, "bf16", "norm index keys"),
        # the hidden rows of a 4096-row prefill chunk
        _norm(4096, 8192, True, 128, "bf16", "norm prefill"),
        # a ragged batch of an odd width, one scale per row
        _norm(777, 5000, True, 0, "fp16", "norm odd width"),
        # two short chats behind a short system prompt: latency
        _attn(2, 1, 4, 2, 64, 300, 1, 40, True, 16, "bf16", "attn smallest"),
        # an ordinary decode batch behind a 4096-token system prompt, weights for the eviction
        _attn(16, 1, 4, 8, 128, 4096, 64, 1024, True, 64, "bf16", "attn ordinary"),
        # 64 requests about one long document
        _attn(64, 1, 8, 8, 128, 32768, 64, 1024, False, 64, "bf16", "attn long prefix"),
        # four drafted tokens a request are verified at once; one key head, odd prefix, small heads
        _attn(9, 4, 16, 1, 64, 10001, 33, 2000, False, 32, "fp16", "attn drafted"),
        # long private histories behind a short prompt, weights for the eviction
        _attn(64, 1, 8, 8, 128, 512, 1024, 8192, True, 64, "bf16", "attn private"),
        # the steady state of decoding: every request one token over its budget
        _evict(64, 8, 128, 2049, 2049, 2048, 128, 4, 64, "bf16", "evict one slot"),
        # a 65536-token prefill compacted to the indexer's 2048 keys
        _evict(4, 8, 128, 65536, 65536, 2048, 256, 4, 64, "bf16", "evict after prefill"),
        # a mixed batch, some of it within the budget
        _evict(64, 8, 128, 256, 16384, 1000, 100, 3, 64, "bf16", "evict mixed"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 6.5e12, w["flops"] / 1.5e15)


def draw(rng):
    most = {}
    for c in listed():
        most[c["op"]] = max(most.get(c["op"], 0.0), _cost(c))
    while True:
        op = rng.choice(["norm", "attn", "attn", "evict"])
        if op == "norm":
            group = rng.choice([0, 0, 32, 64, 128])
            cols = _log_int(rng, 64, 16384)
            if group:
                cols = max(1, cols // group) * group
            c = _norm(_log_int(rng, 1, 65536), cols, rng.random() < 0.7, group,
                      rng.choice(["bf16", "bf16", "fp16", "fp32"]))
        elif op == "attn":
            hi = _log_int(rng, 1, 8192)
            c = _attn(_log_int(rng, 1, 64), rng.choice([1, 1, 1, 2, 4, 7]),
                      rng.choice([1, 2, 4, 5, 7, 8, 16]), rng.choice([1, 2, 4, 8]),
                      rng.choice([64, 128, 128]), _log_int(rng, 64, 32768), _log_int(rng, 1, hi), hi,
                      rng.random() < 0.5, rng.choice([16, 32, 64, 64, 128]),
                      rng.choice(["bf16", "bf16", "fp16"]))
        else:
            hi = _log_int(rng, 64, 65536)
            budget = _log_int(rng, 32, hi)
            recent = rng.randint(0, budget // 4)
            c = _evict(_log_int(rng, 1, 64), rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128]),
                       _log_int(rng, 32, hi), hi, budget, recent, rng.randint(0, min(8, budget - recent)),
                       rng.choice([16, 32, 64, 64, 128]), rng.choice(["bf16", "bf16", "fp16"]))
        if _cost(c) <= most[op]:
            return c


def _lens(case):
    """Private lengths of the batch, spread over [lo, hi]: the same ones for every seed, in another order."""
    lo, hi, n = case["lo"], case["hi"], case["batch"]
    return [hi if b == 0 else lo + int((hi - lo) * ((b * 0.6180339887498949) % 1.0)) for b in range(n)]


# ------------------------------------------------------------------ inputs

def _cache(case, pages, g):
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    make = lambda: torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(TYPES[case["dt"]])  # noqa: E731
    return make(), make()


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    if case["op"] == "norm":
        t = TYPES[case["dt"]]
        shape = (case["rows"], case["cols"])
        # hidden states have a few columns that are much larger than the rest
        big = 1.0 + 20.0 * (torch.rand(case["cols"], generator=g, device=DEV) < 0.005).float()
        x = (torch.randn(shape, generator=g, device=DEV) * big).to(t)
        s = {"x": x, "weight": (1.0 + 0.2 * torch.randn(case["cols"], generator=g, device=DEV)).to(t)}
        s["residual"] = (2.0 * torch.randn(shape, generator=g, device=DEV)).to(t) if case["residual"] else None
        s["residual_out"] = torch.empty_like(s["residual"]) if case["residual"] else None
        s["out"] = torch.empty(shape, device=DEV, dtype=torch.float8_e4m3fn)
        s["scale"] = torch.empty((case["rows"], case["cols"] // case["group"]) if case["group"] else (case["rows"],),
                                 device=DEV, dtype=torch.float32)
        return dict(s, case=case, ws=None)
    order = torch.randperm(case["batch"], generator=g, device=DEV)
    lens = torch.tensor(_lens(case), device=DEV, dtype=torch.int32)[order].contiguous()
    most = -(-case["hi"] // case["page"])          # pages of the longest request
    prefix_pages = -(-case.get("prefix", 0) // case["page"])
    pages = prefix_pages + case["batch"] * most
    ids = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    k, v = _cache(case, pages, g)
    s = {"case": case, "k": k, "v": v, "lens": lens, "ws": None,
         "table": ids[prefix_pages:].reshape(case["batch"], most).contiguous()}
    slots = (case["batch"], case["kv_heads"], most * case["page"])
    # what keys have gathered so far: a few hold most of it
    gathered = torch.exp(1.5 * torch.randn(slots, generator=g, device=DEV))
    if case["op"] == "attn":
        heads = case["kv_heads"] * case["group"]
        q = 2.0 * torch.randn((case["batch"], case["tokens"], heads, case["dim"]), generator=g, device=DEV)
        s |= {"q": q.to(TYPES[case["dt"]]), "prefix_table": ids[:prefix_pages].contiguous(),
              "weights": gathered if case["weights"] else None,
              "weights_out": torch.zeros_like(gathered) if case["weights"] else None}
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(q.shape[:3], device=DEV, dtype=torch.float32)
    else:
        at = torch.arange(slots[2], device=DEV, dtype=torch.int32)
        s |= {"weights": gathered, "positions": at.expand(slots).contiguous(), "next_pos": lens.clone(),
              "weights_out": torch.zeros_like(gathered), "lens_out": torch.empty_like(lens)}
        s["positions_out"] = torch.full_like(s["positions"], -1)
    return s


# ------------------------------------------------------------------ the framework's calls

def _run_own(s):
    idx, c = _package(), s["case"]
    if c["op"] == "norm":
        idx.idx_add_rmsnorm_quant(s["x"], s["weight"], residual=s["residual"], residual_out=s["residual_out"],
                                  eps=1e-6, group=c["group"], out=s["out"], scale=s["scale"])
        return [s["out"], s["scale"], s["residual_out"]]
    if c["op"] == "attn":
        if s["ws"] is None:  # the program's workspace, kept with its buffers
            s["ws"] = torch.empty(max(256, idx.idx_prefix_attention_workspace(
                *s["q"].shape[:3], c["kv_heads"], c["dim"], c["prefix"], c["hi"], c["weights"])),
                device=DEV, dtype=torch.uint8)
        idx.idx_prefix_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], prefix_table=s["prefix_table"],
                                 prefix_len=c["prefix"], max_len=c["hi"], weights=s["weights"],
                                 weights_out=s["weights_out"], out=s["out"], lse=s["lse"], ws=s["ws"])
        return [s["out"], s["lse"], s["weights_out"]]
    if s["ws"] is None:
        s["ws"] = torch.empty(max(256, idx.idx_cache_evict_workspace(
            c["batch"], c["kv_heads"], c["budget"], c["hi"])), device=DEV, dtype=torch.uint8)
    idx.idx_cache_evict(s["k"], s["v"], s["table"], s["lens"], s["weights"], s["positions"], s["next_pos"],
                        c["budget"], recent=c["recent"], sink=c["sink"], max_len=c["hi"],
                        lens_out=s["lens_out"], weights_out=s["weights_out"],
                        positions_out=s["positions_out"], ws=s["ws"])
    return [s["lens_out"], s["weights_out"], s["positions_out"], s["k"], s["v"]]


# ------------------------------------------------------------------ the plain forms

def _plain_norm(s):
    c, t = s["case"], s["x"].dtype
    # 64 bits: a code next to a rounding border has to fall on the right side of it
    h = s["x"].double() + (s["residual"].double() if s["residual"] is not None else 0.0)
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + 1e-6) * s["weight"].double()
    y = y.reshape(c["rows"], -1, c["group"] or c["cols"])
    scale = (y.abs().amax(2, keepdim=True) / 448.0).clamp_min(2.0 ** -100).float()
    codes = (y / scale.double()).clamp(-448.0, 448.0).float().to(torch.float8_e4m3fn).reshape(c["rows"], -1)
    scale = scale[:, :, 0] if c["group"] else scale[:, 0, 0]
    return [codes, scale.contiguous(), h.to(t) if s["residual"] is not None else None]


def _rows_of(cache, table):
    """[..., heads, slots, dim] in 32 bits of the pages that table [..., pages] names."""
    x = cache[table.long()].float().transpose(-4, -3)
    return x.reshape(*x.shape[:-3], x.shape[-3] * x.shape[-2], x.shape[-1])


def _plain_attn(s):
    c = s["case"]
    B, Q, G, K, D, P = c["batch"], c["tokens"], c["group"], c["kv_heads"], c["dim"], c["prefix"]
    # [K, B * Q * G, D]: the batch's rows of a key head share the prefix
    q = s["q"].float().reshape(B, Q, K, G, D) * D ** -0.5
    qp = q.permute(2, 0, 1, 3, 4).reshape(K, B * Q * G, D)
    kp, vp = _rows_of(s["k"], s["prefix_table"])[:, :P], _rows_of(s["v"], s["prefix_table"])[:, :P]
    sp = (qp @ kp.transpose(1, 2)).reshape(K, B, Q, G, P)
    ks, vs = _rows_of(s["k"], s["table"]), _rows_of(s["v"], s["table"])
    N = ks.shape[2]
    ss = (q.permute(0, 2, 1, 3, 4).reshape(B, K, Q * G, D) @ ks.transpose(2, 3)).reshape(B, K, Q, G, N)
    at = torch.arange(N, device=DEV)
    sees = s["lens"].long()[:, None] - (Q - 1) + torch.arange(Q, device=DEV)     # [B, Q]
    ss = ss.masked_fill((at >= sees[:, :, None])[:, None, :, None, :], -math.inf).permute(1, 0, 2, 3, 4)
    m = torch.maximum(sp.amax(4), ss.amax(4))
    ep, es = torch.exp(sp - m[..., None]), torch.exp(ss - m[..., None])
    total = ep.sum(4) + es.sum(4)
    o = (ep.reshape(K, B * Q * G, P) @ vp).reshape(K, B, Q, G, D)
    o = o + (es.transpose(0, 1).reshape(B, K, Q * G, N) @ vs).reshape(B, K, Q, G, D).transpose(0, 1)
    o = (o / total[..., None]).permute(1, 2, 0, 3, 4).reshape(B, Q, K * G, D).to(s["q"].dtype)
    lse = (m + torch.log(total)).permute(1, 2, 0, 3).reshape(B, Q, K * G)
    if s["weights"] is None:
        return [o, lse, None]
    got = (es / total[..., None]).sum((2, 3)).transpose(0, 1)                    # [B, K, N]
    n = s["lens"].long()[:, None, None]
    w = torch.where(at < n - Q, s["weights"], 0.0) + got
    return [o, lse, torch.where(at < n, w, 0.0)]


def _plain_evict(s):
    c = s["case"]
    w, pos, n = s["weights"], s["positions"], s["lens"].long()[:, None, None]
    slots, budget = w.shape[2], c["budget"]
    at = torch.arange(slots, device=DEV)
    guarded = (pos < c["sink"]) | (pos >= s["next_pos"][:, None, None] - c["recent"])
    rank = torch.where(guarded, math.inf, w).masked_fill(at >= n, -math.inf)
    order = torch.sort(rank, dim=2, descending=True, stable=True).indices
    room = min(budget, slots)
    keep = torch.zeros(w.shape, dtype=torch.bool, device=DEV).scatter_(2, order[:, :, :room], True) & (at < n)
    new = torch.clamp(n, max=budget)
    hole = ~keep & (at < new)
    moves = keep & (at >= new)
    # the i-th hole takes the i-th kept slot above the budget
    dst, src = hole.nonzero(), moves.nonzero()
    to, frm = dst.unbind(1), src.unbind(1)
    w_out = torch.where(at < new, w, 0.0)
    pos_out = torch.where(at < new, pos, -1)
    w_out[to], pos_out[to] = w[frm], pos[frm]
    table, page = s["table"].long(), c["page"]
    for cache in (s["k"], s["v"]):
        cache[table[to[0], to[2] // page], to[1], to[2] % page] = \
            cache[table[frm[0], frm[2] // page], frm[1], frm[2] % page]
    return [new[:, 0, 0].to(torch.int32), w_out, pos_out, s["k"], s["v"]]


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _plain_norm, "attn": _plain_attn, "evict": _plain_evict}[state["case"]["op"]](state)


# ------------------------------------------------------------------ work and the exact values

def work(case):
    es = 4 if case["dt"] == "fp32" else 2
    if case["op"] == "norm":
        n = case["rows"] * case["cols"]
        scales = n // case["group"] if case["group"] else case["rows"]
        return {"bytes": n * (es * (3 if case["residual"] else 1) + 1) + 4 * scales + es * case["cols"],
                "flops": 8 * n}
    lens, K, D = _lens(case), case["kv_heads"], case["dim"]
    if case["op"] == "attn":
        B, Q, H = case["batch"], case["tokens"], case["kv_heads"] * case["group"]
        seen = sum(max(0, n - Q + 1 + t) for n in lens for t in range(Q))
        return {"bytes": (case["prefix"] + sum(lens)) * K * D * 2 * es + 2 * B * Q * H * D * es + 4 * B * Q * H
                + (8 * K * sum(lens) if case["weights"] else 0),
                "flops": 4 * D * H * (B * Q * case["prefix"] + seen)}
    moved = 0.0
    for n in lens:
        if n > case["budget"]:
            free = max(1, n - case["sink"] - case["recent"])      # slots that compete by their weight
            above = max(0, n - case["budget"] - case["recent"])   # of them, those above the budget
            moved += min(case["recent"], n - case["budget"]) + (case["budget"] - case["sink"] - case["recent"]) * above / free
    table = 8 * K * sum(n + min(n, case["budget"]) for n in lens)
    return {"bytes": table + moved * K * 4 * D * es, "flops": 16 * K * sum(lens)}


def _exact_norm(s):
    c = s["case"]
    codes, scales, sums = [], [], []
    for lo in range(0, c["rows"], 4096):
        h = s["x"][lo:lo + 4096].to(torch.float64)
        if s["residual"] is not None:
            h = h + s["residual"][lo:lo + 4096].to(torch.float64)
            sums.append(h)
        y = s["weight"].to(torch.float64) * h / torch.sqrt(torch.linalg.vector_norm(h, dim=1) ** 2 / c["cols"] + 1e-6)[:, None]
        parts = torch.stack(y.split(c["group"] or c["cols"], 1), 1)
        scale = torch.clamp(parts.abs().amax(2) / 448, min=2.0 ** -100)
        # e4m3 has three fraction bits down to the exponent -6
        v = parts / scale.float().double()[:, :, None]
        step = torch.exp2(torch.clamp(torch.frexp(v)[1] - 1, min=-6).double() - 3)
        codes.append(torch.clamp(torch.round(v / step) * step, -448, 448).reshape(y.shape))
        scales.append(scale if c["group"] else scale[:, 0])
    return [torch.cat(codes), torch.cat(scales), torch.cat(sums) if sums else None]


def _exact_attn(s):
    c = s["case"]
    Q, G, K, P, page = c["tokens"], c["group"], c["kv_heads"], c["prefix"], c["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    w = None if s["weights"] is None else torch.zeros(s["weights"].shape, dtype=torch.float64, device=DEV)
    slot = torch.arange(P, device=DEV)
    prefix = [x[s["prefix_table"].long()[slot // page], :, slot % page].double() for x in (s["k"], s["v"])]
    for b, n in enumerate(s["lens"].tolist()):
        slot = torch.arange(n, device=DEV)
        k, v = (torch.cat([p, x[s["table"][b].long()[slot // page], :, slot % page].double()])
                for p, x in zip(prefix, (s["k"], s["v"])))
        for h in range(K):
            heads = slice(h * G, h * G + G)
            z = torch.einsum("tgd,nd->tgn", s["q"][b, :, heads].double(), k[:, h]) / math.sqrt(c["dim"])
            for t in range(Q):
                z[t, :, P + max(0, n - (Q - 1 - t)):] = -math.inf
            p = torch.softmax(z, 2)
            out[b, :, heads] = torch.einsum("tgn,nd->tgd", p, v[:, h])
            lse[b, :, heads] = torch.logsumexp(z, 2)
            if w is not None:
                w[b, h, :n] = p[:, :, P:].sum((0, 1))
                old = max(0, n - Q)
                w[b, h, :old] += s["weights"][b, h, :old].double()
    return [out, lse, w]


def _exact_evict(s):
    """By sorting on the host; the caches' rows are moved one request and head at a time."""
    c = s["case"]
    w_out, p_out = torch.zeros_like(s["weights"], dtype=torch.float64), torch.full_like(s["positions"], -1)
    k, v = s["k"].clone(), s["v"].clone()
    lens, page = s["lens"].tolist(), c["page"]
    for b, n in enumerate(lens):
        new = min(n, c["budget"])
        for h in range(c["kv_heads"]):
            w, pos = s["weights"][b, h, :n].double().cpu().numpy(), s["positions"][b, h, :n].cpu().numpy()
            guarded = (pos < c["sink"]) | (pos >= n - c["recent"])
            kept = np.sort(np.lexsort((np.arange(n), np.where(guarded, 0.0, -w), ~guarded))[:new])
            frm = kept[kept >= new]
            to = np.setdiff1d(np.arange(new), kept)
            w_out[b, h, :new], p_out[b, h, :new] = s["weights"][b, h, :new].double(), s["positions"][b, h, :new]
            if len(to):
                i, j = torch.from_numpy(to).to(DEV), torch.from_numpy(frm).to(DEV)
                w_out[b, h, i], p_out[b, h, i] = s["weights"][b, h, j].double(), s["positions"][b, h, j]
                t = s["table"][b].long()
                for new_cache, cache in ((k, s["k"]), (v, s["v"])):
                    new_cache[t[i // page], h, i % page] = cache[t[j // page], h, j % page]
    return [torch.tensor([min(n, c["budget"]) for n in lens], dtype=torch.int32, device=DEV), w_out, p_out,
            k.double(), v.double()]


def exact(case, seed):
    return {"norm": _exact_norm, "attn": _exact_attn, "evict": _exact_evict}[case["op"]](prepare(case, seed))
