"""Cases of the operators of a paged cache held in 4 bits: the append that writes it, the attention that reads it
(with a sliding window and first tokens that stay visible), and the calls that say which request holds which page
(fork, resize, compact).  `run` is one call; the plain forms are elementary torch operations.

A cache in 4 bits is MXFP4: e2m1 codes two per byte, element 2i in the low nibble, and one e8m0 scale per 32
elements.  The format fixes every bit of what the append writes, so it is returned as the bytes themselves."""
import math

import numpy as np
import torch

own = False
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_idx = None


def _package():
    global _idx
    if _idx is None:
        import sparse_attention_indexer_tiles_gb300 as pkg
        _idx = pkg
    return _idx


# ------------------------------------------------------------------ cases

def _append(batch, lo, hi, q_lo, q_hi, kv_heads, dim, page, dt, fused, name=None):
    return {"op": "append", "batch": batch, "lo": lo, "hi": hi, "q_lo": q_lo, "q_hi": q_hi, "kv_heads": kv_heads,
            "dim": dim, "page": page, "dt": dt, "fused": fused, **({"name": name} if name else {})}


def _attn(batch, lo, hi, q_lo, q_hi, group, kv_heads, dim, window, sink, page, dt, behind=0, name=None):
    return {"op": "attn", "batch": batch, "lo": lo, "hi": hi, "q_lo": q_lo, "q_hi": q_hi, "group": group,
            "kv_heads": kv_heads, "dim": dim, "window": window, "sink": sink, "page": page, "dt": dt,
            "behind": behind, **({"name": name} if name else {})}


def _fork(groups, beams, prompt, hi, page, name=None):
    return {"op": "fork", "groups": groups, "beams": beams, "prompt": prompt, "hi": hi, "page": page,
            **({"name": name} if name else {})}


def _resize(batch, lo, hi, turn, shared, spare, kv_heads, dim, page, name=None):
    return {"op": "resize", "batch": batch, "lo": lo, "hi": hi, "turn": turn, "shared": shared, "spare": spare,
            "kv_heads": kv_heads, "dim": dim, "page": page, **({"name": name} if name else {})}


def _compact(batch, lo, hi, spare, kv_heads, dim, page, name=None):
    return {"op": "compact", "batch": batch, "lo": lo, "hi": hi, "spare": spare, "kv_heads": kv_heads, "dim": dim,
            "page": page, **({"name": name} if name else {})}


def listed():
    return [
        # a decode step's new keys and values, one token for each of 64 requests
        _append(64, 1, 4096, 1, 1, 8, 128, 64, "bf16", False, "append one token each"),
        # four prompts at once, keys and values as slices of the fused projection
        _append(4, 1000, 16384, 1000, 16384, 8, 128, 64, "bf16", True, "append prompts"),
        # two short chats: latency
        _attn(2, 1, 40, 1, 1, 4, 2, 64, 0, 0, 16, "bf16", name="attn smallest"),
        # a decode batch over its whole history
        _attn(64, 1024, 32768, 1, 1, 8, 8, 128, 0, 0, 64, "bf16", name="attn decode"),
        # a decode batch of long streams with a window and four first tokens
        _attn(16, 32768, 131072, 1, 1, 4, 8, 128, 4096, 4, 64, "fp16", name="attn long window"),
        # ragged prompts behind an earlier chunk, windowed layer, padded to a round number of tokens
        _attn(3, 3000, 10000, 1500, 8192, 8, 8, 128, 1024, 4, 64, "bf16", behind=37, name="attn prompts"),
        # beam search on one request
        _fork(1, 4, 300, 500, 16, "fork one request"),
        # beam search on 128 requests of up to 32768 tokens
        _fork(128, 8, 4096, 32768, 16, "fork beams"),
        # a decode step: every request grows by a token, some into a page they share since a fork
        _resize(256, 16, 4096, False, 32, 1000, 8, 64, 16, "resize one step"),
        # requests leave, others come, drafts are taken back
        _resize(512, 64, 16384, True, 128, 4000, 1, 128, 64, "resize turn-over"),
        # a small pool after its requests have come and gone
        _compact(8, 100, 1000, 150, 2, 64, 16, "compact small"),
        # a pool of 2 GB, half of it live
        _compact(64, 256, 8192, 4000, 8, 128, 64, "compact pool"),
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
        op = rng.choice(["append", "attn", "attn", "attn", "fork", "resize", "compact"])
        heads, dim, page = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 64, 128])
        dt = rng.choice(["bf16", "bf16", "fp16"])
        if op in ("append", "attn"):
            hi = _log_int(rng, 1, 131072 if op == "attn" else 16384)
            lo = _log_int(rng, 1, hi)
            kind = rng.random()
            q_hi = 1 if kind < 0.5 else rng.randint(1, 16) if kind < 0.7 else _log_int(rng, 1, 8192)
            q_hi = min(q_hi, lo)
            q_lo = _log_int(rng, 1, q_hi)
            batch = _log_int(rng, 1, 64)
            window = rng.choice([0, _log_int(rng, 1, 8192)])
            if op == "append":
                c = _append(batch, lo, hi, q_lo, q_hi, heads, dim, page, dt, rng.random() < 0.5)
            else:
                c = _attn(batch, lo, hi, q_lo, q_hi, rng.choice([1, 2, 4, 5, 7, 8, 16]), heads, dim, window,
                          rng.randint(0, 64) if window else 0, page, dt, rng.choice([0, 0, 5]))
            small = batch * hi * heads * dim <= 1 << 31
            # the scores of one request and key head, in 32 bits
            if op == "attn":
                small = small and q_hi * c["group"] * hi <= 1 << 30
        elif op == "fork":
            hi = _log_int(rng, 1, 32768)
            c = _fork(_log_int(rng, 1, 128), rng.randint(1, 8), _log_int(rng, 1, hi), hi, page)
            small = True
        else:
            hi = _log_int(rng, 1, 32768)
            lo, batch = _log_int(rng, 1, hi), _log_int(rng, 1, 512)
            spare = _log_int(rng, 1, 4000)
            if op == "resize":
                c = _resize(batch, lo, hi, rng.random() < 0.5, rng.randint(0, batch // 2), spare, heads, dim, page)
            else:
                c = _compact(batch, lo, hi, spare, heads, dim, page)
            small = (batch * (lo + hi) / 2 * 1.3 + spare * page) * heads * dim <= 1 << 29
        if small and _cost(c) <= most[op]:
            return c


def _spread(lo, hi, n):
    """n whole numbers over [lo, hi], the first of them hi: the same ones for every seed."""
    return [hi if b == 0 else lo + int((hi - lo) * ((b * 0.6180339887498949) % 1.0)) for b in range(n)]


def _tokens(case):
    """(cached lengths with the new tokens, new tokens) of a batch of requests."""
    lens, new = _spread(case["lo"], case["hi"], case["batch"]), _spread(case["q_lo"], case["q_hi"], case["batch"])
    return lens, [min(n, q) for n, q in zip(lens, new)]


def _resize_lens(case):
    """(lengths, new lengths); row 2i + 1 is a fork of row 2i for the first `shared` pairs."""
    lens = _spread(case["lo"], case["hi"], case["batch"])
    for i in range(case["shared"]):
        lens[2 * i + 1] = lens[2 * i]
    new = []
    for i, n in enumerate(lens):
        kind = (i * 7 // 2) % 5 if case["turn"] else 1
        # a request ends; grows by a token; by a chunk; takes a draft back; comes in a reused row
        new.append((0, n + 1, n + 777, max(0, n - 3), max(1, n // 2))[kind])
    return lens, new


def _pages(n, page):
    return -(-n // page)


def _copies(case):
    """How many partly filled shared pages such a resize copies."""
    lens, new = _resize_lens(case)
    page, count = case["page"], 0
    for i in range(case["shared"]):
        a, b = 2 * i, 2 * i + 1
        n = lens[a]
        if n % page == 0:
            continue
        holds = [_pages(new[j], page) >= _pages(n, page) for j in (a, b)]
        if all(holds):
            count += sum(new[j] > n for j in (a, b))
    return count


# ------------------------------------------------------------------ inputs

def _codes(shape, g):
    """Codes of normal values under a block scale near their spread: byte pairs drawn through a table."""
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    v = 2.2 * torch.erfinv(torch.linspace(-0.9961, 0.9961, 256, device=DEV)) * math.sqrt(2.0)
    nibble = torch.bucketize(v.abs(), edges) + 8 * (v < 0)
    byte = (nibble[:, None] + 16 * nibble[None, :]).reshape(-1).to(torch.uint8)
    out = torch.empty(shape, dtype=torch.uint8, device=DEV)
    flat = out.view(-1)
    for lo in range(0, flat.numel(), 1 << 28):
        n = min(1 << 28, flat.numel() - lo)
        flat[lo:lo + n] = byte[torch.randint(0, 65536, (n,), generator=g, device=DEV, dtype=torch.int32)]
    return out


def _scales(shape, g):
    """Block scales: most near 1/2, a few blocks (outlier columns, first tokens) larger."""
    r = torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8)
    return 125 + (r >= 64).to(torch.uint8) + (r >= 224).to(torch.uint8) + 2 * (r >= 254).to(torch.uint8)


def _prepare_tokens(case, g):
    lens, new = _tokens(case)
    order = torch.randperm(case["batch"], generator=g, device=DEV).tolist()
    lens, new = [lens[i] for i in order], [new[i] for i in order]
    page, heads, dim = case["page"], case["kv_heads"], case["dim"]
    most = _pages(case["hi"], page)
    pages = sum(_pages(n, page) for n in lens) + 1
    ids = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((case["batch"], most), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(lens):
        table[b, :_pages(n, page)] = ids[at:at + _pages(n, page)]
        at += _pages(n, page)
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    s = {"case": case, "table": table, "lens": torch.tensor(lens, dtype=torch.int32, device=DEV),
         "q_start": torch.from_numpy(starts).to(DEV), "ws": None}
    shape = (pages, heads, page)
    t = TYPES[case["dt"]]
    if case["op"] == "append":
        for name in ("k_codes", "v_codes"):
            s[name] = torch.zeros(*shape, dim // 2, dtype=torch.uint8, device=DEV)
        for name in ("k_sf", "v_sf"):
            s[name] = torch.zeros(*shape, dim // 32, dtype=torch.uint8, device=DEV)
        width = heads * dim
        # a fused projection's rows hold four times as many query columns before the keys and the values
        x = torch.empty(int(starts[-1]), 6 * width if case["fused"] else 2 * width, dtype=t, device=DEV)
        big = 1.0 + 10.0 * (torch.rand(width, generator=g, device=DEV) < 0.01).float()
        for part in (x[:, -2 * width:-width], x[:, -width:]):
            part.copy_(torch.randn(part.shape, generator=g, device=DEV) * big)
        s["k"], s["v"] = (p.unflatten(1, (heads, dim)) for p in (x[:, -2 * width:-width], x[:, -width:]))
        return s
    for name in ("k", "v"):
        s[name + "_codes"], s[name + "_sf"] = _codes((*shape, dim // 2), g), _scales((*shape, dim // 32), g)
    rows = int(starts[-1]) + case["behind"]
    q = 1.5 * torch.randn((rows, heads * case["group"], dim), generator=g, device=DEV)
    s["q"] = q.to(t)
    s["out"] = torch.zeros_like(s["q"])
    s["lse"] = torch.zeros(q.shape[:2], dtype=torch.float32, device=DEV)
    return s


def _used(lens, page, width):
    """[rows, width]: the entries of a page table that lengths take."""
    return torch.arange(width, device=DEV) < ((lens.long() + page - 1) // page)[:, None]


def _refs(table, lens, page, pages):
    return torch.bincount(table[_used(lens, page, table.shape[1])].long(), minlength=pages).to(torch.int32)


def _pool(case, pages, g):
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    return [torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(generator=g) for _ in range(2)]


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    if case["op"] in ("append", "attn"):
        return _prepare_tokens(case, g)
    page = case["page"]
    if case["op"] == "fork":
        groups, beams = case["groups"], case["beams"]
        rows, hi, prompt = groups * beams, case["hi"], min(case["prompt"], case["hi"])
        per_group = [n for n in _spread(prompt, hi, groups) for _ in range(beams)]
        width, shared = _pages(hi, page), prompt // page
        lens = torch.tensor(per_group, dtype=torch.int32, device=DEV)
        pages = groups * (shared + beams * (width - shared))
        ids = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        table = torch.cat([ids[:groups * shared].view(groups, 1, shared).expand(groups, beams, shared),
                           ids[groups * shared:].view(groups, beams, width - shared)], 2).reshape(rows, width)
        # every beam goes on from one of its group; some requests end
        pick = torch.randint(0, beams, (groups, beams), generator=g, device=DEV)
        parent = (pick + beams * torch.arange(groups, device=DEV)[:, None]).view(-1)
        parent[torch.rand(rows, generator=g, device=DEV) < 0.02] = -1
        s = {"parent": parent.to(torch.int32)}
    else:
        if case["op"] == "resize":
            old, new = _resize_lens(case)
            shared = case["shared"]
        else:
            old, new, shared = _spread(case["lo"], case["hi"], case["batch"]), None, 0
        width = _pages(max(old + (new or [])), page)
        used = sum(_pages(n, page) for n in old)
        pages = used + 2 * shared + case["spare"] + (sum(max(0, _pages(m, page) - _pages(n, page)) for n, m in zip(old, new)) if new else 0)
        ids = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        lens = torch.tensor(old, dtype=torch.int32, device=DEV)
        table = torch.full((case["batch"], width), -1, dtype=torch.int32, device=DEV)
        table[_used(lens, page, width)] = ids[:used]
        if shared:
            table[1:2 * shared:2] = table[0:2 * shared:2]
        s = {"caches": _pool(case, pages, g)}
        if new:
            s["new_lens"] = torch.tensor(new, dtype=torch.int32, device=DEV)
        else:
            s["live"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    table = table.contiguous()
    s |= {"case": case, "table": table, "lens": lens, "refs": _refs(table, lens, page, pages), "ws": None,
          "table_out": torch.full_like(table, -1), "lens_out": torch.zeros_like(lens)}
    s["refs_out"] = torch.zeros_like(s["refs"])
    return s


# ------------------------------------------------------------------ the framework's calls

def _workspace(s, need):
    if s["ws"] is None:  # the program's workspace, kept with its buffers
        s["ws"] = torch.empty(max(256, need), device=DEV, dtype=torch.uint8)
    return s["ws"]


def _run_own(s):
    idx, c = _package(), s["case"]
    if c["op"] == "append":
        idx.idx_cache_append_mxfp4(s["k"], s["v"], s["k_codes"], s["k_sf"], s["v_codes"], s["v_sf"], s["table"],
                                   s["lens"], q_start=s["q_start"])
        return [s["k_codes"], s["k_sf"], s["v_codes"], s["v_sf"]]
    if c["op"] == "attn":
        rows, heads, dim = s["q"].shape
        ws = _workspace(s, idx.idx_window_attention_mxfp4_workspace(
            c["batch"], rows, c["q_hi"], heads, c["kv_heads"], dim, c["hi"], c["window"], c["sink"])
            if s["ws"] is None else 0)
        idx.idx_window_attention_mxfp4(s["q"], s["k_codes"], s["k_sf"], s["v_codes"], s["v_sf"], s["table"], s["lens"],
                                       q_start=s["q_start"], max_q=c["q_hi"], max_len=c["hi"], window=c["window"],
                                       sink=c["sink"], out=s["out"], lse=s["lse"], ws=ws)
        return [s["out"], s["lse"]]
    outs = {"refs_out": s["refs_out"], "table_out": s["table_out"]}
    if c["op"] == "fork":
        idx.idx_cache_fork(s["refs"], s["table"], s["lens"], s["parent"], page_size=c["page"],
                           lens_out=s["lens_out"], **outs)
        return [s["refs_out"], s["table_out"], s["lens_out"]]
    rows, width = s["table"].shape
    if c["op"] == "resize":
        ws = _workspace(s, idx.idx_cache_resize_workspace(rows, s["refs"].numel(), width) if s["ws"] is None else 0)
        idx.idx_cache_resize(s["caches"], s["refs"], s["table"], s["lens"], s["new_lens"], page_size=c["page"],
                             lens_out=s["lens_out"], ws=ws, **outs)
        return [s["refs_out"], s["table_out"], s["lens_out"], *s["caches"]]
    ws = _workspace(s, idx.idx_cache_compact_workspace(rows, s["refs"].numel()) if s["ws"] is None else 0)
    idx.idx_cache_compact(s["caches"], s["refs"], s["table"], s["lens"], page_size=c["page"], live=s["live"], ws=ws,
                          **outs)
    return [s["refs_out"], s["table_out"], s["live"], *s["caches"]]


# ------------------------------------------------------------------ the plain forms

def _quantise(x):
    """(codes [..., D / 2], scales [..., D / 32]) of x [..., D]; powers of two, so 32 bits are exact."""
    y = x.float().unflatten(-1, (-1, 32))
    top = y.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, torch.frexp(top)[1] - 3, 0).clamp(-127, 127)
    # in two steps: 2^-e alone may not be a normal number
    y = torch.ldexp(torch.ldexp(y, -(e // 2)), -(e - e // 2))
    a = y.abs()
    code = sum((a > edge if tie_down else a >= edge).to(torch.uint8) for edge, tie_down in (
        (0.25, True), (0.75, False), (1.25, True), (1.75, False), (2.5, True), (3.5, False), (5.0, True)))
    code = (code + 8 * torch.signbit(y).to(torch.uint8)).flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], (e[..., 0] + 127).to(torch.uint8)


def _plain_append(s):
    page, n = s["case"]["page"], s["k"].shape[0]
    start = s["q_start"].long()
    token = torch.arange(n, device=DEV)
    request = torch.searchsorted(start[1:], token, right=True)
    position = s["lens"].long()[request] - start[request + 1] + token
    where = s["table"].long()[request, position // page]
    for name in ("k", "v"):
        codes, sf = _quantise(s[name])
        s[name + "_codes"][where, :, position % page] = codes
        s[name + "_sf"][where, :, position % page] = sf
    return [s["k_codes"], s["k_sf"], s["v_codes"], s["v_sf"]]


def _values(codes, sf, table, slots, page):
    """[heads, slots, D] in 32 bits of a request's cached rows."""
    where = table.long()[slots // page]
    c, f = codes[where, :, slots % page], sf[where, :, slots % page]
    lut = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=DEV)
    x = torch.stack([lut[(c & 15).int()], lut[(c >> 4).int()]], -1).flatten(-2)
    return torch.ldexp(x.unflatten(-1, (-1, 32)), f[..., None].int() - 127).flatten(-2).transpose(0, 1)


def _plain_attn(s):
    c = s["case"]
    G, K, D, W, S, page = c["group"], c["kv_heads"], c["dim"], c["window"], c["sink"], c["page"]
    out, lse = torch.zeros_like(s["q"]), torch.zeros_like(s["lse"])
    start = s["q_start"].tolist()
    for b, n in enumerate(s["lens"].tolist()):
        new = start[b + 1] - start[b]
        if W:  # the first tokens, and from the oldest row's window on
            slots = torch.arange(n, device=DEV)
            slots = slots[(slots < S) | (slots > n - new - W)]
        else:
            slots = torch.arange(n, device=DEV)
        k = _values(s["k_codes"], s["k_sf"], s["table"][b], slots, page)
        v = _values(s["v_codes"], s["v_sf"], s["table"][b], slots, page)
        pos = torch.arange(n - new, n, device=DEV)[:, None]
        hidden = slots > pos
        if W:
            hidden |= (slots >= S) & (slots <= pos - W)
        for h in range(K):
            q = s["q"][start[b]:start[b + 1], h * G:(h + 1) * G].float() * D ** -0.5
            z = (q.transpose(0, 1).reshape(G * new, D) @ k[h].T).view(G, new, -1)
            z.masked_fill_(hidden, -math.inf)
            m = z.amax(2, keepdim=True)
            e = torch.exp(z - m)
            total = e.sum(2, keepdim=True)
            o = (e.view(G * new, -1) @ v[h]).view(G, new, D) / total
            out[start[b]:start[b + 1], h * G:(h + 1) * G] = o.transpose(0, 1).to(out.dtype)
            lse[start[b]:start[b + 1], h * G:(h + 1) * G] = (m + torch.log(total))[:, :, 0].T
    return [out, lse]


def _plain_fork(s):
    page, width = s["case"]["page"], s["table"].shape[1]
    parent = s["parent"].long()
    lens = torch.where(parent >= 0, s["lens"][parent.clamp_min(0)], 0)
    table = torch.where(_used(lens, page, width), s["table"][parent.clamp_min(0)], -1)
    refs = s["refs"].clone()
    for t, n, sign in ((s["table"], s["lens"], -1), (table, lens, 1)):
        held = t[_used(n, page, width)].long()
        refs.index_add_(0, held, torch.full_like(held, sign, dtype=torch.int32))
    return [refs, table, lens]


def _plain_resize(s):
    page, (rows, width) = s["case"]["page"], s["table"].shape
    old, new, table, refs = s["lens"].long(), s["new_lens"].long(), s["table"].clone(), s["refs"].clone()
    have, want = _used(old, page, width), _used(new, page, width)
    held = table[have & ~want].long()
    refs.index_add_(0, held, torch.full_like(held, -1, dtype=torch.int32))
    # a partly filled last page that others hold too
    last = (old - 1).clamp_min(0) // page
    at = table[torch.arange(rows, device=DEV), last].long()
    copy = (new > old) & (old % page != 0) & (refs[at.clamp_min(0)] > 1)
    needs = copy.long() + (want & ~have).sum(1)
    free = (refs <= 0).nonzero()[:, 0]
    ends = torch.cumsum(needs, 0)
    served = (needs == 0) | (ends <= free.numel())
    takes = want & ~have & served[:, None]
    takes[torch.arange(rows, device=DEV), last] |= copy & served
    rank = torch.cumsum(takes.view(-1), 0).view(rows, width) - 1
    copied = copy & served
    refs.index_add_(0, at[copied], torch.full_like(at[copied], -1, dtype=torch.int32))
    refs[free[:int(takes.sum())]] = 1
    table[takes] = free[rank[takes]].to(torch.int32)
    for cache in s["caches"]:
        cache[table[copied, last[copied]].long()] = cache[at[copied]]
    lens = torch.where(served, new, old)
    return [refs, torch.where(_used(lens, page, width), table, -1), lens.to(torch.int32), *s["caches"]]


def _plain_compact(s):
    page, width, refs = s["case"]["page"], s["table"].shape[1], s["refs"]
    used = refs > 0
    live = used.sum()
    at = torch.arange(refs.numel(), device=DEV)
    holes, movers = (~used & (at < live)).nonzero()[:, 0], (used & (at >= live)).nonzero()[:, 0]
    to = at.clone()
    to[movers] = holes
    refs_out = torch.where(used & (at < live), refs, 0)
    refs_out[holes] = refs[movers]
    for cache in s["caches"]:
        cache[holes] = cache[movers]
    taken = _used(s["lens"], page, width)
    table = torch.where(taken, to[s["table"].clamp_min(0).long()].to(torch.int32), -1)
    return [refs_out, table, live.to(torch.int32).view(1), *s["caches"]]


_PLAIN = {"append": _plain_append, "attn": _plain_attn, "fork": _plain_fork, "resize": _plain_resize,
          "compact": _plain_compact}


def run(state):
    if own:
        return _run_own(state)
    return _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ work and the exact values

def _seen(case, n, new):
    """(pairs of a new token and a key it sees, keys that one of them sees) of a request."""
    W, S = case["window"], case["sink"]
    if not W:
        return sum(range(n - new + 1, n + 1)), n
    pairs = sum(min(p + 1, W) + min(S, max(0, p + 1 - W)) for p in range(n - new, n))
    keys = min(n, W + new - 1)
    return pairs, keys + min(S, n - keys)


def work(case):
    op, page = case["op"], case["page"]
    if op in ("append", "attn"):
        lens, new = _tokens(case)
        K, D, T = case["kv_heads"], case["dim"], sum(new)
        row = 2 * (D // 2 + D // 32)
        if op == "append":
            return {"bytes": T * K * (4 * D + row) + 12 * case["batch"], "flops": 8 * T * K * D}
        seen = [_seen(case, n, q) for n, q in zip(lens, new)]
        H = K * case["group"]
        return {"bytes": sum(k for _, k in seen) * K * row + T * H * (4 * D + 4) + 12 * case["batch"],
                "flops": 4 * D * H * sum(p for p, _ in seen)}
    if op == "fork":
        per = [_pages(n, page) for n in _spread(min(case["prompt"], case["hi"]), case["hi"], case["groups"])]
        entries, rows = sum(per) * case["beams"], case["groups"] * case["beams"]
        shared = min(case["prompt"], case["hi"]) // page
        pages = case["groups"] * (shared + case["beams"] * (_pages(case["hi"], page) - shared))
        return {"bytes": 8 * entries + 8 * pages + 12 * rows, "flops": 2 * entries}
    size = 4 * case["kv_heads"] * page * case["dim"]        # K and V of a page, 16-bit
    if op == "resize":
        old, new = _resize_lens(case)
        entries = sum(_pages(n, page) + _pages(m, page) for n, m in zip(old, new))
        pages = sum(max(_pages(n, page), _pages(m, page)) for n, m in zip(old, new)) + 2 * case["shared"] + case["spare"]
        return {"bytes": 4 * entries + 8 * pages + 12 * case["batch"] + 2 * size * _copies(case), "flops": entries + pages}
    used = sum(_pages(n, page) for n in _spread(case["lo"], case["hi"], case["batch"]))
    pages = used + case["spare"]
    moved = used * (1 - used / pages)                       # of live pages in any order, those above the live count
    return {"bytes": 8 * used + 8 * pages + 2 * size * moved, "flops": used + pages}


def _exact_append(s):
    """Block by block through the nearest of the sixteen values, in 64 bits on the host."""
    c, out = s["case"], []
    start, lens, table = s["q_start"].tolist(), s["lens"].tolist(), s["table"].cpu().numpy()
    where = np.concatenate([np.arange(n - (b - a), n) for n, a, b in zip(lens, start, start[1:])])
    request = np.repeat(np.arange(c["batch"]), np.diff(start))
    pages, offsets = table[request, where // c["page"]], where % c["page"]
    grid = np.array(MAGNITUDES)
    for name in ("k", "v"):
        codes, sfs = (s[name + part].cpu().numpy().copy() for part in ("_codes", "_sf"))
        x = s[name].double().cpu().numpy()
        for lo in range(0, x.shape[0], 2048):
            y = x[lo:lo + 2048].reshape(-1, x.shape[1], c["dim"] // 32, 32)
            top = np.abs(y).max(3)
            e = np.where(top > 0, np.floor(np.log2(np.where(top > 0, top, 1.0))) - 2, 0).clip(-127, 127)
            a = np.abs(y) / np.exp2(e)[..., None]
            high = np.searchsorted(grid, a).clip(1, 7)
            low = high - 1
            gap = (grid[high] - a) - (a - grid[low])
            code = np.where((gap < 0) | ((gap == 0) & (high % 2 == 0)), high, low)
            code = np.where(a >= 6, 7, code) + 8 * np.signbit(y)
            code = code.reshape(-1, x.shape[1], c["dim"]).astype(np.uint8)
            here = pages[lo:lo + 2048], slice(None), offsets[lo:lo + 2048]
            codes[here] = code[..., 0::2] | code[..., 1::2] << 4
            sfs[here] = (e + 127).astype(np.uint8)
        out += [torch.from_numpy(codes), torch.from_numpy(sfs)]
    return out


def _exact_attn(s):
    c = s["case"]
    G, page = c["group"], c["page"]
    lut = torch.tensor([(-1.0 if i & 8 else 1.0) * MAGNITUDES[i & 7] for i in range(16)], dtype=torch.float64, device=DEV)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    start = s["q_start"].tolist()
    for b, n in enumerate(s["lens"].tolist()):
        new = start[b + 1] - start[b]
        slot = torch.arange(n, device=DEV)
        if c["window"]:
            slot = torch.cat([slot[:c["sink"]], slot[max(c["sink"], n - new - c["window"] + 1):]])
        ids = s["table"][b].long()[slot // page]
        for h in range(c["kv_heads"]):
            kv = []
            for name in ("k", "v"):
                byte = s[name + "_codes"][ids, h, slot % page].long()
                x = torch.empty(len(slot), c["dim"], dtype=torch.float64, device=DEV)
                x[:, 0::2], x[:, 1::2] = lut[byte % 16], lut[byte // 16]
                power = torch.pow(2.0, s[name + "_sf"][ids, h, slot % page].double() - 127)
                kv.append(x * power.repeat_interleave(32, 1))
            heads = slice(h * G, h * G + G)
            rows = 1 + (1 << 27) // (G * max(1, len(slot)))   # new tokens at a time
            for lo in range(0, new, rows):
                at = torch.arange(lo, min(new, lo + rows), device=DEV)
                z = torch.einsum("tgd,nd->tgn", s["q"][start[b] + at, heads].double(), kv[0]) / math.sqrt(c["dim"])
                p = (n - new + at)[:, None, None]
                sees = slot <= p
                if c["window"]:
                    sees &= (slot < c["sink"]) | (slot > p - c["window"])
                z = torch.where(sees, z, -math.inf)
                lse[start[b] + at, heads] = torch.logsumexp(z, 2)
                out[start[b] + at, heads] = torch.einsum("tgn,nd->tgd", torch.softmax(z, 2), kv[1])
    return [out, lse]


def _exact_fork(s):
    page = s["case"]["page"]
    table, lens, parent = (s[k].cpu().numpy() for k in ("table", "lens", "parent"))
    rows = [table[p, :_pages(int(lens[p]), page)] if p >= 0 else table[0, :0] for p in parent]
    out = np.full_like(table, -1)
    for i, r in enumerate(rows):
        out[i, :len(r)] = r
    refs = np.bincount(np.concatenate(rows), minlength=s["refs"].numel()).astype(np.int32)
    return [torch.from_numpy(refs), torch.from_numpy(out),
            torch.tensor([int(lens[p]) if p >= 0 else 0 for p in parent], dtype=torch.int32)]


def _exact_resize(s):
    """Row by row, as the definition says it; the caches' pages are copied one at a time."""
    page = s["case"]["page"]
    old, new = s["lens"].tolist(), s["new_lens"].tolist()
    rows = [r[:_pages(n, page)] for r, n in zip(s["table"].tolist(), old)]
    for i, m in enumerate(new):
        rows[i] = rows[i][:_pages(m, page)]
    count = np.bincount(np.concatenate([np.array(r, dtype=np.int64) for r in rows]), minlength=s["refs"].numel())
    free = iter(np.flatnonzero(count == 0).tolist())
    caches = [x.clone() for x in s["caches"]]
    for i, (n, m) in enumerate(zip(old, new)):
        if m > n:
            if n % page and count[rows[i][-1]] > 1:
                to = next(free)
                for x, y in zip(caches, s["caches"]):
                    x[to] = y[rows[i][-1]]
                rows[i][-1] = to
            rows[i] += [next(free) for _ in range(_pages(m, page) - len(rows[i]))]
    table = torch.full(s["table"].shape, -1, dtype=torch.int32)
    for i, r in enumerate(rows):
        table[i, :len(r)] = torch.tensor(r, dtype=torch.int32)
    refs = np.bincount(np.concatenate([np.array(r, dtype=np.int64) for r in rows]), minlength=len(count))
    return [torch.from_numpy(refs.astype(np.int32)), table, torch.tensor(new, dtype=torch.int32), *caches]


def _exact_compact(s):
    page = s["case"]["page"]
    refs, lens, table = s["refs"].cpu().numpy(), s["lens"].tolist(), s["table"].cpu().numpy()
    live = int((refs > 0).sum())
    holes = [p for p in range(live) if refs[p] <= 0]
    moved = dict(zip([p for p in range(live, len(refs)) if refs[p] > 0], holes))
    out, refs_out = np.full_like(table, -1), np.zeros_like(refs)
    caches = [x.clone() for x in s["caches"]]
    for p in np.flatnonzero(refs > 0).tolist():
        refs_out[moved.get(p, p)] = refs[p]
        if p in moved:
            for x, y in zip(caches, s["caches"]):
                x[moved[p]] = y[p]
    for i, n in enumerate(lens):
        out[i, :_pages(n, page)] = [moved.get(p, p) for p in table[i, :_pages(n, page)].tolist()]
    return [torch.from_numpy(refs_out), torch.from_numpy(out), torch.tensor([live], dtype=torch.int32), *caches]


def exact(case, seed):
    return {"append": _exact_append, "attn": _exact_attn, "fork": _exact_fork, "resize": _exact_resize,
            "compact": _exact_compact}[case["op"]](prepare(case, seed))
