"""The 4-bit key/value cache beside speculative verification: what is measured.

A target model that scores drafted positions attends over a cache of the
verified context and over the drafted positions themselves, verifies, and keeps
the keys and values of the accepted positions.  Two operators (and the reading
back of what the second wrote) do that with a paged cache held in 4 bits:

- ``attend``: attention of the n = k + 1 scored positions of every sequence
  (node 0, the last verified token, and its drafts: a chain, or a tree given by
  its parents) over the sequence's cached context in 4 bits and over the
  positions' own keys and values.
- ``keep``: the accepted rows of the scored positions' keys and values are
  quantised into the cache as they are written behind each sequence's length,
  and a range of every sequence is read back.

Cache layout.  A page holds ``page`` tokens (a power of two, at least 16) of
every key/value head; a block is T = min(page, 64) tokens of one head.
``pages`` is uint8 [pages][heads][page / T][T * (D + 8)], a block being

- T rows of D / 2 bytes, the key codes: the 32-bit word w of a row holds the
  dims 8w..8w+7, dim 8w + 2i in bits 4i..4i+3 and dim 8w + 2i + 1 in bits
  16 + 4i..19 + 4i;
- T pairs (scale, zero) of the model's 16-bit type, the keys' parameters;
- D rows of T / 2 bytes, the value codes: row d, tokens in the same word order;
- T pairs (scale, zero), the values' parameters.

An element stands for zero + scale * code.  A token's row x[0..D) of one head
is written with zero = min x, scale = (max x - min x) / 15 rounded to the
16-bit type, and code = round((x - zero) / scale) to even, within 0..15.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
ORDER = (0, 2, 4, 6, 1, 3, 5, 7)  # the dim (or token) held by nibble i of a word, lowest bits first


# ---- the cases ----------------------------------------------------------------

def listed():
    return [
        # one short conversation, plain decoding of one token: latency counts
        _attend("attend_token", B=1, n=1, hq=32, hkv=8, d=128, page=64, lo=700, hi=700),
        # one sequence with 8 drafted tokens far into a long context (split over the whole device)
        _attend("attend_long", B=1, n=9, hq=32, hkv=8, d=128, page=64, lo=131001, hi=131001),
        # the batched verification step: 64 sequences, 4 drafts each, ragged contexts
        _attend("attend_batch", B=64, n=5, hq=32, hkv=8, d=128, page=64, lo=500, hi=8000),
        # many sequences, 8 drafts each, wide query groups, short ragged contexts down to an empty one
        _attend("attend_wide", B=256, n=9, hq=64, hkv=8, d=128, page=32, lo=0, hi=3001),
        # candidate trees of 8 nodes (binary), a head for every query head, fp16, small heads
        _attend("attend_tree", B=64, n=9, hq=16, hkv=16, d=64, page=16, lo=100, hi=2300, tree="binary", type="fp16"),
        # a large candidate tree
        _attend("attend_tree63", B=16, n=64, hq=32, hkv=4, d=128, page=128, lo=1000, hi=6001, tree="binary"),
        # the largest: 128 sequences with 3 drafts, contexts of about 8,000 tokens
        _attend("attend_large", B=128, n=4, hq=32, hkv=8, d=128, page=64, lo=6200, hi=9800),
        # the cached context alone, with its log-sum-exp, for joining with another part of the context
        _attend("attend_part", B=32, n=1, hq=40, hkv=8, d=128, page=64, lo=0, hi=16000, alone=True),
        # what one sequence keeps after a round of 8 drafts
        _keep("keep_one", B=1, n=9, hkv=8, d=128, page=64, lo=700, hi=700, read=16),
        # the accepted rows of the batched verification step
        _keep("keep_batch", B=64, n=5, hkv=8, d=128, page=64, lo=500, hi=8000, read=5),
        # the accepted paths of candidate trees, fp16
        _keep("keep_tree", B=64, n=9, hkv=16, d=64, page=16, lo=100, hi=2300, read=64, tree="binary", type="fp16"),
        # prompts of up to 8,191 tokens written whole, and read back
        _keep("keep_prompt", B=16, n=8191, hkv=8, d=128, page=64, lo=0, hi=0, read=8191),
    ]


def _attend(name, **c):
    return {"name": name, "op": "attend", "tree": "", "type": "bf16", "alone": False, **c}


def _keep(name, **c):
    return {"name": name, "op": "keep", "tree": "", "type": "bf16", **c}


def draw(rng):
    def log(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))

    d, hkv, page = rng.choice((64, 128, 128)), rng.choice((1, 2, 4, 8, 16)), rng.choice((16, 32, 64, 128))
    tree, kind = rng.choice(("", "", "binary", "star")), rng.choice(("bf16", "bf16", "fp16"))
    if rng.random() < 0.65:
        hq = hkv * rng.choice((1, 2, 3, 4, 5, 7, 8))
        n = log(1, 64) if tree else log(1, 20)
        B = log(1, 256)
        most = min(131072, 8_000_000 * 128 // (B * hkv * d), 120_000_000 // (B * n * hq))
        hi = log(1, max(2, most))
        lo = rng.choice((0, hi // 8, hi // 2, hi))
        alone = not tree and rng.random() < 0.25
        c = _attend("", B=B, n=n, hq=hq, hkv=hkv, d=d, page=page, lo=lo, hi=hi, tree=tree, type=kind, alone=alone)
    else:
        prompt = rng.random() < 0.4
        n = log(20, 8191) if prompt else log(1, 64 if tree else 20)
        B = log(1, 256)
        B = max(1, min(B, 16 * 8191 * 8 * 128 // (n * hkv * d)))
        hi = rng.choice((0, log(1, 4000)))
        read = min(n + rng.choice((0, 11, 64)), 8191)
        c = _keep("", B=B, n=n, hkv=hkv, d=d, page=page, lo=hi // 3, hi=hi, read=read, tree="" if prompt else tree, type=kind)
    c.pop("name")
    return c


def _lens(c):
    """The sequences' cached lengths: ragged over [lo, hi], the first one hi."""
    return [c["lo"] + int((c["hi"] - c["lo"]) * (1.0 - (b * 0.6180339887498949) % 1.0) + 0.5) for b in range(c["B"])]


def _parents(c):
    """Parent of node i + 1, for each of the n - 1 drafted nodes."""
    shape = c["tree"] or "chain"
    return [{"chain": i, "binary": i // 2, "star": 0}[shape] for i in range(c["n"] - 1)]


def _kept(c):
    """For each sequence the list of accepted nodes, or None for a sequence that failed (it keeps nothing)."""
    n, par, got = c["n"], _parents(c), []
    for b in range(c["B"]):
        if n > 64:  # a prompt: rows 0 .. its length - 1, lengths from a quarter of the longest up
            got.append(list(range(1, n - (b * 7919 % max(1, 3 * n // 4)))))
        elif c["B"] > 4 and b % 13 == 5:
            got.append(None)
        elif not c["tree"]:
            got.append(list(range(1, 1 + (n - 1 if b == 0 else (b * 5 + 2) % n))))
        else:
            node, path = (n - 1 if b == 0 else b * 7 % n), []
            while node > 0:
                path.append(node)
                node = par[node - 1]
            got.append(path[::-1])
    return got


def _new_lens(c):
    return [x + (0 if path is None else 1 + len(path)) for x, path in zip(_lens(c), _kept(c))]


# ---- inputs -------------------------------------------------------------------

def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    T, lens = TYPES[c["type"]], _lens(c)
    B, n, hkv, d, page = c["B"], c["n"], c["hkv"], c["d"], c["page"]
    need = [-(-(x + n) // page) for x in lens]
    total = sum(need) + 3
    order = torch.randperm(total, generator=g, device=dev).to(torch.int32).cpu()
    table = torch.full((B, max(need)), -1, dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    s = {
        "case": c, "table": table.to(dev), "lens": torch.tensor(lens, dtype=torch.int32, device=dev),
        "pages": _pages(c, total, T, g, dev),
    }
    # the fused projection's rows: query, key and value heads of a token side by side
    hq = c.get("hq", 0)
    qkv = torch.randn((B, n, hq + 2 * hkv, d), generator=g, device=dev)
    qkv[:, :, :hq] *= 1.5
    qkv[:, :, hq:hq + hkv] += 2.0 * torch.randn((hkv, d), generator=g, device=dev)  # keys keep an offset in each channel
    qkv = qkv.to(T)
    s["q"], s["k"], s["v"] = qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:]
    if c["tree"]:
        s["parents"] = torch.tensor([_parents(c)] * B, dtype=torch.int32, device=dev).reshape(B, n - 1)
    if c["op"] == "keep":
        paths = _kept(c)
        s["n_accepted"] = torch.tensor([-1 if p is None else len(p) for p in paths], dtype=torch.int32, device=dev)
        if c["tree"]:
            rows = [([] if p is None else p) for p in paths]
            s["nodes"] = torch.tensor([r + [-1] * (n - len(r)) for r in rows], dtype=torch.int32, device=dev)
        s["first"] = torch.tensor([max(0, x - c["read"]) for x in _new_lens(c)], dtype=torch.int32, device=dev)
    return s


def _pages(c, total, T, g, dev):
    """Pages as a quantiser leaves them: bell-shaped codes, scales spread over a few octaves, zeros below."""
    d, t = c["d"], min(c["page"], 64)
    blocks = total * c["hkv"] * (c["page"] // t)
    out = torch.empty((blocks, t * (d + 8)), dtype=torch.uint8, device=dev)
    step = max(1, (1 << 28) // (t * d))
    for a in range(0, blocks, step):
        m = min(step, blocks - a)
        for part in range(2):
            x = torch.randn((2, m, t * d // 2), generator=g, device=dev, dtype=torch.float16).mul_(2.7).add_(7.5).round_().clamp_(0, 15).to(torch.uint8)
            o = part * t * (d + 8) // 2
            out[a:a + m, o:o + t * d // 2] = x[0] + 16 * x[1]
            scale = (0.25 * torch.exp(0.4 * torch.randn((m, t, 1), generator=g, device=dev))).to(T)
            zero = (-7.5 * scale.float() + 0.5 * torch.randn((m, t, 1), generator=g, device=dev)).to(T)
            out[a:a + m, o + t * d // 2:o + t * (d + 8) // 2] = torch.cat((scale, zero), 2).reshape(m, t * 2).view(torch.uint8)
    return out.reshape(total, c["hkv"], -1)


# ---- the operators --------------------------------------------------------------

def run(state):
    s, c = state, state["case"]
    if own:
        import draft_token_verification_verify_b200 as sv

        cache = s.get("cache")
        if cache is None:  # the handle a program makes once for its pages
            cache = s["cache"] = sv.KvCache(s["pages"], c["d"], TYPES[c["type"]])
        if c["op"] == "keep":
            lens = sv.cache_append(cache, s["table"], s["lens"], s["k"], s["v"], n_accepted=s["n_accepted"], nodes=s.get("nodes"))
            k, v = sv.cache_read(cache, s["table"], lens, c["read"], first=s["first"])
            return {"lens": lens, "k": k, "v": v}
        if c["alone"]:
            lse = torch.empty((c["B"], c["n"], c["hq"]), dtype=torch.float32, device=s["q"].device)
            return {"out": sv.cache_attend(s["q"], cache, s["table"], s["lens"], out_lse=lse), "lse": lse}
        return {"out": sv.cache_attend(s["q"], cache, s["table"], s["lens"], s["k"], s["v"], parents=s.get("parents"))}
    return _plain_keep(s, c) if c["op"] == "keep" else _plain_attend(s, c)


def _words(x, t, inner):
    """Codes [.., rows, inner] from the packed bytes [.., rows * inner / 2]."""
    w = x.contiguous().view(torch.int32).reshape(*x.shape[:-1], -1, inner // 8)
    shift = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], dtype=torch.int32, device=x.device)
    return ((w[..., None] >> shift) & 15).flatten(-2)


def _read(pages, table, d, page, T):
    """Keys and values [B, tokens, heads, D] in 32 bits of all pages in the table."""
    t = min(page, 64)
    x = pages[table.clamp(min=0).long()].reshape(*table.shape, pages.shape[1], page // t, t * (d + 8))
    half = t * (d + 8) // 2
    got = []
    for part in range(2):
        y = x[..., part * half:(part + 1) * half]
        codes = _words(y[..., :t * d // 2], t, d if part == 0 else t).float()
        codes = codes if part == 0 else codes.transpose(-1, -2)
        p = y[..., t * d // 2:].contiguous().view(T).reshape(*codes.shape[:-1], 2).float()
        z = codes * p[..., :1] + p[..., 1:]  # [B, pages, heads, blocks, t, D]
        got.append(z.permute(0, 1, 3, 4, 2, 5).reshape(table.shape[0], -1, pages.shape[1], d))
    return got


def _plain_attend(s, c):
    q, T, n, d = s["q"], TYPES[c["type"]], c["n"], c["d"]
    B, hq, hkv, dev = c["B"], c["hq"], c["hkv"], s["q"].device
    k, v = _read(s["pages"], s["table"], d, c["page"], T)
    keys = torch.arange(k.shape[1], device=dev)
    seen = (keys[None] < s["lens"][:, None])[:, None].expand(B, n, -1)
    if not c["alone"]:
        if c["tree"]:
            step = torch.eye(n, device=dev).repeat(B, 1, 1)
            step[:, 1:] += torch.nn.functional.one_hot(s["parents"].long(), n)
            own_path = torch.linalg.matrix_power(step, n) > 0
        else:
            own_path = torch.ones((n, n), device=dev).tril().bool().expand(B, n, n)
        seen = torch.cat((seen, own_path), 2)
        k, v = torch.cat((k, s["k"].float()), 1), torch.cat((v, s["v"].float()), 1)
    qg = q.float().reshape(B, n, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(B, hkv, -1, d)
    z = (qg @ k.permute(0, 2, 3, 1)) / math.sqrt(d)
    z = z.reshape(B, hkv, hq // hkv, n, -1).masked_fill(~seen[:, None, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    p = torch.exp(z - top.masked_fill(top == -math.inf, 0.0))
    total = p.sum(-1, keepdim=True)
    v = v.masked_fill(~seen.any(1)[:, :, None, None], 0.0)
    o = (p.reshape(B, hkv, -1, p.shape[-1]) @ v.permute(0, 2, 1, 3)).reshape(B, hkv, hq // hkv, n, d)
    o = (o / total.masked_fill(total == 0, 1.0)).permute(0, 3, 1, 2, 4).reshape(B, n, hq, d).to(T)
    if not c["alone"]:
        return {"out": o}
    lse = (torch.log(total) + top).squeeze(-1).permute(0, 3, 1, 2).reshape(B, n, hq)
    return {"out": o, "lse": lse}


def _stored(x, T):
    """What the quantised rows x [.., D] stand for, in 32 bits."""
    x = x.float()
    zero = x.amin(-1, keepdim=True)
    scale = ((x.amax(-1, keepdim=True) - zero) / 15).to(T).float()
    code = torch.where(scale > 0, (x - zero) / scale, 0.0).round().clamp(0, 15)
    return code * scale + zero


def _plain_keep(s, c):
    B, n, T, dev = c["B"], c["n"], TYPES[c["type"]], s["k"].device
    count = s["n_accepted"] + 1
    lens = s["lens"] + count
    # the rows read back: from the cache as it was, or from the rows that were kept
    at = s["first"].long()[:, None] + torch.arange(c["read"], device=dev)
    new = at - s["lens"].long()[:, None]
    row = new.clamp(0, n - 1)
    if "nodes" in s:
        row = torch.where(row > 0, s["nodes"].long().gather(1, (row - 1).clamp(min=0)), 0).clamp(min=0)
    sel = row[:, :, None, None].expand(-1, -1, c["hkv"], c["d"])
    # the pages that hold the rows read back, as they were
    page, from_page = c["page"], (s["first"] // c["page"]).long()
    pages = from_page[:, None] + torch.arange((c["read"] + page - 2) // page + 1, device=dev)
    held = s["table"].gather(1, pages.clamp(max=s["table"].shape[1] - 1))
    was = _read(s["pages"], held, c["d"], page, T)
    at_page = (at - (from_page * page)[:, None])[:, :, None, None].expand(-1, -1, c["hkv"], c["d"])
    out = []
    for part, x in enumerate((s["k"], s["v"])):
        y = _stored(x, T).gather(1, sel)
        y = torch.where((new >= 0)[:, :, None, None], y, was[part].gather(1, at_page))
        out.append(y.masked_fill((at >= lens[:, None])[:, :, None, None], 0.0).to(T))
    return {"lens": lens, "k": out[0], "v": out[1]}


# ---- what a pass cannot do without ------------------------------------------------

def work(case):
    c = case
    token = c["hkv"] * (c["d"] + 8)  # bytes of one cached token, keys and values
    row = c["hkv"] * c["d"] * 2      # bytes of its keys, or its values, as they come
    if c["op"] == "keep":
        kept = sum(b - a for a, b in zip(_lens(c), _new_lens(c)))
        read = sum(min(x, c["read"]) for x in _new_lens(c))
        return {"bytes": kept * (2 * row + token) + read * token + c["B"] * c["read"] * 2 * row, "flops": 0}
    B, n, lens, q = c["B"], c["n"], _lens(c), c["hq"] * c["d"]
    par, depth = _parents(c), [1]
    for p in par:
        depth.append(depth[p] + 1)
    pairs = sum(n * x for x in lens) + (0 if c["alone"] else B * sum(depth))
    moved = sum(lens) * token + B * n * (2 * q * 2 + (4 * c["hq"] if c["alone"] else 2 * row))
    return {"bytes": moved, "flops": 4 * q * pairs}


# ---- the definition in 64 bits ------------------------------------------------------

def exact(case, seed):
    s, c = prepare(case, seed), case
    T, n, d, hkv = TYPES[c["type"]], c["n"], c["d"], c["hkv"]
    if c["op"] == "keep":
        return _exact_keep(s, c)
    hq, group = c["hq"], c["hq"] // hkv
    par, outs, lses = _parents(c), [], []
    path = torch.zeros((n, n), dtype=torch.bool)
    for i in range(n):
        j = i
        while j >= 0:
            path[i, j] = True
            j = par[j - 1] if j > 0 else -1
    path = path.to(s["q"].device)
    for b, m in enumerate(_lens(c)):
        k, v = _exact_tokens(s, c, b, 0, m)
        mask = torch.ones((n, m), dtype=torch.bool, device=path.device)
        if not c["alone"]:
            k, v = torch.cat((k, s["k"][b].double())), torch.cat((v, s["v"][b].double()))
            mask = torch.cat((mask, path), 1)
        out = torch.zeros((n, hq, d), dtype=torch.float64, device=path.device)
        lse = torch.full((n, hq), -math.inf, dtype=torch.float64, device=path.device)
        if k.shape[0]:
            for h in range(hkv):
                mine = slice(h * group, (h + 1) * group)
                z = torch.einsum("ngd,td->ngt", s["q"][b, :, mine].double(), k[:, h]) * d ** -0.5
                z = torch.where(mask[:, None], z, -math.inf)
                out[:, mine] = torch.einsum("ngt,td->ngd", torch.softmax(z, -1), v[:, h])
                lse[:, mine] = torch.logsumexp(z, -1)
        outs.append(out)
        lses.append(lse)
    got = {"out": torch.stack(outs)}
    if c["alone"]:
        got["lse"] = torch.stack(lses)
    return got


def _exact_tokens(s, c, b, first, end):
    """Keys and values [end - first, heads, D] of sequence b's cached tokens, in 64 bits."""
    d, page, T = c["d"], c["page"], TYPES[c["type"]]
    t = min(page, 64)
    if end <= first:
        return [torch.zeros((0, c["hkv"], d), dtype=torch.float64, device=s["pages"].device)] * 2
    ids = s["table"][b, first // page:(end - 1) // page + 1].long()
    x = s["pages"][ids].reshape(len(ids), c["hkv"], page // t, -1)
    cut, kb = t * (d + 8) // 2, t * d // 2
    got = []
    for raw, rows, cols in ((x[..., :cut], t, d), (x[..., cut:], d, t)):
        pairs = torch.stack((raw[..., :kb] & 15, raw[..., :kb] >> 4), -1)      # the two codes of a byte
        pairs = pairs.reshape(*x.shape[:3], rows, cols // 8, 8)
        codes = torch.empty_like(pairs)
        codes[..., list(ORDER)] = pairs
        codes = codes.reshape(*x.shape[:3], rows, cols)
        codes = codes if cols == d else codes.movedim(-1, -2)
        params = raw[..., kb:].contiguous().view(T).reshape(*x.shape[:3], t, 2).double()
        val = params[..., 1, None] + params[..., 0, None] * codes.double()
        val = val.movedim(1, 3).reshape(len(ids) * page, c["hkv"], d)
        got.append(val[first - first // page * page:][:end - first])
    return got


def _exact_keep(s, c):
    T = TYPES[c["type"]]
    got = {"lens": None, "k": [], "v": []}
    for b, (old, path) in enumerate(zip(_lens(c), _kept(c))):
        rows = [] if path is None else [0] + path
        end = old + len(rows)
        first = max(0, end - c["read"])
        was = _exact_tokens(s, c, b, min(first, old), old)
        for name, x, w in (("k", s["k"], was[0]), ("v", s["v"], was[1])):
            x = x[b, rows].double()
            parts = [w]
            if len(rows):
                lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
                step = ((hi - lo) / 15).to(T).double()
                parts.append(lo + step * torch.clamp(torch.round((x - lo) / torch.where(step > 0, step, 1.0)), 0, 15))
            y = torch.cat(parts)[max(0, first - old):] if first > old else torch.cat(parts)
            pad = torch.zeros((c["read"] - y.shape[0], *y.shape[1:]), dtype=torch.float64, device=y.device)
            got[name].append(torch.cat((y, pad)))
    return {"lens": None, "k": torch.stack(got["k"]), "v": torch.stack(got["v"])}
