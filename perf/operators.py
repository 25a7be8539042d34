"""Cases of the paged key-value cache operators: attention of new tokens over the cache (the whole
prefix, or the tokens an indexer picked), appending keys and values, and the upkeep of the pages
(resize, fork, compact).

A cache is a pool of pages [num_pages, page_size, Hkv, d]; sequence n keeps tokens
i * page_size .. (i + 1) * page_size - 1 in page page_table[n, i] (-1: no page), and refs[p] counts
the table entries that name page p.

`own` false: run() computes each operator from elementary torch operations in 32 bits.  `own` true:
run() calls the library's entry points.
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # a serving batch of 32 sequences of up to 32K tokens, one new token each
        dict(name="decode_32k", op="attention", nseq=32, T=1, Hq=32, Hkv=8, d=128, L=32768,
             spread=16384, page=64, topk=0, dtype="bf16", lse=False),
        # one short chat turn on an idle server: latency is all
        dict(name="decode_one_short", op="attention", nseq=1, T=1, Hq=16, Hkv=2, d=128, L=777,
             spread=0, page=16, topk=0, dtype="bf16", lse=False),
        # four drafted tokens per sequence, small heads, an odd group and pages of 48 tokens; the
        # log-sum-exp is kept to join the result with another part of the context
        dict(name="draft4_fp16_d64", op="attention", nseq=9, T=4, Hq=24, Hkv=4, d=64, L=8191,
             spread=5003, page=48, topk=0, dtype="fp16", lse=True),
        # 16 sequences of 128K tokens that read the 2048 tokens their indexer picked
        dict(name="selected_128k", op="attention", nseq=16, T=1, Hq=32, Hkv=4, d=128, L=131072,
             spread=0, page=64, topk=2048, dtype="bf16", lse=False),
        # the keys and values of one decode step of 32 sequences
        dict(name="append_step", op="append", nseq=32, T=1, Hkv=8, d=128, L=1024, page=64,
             dtype="bf16"),
        # a chunk of 8191 prompt tokens for each of four sequences, the shorter ones padded
        dict(name="append_prompt", op="append", nseq=4, T=8191, Hkv=8, d=128, L=12000, page=64,
             dtype="bf16"),
        # room for a 16-token draft in each of 32 sequences; some give back what was rejected
        dict(name="resize_draft", op="resize", nseq=32, L=32768, grow=16, shared=0, page=64,
             spare=1024, pools=0, Hkv=8, d=128, dtype="bf16"),
        # 64 beams in groups of four that share their history: the partly filled last pages are
        # copied in the pools of four layers before the next token is written
        dict(name="resize_beams", op="resize", nseq=64, L=2000, grow=1, shared=4, page=64,
             spare=512, pools=8, Hkv=8, d=128, dtype="bf16"),
        # a beam-search step: 32 rows take the tables of their parents
        dict(name="fork_beams", op="fork", nseq=32, L=8192, page=64),
        # a cache of 1024 rows of up to 128K tokens: half the rows change, some are freed
        dict(name="fork_batch", op="fork", nseq=1024, L=131072, page=64),
        # a small pool, half of it free
        dict(name="compact_small", op="compact", nseq=16, L=1024, page=16, pools=2, Hkv=1, d=128,
             dtype="fp16"),
        # eight pools of 128 KB pages, half of them free: 256 pages move in each
        dict(name="compact_pools", op="compact", nseq=32, L=1024, page=64, pools=8, Hkv=8, d=128,
             dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "append", "resize", "fork", "compact"])
    page = rng.choice([1, 8, 16, 16, 32, 48, 64, 64, 100, 128, 256])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "attention":
        d, Hkv = rng.choice([64, 128, 128]), rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 3, 4, 6, 8, 16, 16, 32])
        topk = rng.choice([0, 0, _log(rng, 1, 4096)])
        T = rng.choice([1, 1, 1, 2, 3, 4, 7, 16])
        nseq = _log(rng, 1, 64)
        # no more cache, and no more gathered tokens, than the largest listed case holds
        top = min(131072, (32 * 32768 * 8 * 128) // (nseq * Hkv * d))
        if topk:
            topk = min(topk, max(1, (32 * 16384 * 8 * 128) // (nseq * T * Hkv * d)))
        else:
            top = min(top, max(2, (32 * 16384 * 32 * 128) // (nseq * T * Hq * d)))
        L = _log(rng, 1, max(2, top))
        return dict(op=op, nseq=nseq, T=min(T, L), Hq=Hq, Hkv=Hkv, d=d, L=L,
                    spread=rng.choice([0, L // 2, L - 1]), page=page, topk=topk, dtype=dtype,
                    lse=rng.random() < 0.5)
    if op == "append":
        nseq, Hkv, d = _log(rng, 1, 256), rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
        T = _log(rng, 1, max(2, (4 * 8191) // nseq))
        return dict(op=op, nseq=nseq, T=T, Hkv=Hkv, d=d, L=T + _log(rng, 1, 2000), page=page,
                    dtype=dtype)
    page = max(page, 8)
    if op == "fork":
        return dict(op=op, nseq=_log(rng, 1, 1024), L=_log(rng, 1, 32768), page=page)
    if op == "resize":
        shared = rng.choice([0, 0, 2, 4, 5])
        nseq, L = _log(rng, 1, 64), _log(rng, 1, 4096)
        return dict(op=op, nseq=nseq, L=L, grow=_log(rng, 1, 256), shared=shared, page=page,
                    spare=nseq * (1 + 256 // page) + _log(rng, 1, 1000),
                    pools=rng.choice([0, 1, 2, 4]), Hkv=rng.choice([1, 2, 4]), d=128, dtype=dtype)
    return dict(op=op, nseq=_log(rng, 1, 48), L=_log(rng, 1, 1024), page=page,
                pools=rng.choice([0, 1, 2, 4]), Hkv=rng.choice([1, 2, 4]), d=128, dtype=dtype)


def _ceil(a, b):
    return -(-a // b)


def _lengths(c):
    """Tokens of each sequence: the longest first, the others spread below it; a list that the case
    alone fixes, so that its work is known without the inputs."""
    s = c.get("spread", 0)
    return [c["L"] - (n * 7919) % (s + 1) for n in range(c["nseq"])]


def _append_spans(c):
    """(first position, tokens) that each sequence appends; the last ones are padded."""
    spans = []
    for n in range(c["nseq"]):
        cnt = c["T"] - (n * 1009) % max(1, c["T"] // 3)
        spans.append(((n * 577) % (c["L"] - c["T"] + 1), cnt))
    return spans


def _resize_lengths(c):
    """(old, new) lengths: every seventh sequence gives tokens back, one in eleven ends."""
    out = []
    for n in range(c["nseq"]):
        old = max(1, c["L"] - (n // max(1, c["shared"])) * 37 % max(1, c["L"] // 2))
        new = old + c["grow"]
        if n % 7 == 6:
            new = max(0, old - c["grow"])
        if n % 11 == 10:
            new = 0
        out.append((old, new))
    return out


# ------------------------------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, shape, dtype, std=1.0):
    x = torch.empty(shape, dtype=dtype, device=DEV)
    x.normal_(0.0, std, generator=g)
    return x


def _table(g, counts, width, num_pages):
    """Rows of `counts` pages each from a random order of the pool, -1 behind them."""
    counts = torch.tensor(counts, device=DEV)
    col = torch.arange(width, device=DEV)
    held = col[None, :] < counts[:, None]
    at = torch.cumsum(counts, 0) - counts
    perm = torch.randperm(num_pages, generator=g, device=DEV)
    t = perm[(at[:, None] + col[None, :]).clamp(max=num_pages - 1)]
    return torch.where(held, t, torch.full_like(t, -1)).int()


def _count(table, num_pages):
    t = table[table >= 0].long()
    return torch.bincount(t, minlength=num_pages).int()


def prepare(case, seed):
    g = _gen(seed)
    op, c = case["op"], case
    s = dict(case=c)
    ps = c["page"]
    if op in ("attention", "append"):
        dt = TYPES[c["dtype"]]
        nseq, T, Hkv, d = c["nseq"], c["T"], c["Hkv"], c["d"]
        lens = _lengths(c)
        mp = _ceil(c["L"], ps)
        pages = [_ceil(x, ps) for x in lens] if op == "attention" else [mp] * nseq
        num_pages = sum(pages) + 3
        s["table"] = _table(g, pages, mp, num_pages)
        s["k"] = _normal(g, (num_pages, ps, Hkv, d), dt)
        s["v"] = _normal(g, (num_pages, ps, Hkv, d), dt)
        if op == "append":
            t = torch.arange(T, device=DEV)
            first, cnt = (torch.tensor(x, device=DEV) for x in zip(*_append_spans(c)))
            pos = first[:, None] + t[None, :]
            s["pos"] = torch.where(t[None, :] < cnt[:, None], pos, -1).int()
            s["kn"] = _normal(g, (nseq, T, Hkv, d), dt)
            s["vn"] = _normal(g, (nseq, T, Hkv, d), dt)
            return s
        # the last T positions; rows of a draft that reach before the sequence's start are padding
        last = torch.tensor(lens, device=DEV) - 1
        s["pos"] = (last[:, None] - (T - 1) + torch.arange(T, device=DEV)).clamp(min=-1).int()
        # logits of standard deviation 2, and one token per sequence that stands far out
        s["q"] = _normal(g, (nseq, T, c["Hq"], d), dt, 2.0)
        at = (torch.rand(nseq, generator=g, device=DEV) * (last + 1)).long()
        page = s["table"].long().gather(1, (at // ps)[:, None])[:, 0]
        s["k"][page, at % ps, 0] = s["q"][:, T - 1, 0] / 4
        if c["topk"]:
            # distinct tokens of each query's prefix in random order, -1 behind the last one
            width = max(c["topk"], 1)
            score = torch.rand((nseq, T, c["L"]), generator=g, device=DEV)
            col = torch.arange(c["L"], device=DEV)
            score = torch.where(col > s["pos"][..., None], -1.0, score)
            val, idx = score.topk(min(width, c["L"]), dim=-1)
            idx = torch.where(val < 0, -1, idx)
            pad = torch.full((nseq, T, width - idx.shape[-1]), -1, device=DEV)
            s["idx"] = torch.cat([idx, pad], -1).int().contiguous()
        return s
    nseq, mp = c["nseq"], _ceil(c["L"] + c.get("grow", 0), ps)
    if op == "fork":
        counts = [_ceil(max(1, c["L"] - (n * 7919) % max(1, c["L"] // 2)), ps) for n in range(nseq)]
        num_pages = sum(counts) + 64
        s["table"] = _table(g, counts, mp, num_pages)
        s["refs"] = _count(s["table"], num_pages)
        # half the rows stay, the others follow a row of their group of eight, one in 16 ends
        n = torch.arange(nseq, device=DEV)
        pick = (n // 8) * 8 + torch.randint(0, 8, (nseq,), generator=g, device=DEV)
        parent = torch.where(n % 2 == 0, n, pick.clamp(max=nseq - 1))
        s["parent"] = torch.where(n % 16 == 15, -1, parent).int()
        return s
    dt = TYPES[c["dtype"]]
    if op == "resize":
        ln = _resize_lengths(c)
        counts = [_ceil(o, ps) for o, _ in ln]
        num_pages = sum(counts) + c["spare"]
        t = _table(g, counts, mp, num_pages)
        if c["shared"]:   # each group of rows follows its first row
            n = torch.arange(nseq, device=DEV)
            t = t[n // c["shared"] * c["shared"]].contiguous()
        s["table"] = t
        s["old"] = torch.tensor([o for o, _ in ln], device=DEV, dtype=torch.int32)
        s["new"] = torch.tensor([x for _, x in ln], device=DEV, dtype=torch.int32)
    else:
        counts = [_ceil(max(1, c["L"] - n * 37 % max(1, c["L"] // 2)), ps) for n in range(nseq)]
        num_pages = 2 * sum(counts)
        s["table"] = _table(g, counts, mp, num_pages)
    s["refs"] = _count(s["table"], num_pages)
    s["num_pages"] = num_pages
    s["pools"] = _normal(g, (c["pools"], num_pages, ps, c["Hkv"], c["d"]), dt)
    s["views"] = list(s["pools"].unbind(0))
    return s


# ------------------------------------------------------------------------------------- plain forms

def _plain_attention(s):
    c, ps = s["case"], s["case"]["page"]
    nseq, T, Hq, Hkv, d = c["nseq"], c["T"], c["Hq"], c["Hkv"], c["d"]
    G = Hq // Hkv
    table, pos = s["table"].long().clamp(min=0), s["pos"].long()
    q = s["q"].float() / math.sqrt(d)
    if c["topk"]:
        idx = s["idx"].long()
        tok = idx.clamp(min=0)
        page = table.gather(1, (tok // ps).view(nseq, -1)).view(tok.shape)
        k = s["k"][page, tok % ps].float().permute(0, 1, 3, 2, 4)      # [nseq, T, Hkv, topk, d]
        v = s["v"][page, tok % ps].float().permute(0, 1, 3, 2, 4)
        ok = ((idx >= 0) & (idx <= pos[..., None]))[:, :, None, None, :]
        q = q.view(nseq, T, Hkv, G, d)
    else:
        k = s["k"][table].view(nseq, -1, Hkv, d).float().permute(0, 2, 1, 3)   # [nseq, Hkv, S, d]
        v = s["v"][table].view(nseq, -1, Hkv, d).float().permute(0, 2, 1, 3)
        col = torch.arange(k.shape[2], device=DEV)
        ok = (col <= pos[..., None])[:, None, :, None, :].expand(nseq, Hkv, T, G, -1)
        ok = ok.reshape(nseq, Hkv, T * G, -1)
        q = q.view(nseq, T, Hkv, G, d).transpose(1, 2).reshape(nseq, Hkv, T * G, d)
    z = (q @ k.transpose(-1, -2)).masked_fill(~ok, -math.inf)
    top = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = torch.where(total > 0, (p @ v) / total, 0.0)
    lse = (top + torch.log(total))[..., 0]
    if not c["topk"]:
        o = o.view(nseq, Hkv, T, G, d).transpose(1, 2)
        lse = lse.view(nseq, Hkv, T, G).transpose(1, 2)
    o = o.reshape(nseq, T, Hq, d).to(s["q"].dtype)
    return (o, lse.reshape(nseq, T, Hq)) if c["lse"] else o


def _plain_append(s):
    ps = s["case"]["page"]
    n, t = (s["pos"] >= 0).nonzero(as_tuple=True)
    p = s["pos"][n, t].long()
    page = s["table"][n, p // ps].long()
    s["k"][page, p % ps] = s["kn"][n, t]
    s["v"][page, p % ps] = s["vn"][n, t]
    return s["k"], s["v"]


def _plain_resize(s):
    ps, table, refs = s["case"]["page"], s["table"].long(), s["refs"].long()
    old, new = s["old"].long(), s["new"].long()
    n, col = torch.arange(table.shape[0], device=DEV), torch.arange(table.shape[1], device=DEV)
    oldp, newp = (old + ps - 1) // ps, (new + ps - 1) // ps
    # a partly filled last page that others hold too is copied; where all its holders grow in this
    # call, the last of them keeps it
    tail = (new > old) & (old % ps != 0)
    tcol = (old // ps).clamp(max=table.shape[1] - 1)
    tp = table.gather(1, tcol[:, None])[:, 0].clamp(min=0)
    cnt = torch.zeros_like(refs).index_add(0, tp, tail.long())
    last = torch.full_like(refs, -1).scatter_reduce(0, tp, torch.where(tail, n, -1), "amax")
    cow = tail & (refs[tp] > 1) & ~((cnt[tp] >= refs[tp]) & (last[tp] == n))
    here = cow[:, None] & (col == tcol[:, None])
    need = ((col >= oldp[:, None]) & (col < newp[:, None])) | here
    free = torch.sort((refs != 0).int(), stable=True).indices
    rank = (torch.cumsum(need.flatten().long(), 0) - 1).view(need.shape)
    enough = need.sum() <= (refs == 0).sum()
    fresh = free[rank.clamp(0, free.numel() - 1)]
    gone = ((col >= newp[:, None]) & (col < oldp[:, None])) | here
    held = torch.where(col < torch.minimum(oldp, newp)[:, None], table, -1)
    out = torch.where(need, fresh, held)
    r = refs.index_add(0, table[gone], torch.full_like(table[gone], -1))
    r = r.index_add(0, fresh[need], torch.ones_like(fresh[need]))
    row = (cow & enough).nonzero()[:, 0]
    s["pools"][:, out[row, tcol[row]]] = s["pools"][:, tp[row]]
    return torch.where(enough, out, table).int(), torch.where(enough, r, refs).int(), s["pools"]


def _plain_fork(s):
    table, refs, parent = s["table"], s["refs"], s["parent"].long()
    out = torch.where(parent[:, None] >= 0, table[parent.clamp(min=0)], -1)
    return out, refs + _count(out, refs.numel()) - _count(table, refs.numel())


def _plain_compact(s):
    table, refs = s["table"].long(), s["refs"].long()
    at = torch.arange(refs.numel(), device=DEV)
    live = refs > 0
    n = live.sum()
    move = live & (at >= n)
    hole = torch.sort(live.int(), stable=True).indices          # the free pages, lowest first
    src = move.nonzero()[:, 0]                                  # the pages that move, lowest first
    dst = hole[: src.numel()]
    to = at.scatter(0, src, dst)
    r = torch.zeros_like(refs).index_add(0, to[live], refs[live])
    s["pools"][:, dst] = s["pools"][:, src]
    t = torch.where(table >= 0, to[table.clamp(min=0)], -1)
    return t.int(), r.int(), n.int().view(1), s["pools"]


PLAIN = dict(attention=_plain_attention, append=_plain_append, resize=_plain_resize,
             fork=_plain_fork, compact=_plain_compact)


def run(s):
    op = s["case"]["op"]
    if not own:
        return PLAIN[op](s)
    import long_context_block_b200 as M
    if op == "attention":
        return M.misa_paged_attention(s["q"], s["k"], s["v"], s["table"], s["pos"],
                                      idx=s.get("idx"), return_lse=s["case"]["lse"])
    if op == "append":
        return M.misa_paged_append(s["kn"], s["vn"], s["pos"], s["table"], s["k"], s["v"])
    if op == "resize":
        return *M.misa_pages_resize(s["table"], s["refs"], s["old"], s["new"], s["case"]["page"],
                                    s["views"]), s["pools"]
    if op == "fork":
        return M.misa_pages_fork(s["table"], s["refs"], s["parent"])
    return *M.misa_pages_compact(s["table"], s["refs"], s["views"]), s["pools"]


# -------------------------------------------------------------------------------------------- work

def work(case):
    c, op, ps = case, case["op"], case["page"]
    if op == "attention":
        nseq, T, Hq, Hkv, d = c["nseq"], c["T"], c["Hq"], c["Hkv"], c["d"]
        rows = [[max(0, x - (T - 1) + t) for t in range(T)] for x in _lengths(c)]   # prefixes
        if c["topk"]:
            pairs = sum(min(c["topk"], p) for r in rows for p in r)
            tokens = pairs
            small = 4 * nseq * T * c["topk"]
        else:
            pairs, tokens = sum(p for r in rows for p in r), sum(max(r) for r in rows)
            small = 4 * sum(_ceil(max(r), ps) for r in rows)
        small += 4 * nseq * T + (4 * nseq * T * Hq if c["lse"] else 0)
        return dict(bytes=tokens * Hkv * d * 4 + nseq * T * Hq * d * 4 + small,
                    flops=4 * pairs * Hq * d)
    if op == "append":
        tokens = sum(n for _, n in _append_spans(c))
        # a key and a value of each head, two bytes an element, read and written
        return dict(bytes=tokens * c["Hkv"] * c["d"] * 8 + 4 * c["nseq"] * c["T"], flops=0)
    mp = _ceil(c["L"] + c.get("grow", 0), ps)
    if op == "fork":
        pages = sum(_ceil(max(1, c["L"] - (n * 7919) % max(1, c["L"] // 2)), ps)
                    for n in range(c["nseq"])) + 64
        return dict(bytes=8 * c["nseq"] * mp + 8 * pages + 4 * c["nseq"], flops=0)
    page_bytes = ps * c["Hkv"] * c["d"] * 2 * c["pools"]
    if op == "resize":
        ln = _resize_lengths(c)
        pages, moved = sum(_ceil(o, ps) for o, _ in ln) + c["spare"], 0
        if c["shared"]:
            for g in range(0, c["nseq"], c["shared"]):
                grp = ln[g:g + c["shared"]]
                tails = sum(1 for o, x in grp if x > o and o % ps)
                moved += tails - (1 if tails == len(grp) else 0) if len(grp) > 1 else 0
        return dict(bytes=8 * c["nseq"] * mp + 8 * pages + 8 * c["nseq"] + 2 * moved * page_bytes,
                    flops=0)
    held = sum(_ceil(max(1, c["L"] - n * 37 % max(1, c["L"] // 2)), ps) for n in range(c["nseq"]))
    # half the pool is held, at random: half of the held pages lie in its upper half
    return dict(bytes=8 * c["nseq"] * mp + 16 * held + 2 * (held // 2) * page_bytes, flops=0)


# ------------------------------------------------------------------------------------------- exact

def _exact_attention(s):
    c, ps = s["case"], s["case"]["page"]
    nseq, T, Hq, Hkv, d = c["nseq"], c["T"], c["Hq"], c["Hkv"], c["d"]
    G = Hq // Hkv
    out = torch.zeros((nseq, T, Hq, d), dtype=torch.float64, device=DEV)
    lse = torch.full((nseq, T, Hq), -math.inf, dtype=torch.float64, device=DEV)
    kf, vf = s["k"].view(-1, Hkv, d), s["v"].view(-1, Hkv, d)
    pos = s["pos"].tolist()
    for n in range(nseq):
        for t in range(T):
            if pos[n][t] < 0:
                continue
            tok = torch.arange(pos[n][t] + 1, device=DEV)
            if c["topk"]:
                tok = s["idx"][n, t].long()
                tok = tok[tok >= 0]
            slot = s["table"][n].long()[tok // ps] * ps + tok % ps
            k, v = kf[slot].double(), vf[slot].double()
            z = torch.einsum("hgd,shd->hgs", s["q"][n, t].double().view(Hkv, G, d), k) / d ** 0.5
            lse[n, t] = torch.logsumexp(z, -1).flatten()
            out[n, t] = torch.einsum("hgs,shd->hgd", torch.softmax(z, -1), v).reshape(Hq, d)
    return (out, lse) if c["lse"] else out


def _exact_append(s):
    ps = s["case"]["page"]
    k, v = s["k"].clone(), s["v"].clone()
    table = s["table"].tolist()
    for n, (first, cnt) in enumerate(_append_spans(s["case"])):
        t = 0
        while t < cnt:
            p = first + t
            m = min(cnt - t, ps - p % ps)
            page, o = table[n][p // ps], p % ps
            k[page, o:o + m], v[page, o:o + m] = s["kn"][n, t:t + m], s["vn"][n, t:t + m]
            t += m
    return k.double(), v.double()


def _exact_resize(s):
    """The sequences one after the other, on lists: which page is copied where."""
    ps, table, refs = s["case"]["page"], s["table"].tolist(), s["refs"].tolist()
    ln = _resize_lengths(s["case"])
    free = iter([p for p, r in enumerate(refs) if r == 0])
    left, copies = list(refs), []
    for n, (o, x) in enumerate(ln):
        if x <= o:
            continue
        if o % ps:
            p = table[n][o // ps]
            if left[p] > 1:
                left[p] -= 1
                copies.append((p, next(free)))
        for _ in range(_ceil(o, ps), _ceil(x, ps)):
            next(free)
    pools = s["pools"].clone()
    for a, b in copies:
        pools[:, b] = pools[:, a]
    return None, None, pools.double()


def _exact_compact(s):
    refs = s["refs"].tolist()
    live = [p for p, r in enumerate(refs) if r > 0]
    holes = [p for p in range(len(live)) if refs[p] == 0]
    pools = s["pools"].clone()
    for a, b in zip([p for p in live if p >= len(live)], holes):
        pools[:, b] = pools[:, a]
    return None, None, None, pools.double()


def exact(case, seed):
    if case["op"] == "fork":
        return None
    return dict(attention=_exact_attention, append=_exact_append, resize=_exact_resize,
                compact=_exact_compact)[case["op"]](prepare(case, seed))
