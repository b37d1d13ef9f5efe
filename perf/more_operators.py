"""The operators behind the attention inputs, as cases to measure: a paged key and
value cache in 8 bits with a scale for each page, head and side, the attention
that reads it, and the moves of its pages.

Every case is what a serving step does with one of them:

  append   pages_extend, cache_write: room for each sequence's new tokens, then
           their keys and values in 8 bits
  attend   cache_attention: the new tokens' queries over their sequences' pages
  copy     pages_copy: listed pages of all layers to other pages
  branch   pages_free, pages_fork: losing branches leave, the winners' go on in
           their place (full pages shared, the begun one copied)
  compact  pages_compact: the live pages move together, tables follow

`own` false computes the plain form in elementary torch operations, `own` true
calls the library.
"""
import math
import random

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
FP8 = torch.float8_e4m3fn


def listed():
    return [
        # the decode batch's new tokens, one a sequence: most pages are begun already
        dict(name="append decode batch", op="append", dtype="bf16", B=512, new=1, longest=512, even=False, kv_heads=8, dim=128, page=16, lot=1),
        # the prefill batch's prompts, 8 x 1024 tokens
        dict(name="append prompts", op="append", dtype="bf16", B=8, new=1024, longest=1024, even=True, kv_heads=8, dim=128, page=64, lot=2),
        # one user's next token
        dict(name="attend one token", op="attend", dtype="f16", B=1, new=1, longest=1000, even=True, q_heads=32, kv_heads=8, dim=128, page=16, window=0, lot=3),
        # the decode batch, sequences of all lengths and padding rows
        dict(name="attend decode batch", op="attend", dtype="bf16", B=512, new=1, longest=8192, even=False, q_heads=32, kv_heads=8, dim=128, page=64, window=0, lot=4),
        # chunks of prompts among single tokens, narrow odd heads, a sliding window
        dict(name="attend mixed window", op="attend", dtype="f16", B=37, new=515, longest=5000, even=False, q_heads=21, kv_heads=3, dim=80, page=32, window=1024, lot=5),
        # the prefill batch's last chunk: 8 x 1024 tokens behind 7168 cached ones each
        dict(name="attend prefill", op="attend", dtype="bf16", B=8, new=1024, longest=8192, even=True, q_heads=32, kv_heads=8, dim=128, page=64, window=0, lot=6),
        # one page of all layers, as a sequence is about to write to a shared page
        dict(name="copy one page", op="copy", layers=32, pages=64, n=1, kv_heads=8, dim=128, page=16),
        # a finished prompt's pages into another part of the pool
        dict(name="copy prompt", op="copy", layers=32, pages=512, n=200, kv_heads=8, dim=128, page=16),
        # best of four: one prompt, three more branches
        dict(name="branch best of four", op="branch", layers=32, B=8, sources=1, n=3, longest=1000, kv_heads=8, dim=128, page=16, lot=7),
        # beams of many requests: half of them lose
        dict(name="branch beams", op="branch", layers=8, B=256, sources=64, n=128, longest=1024, kv_heads=8, dim=128, page=16, lot=8),
        # a few sequences have ended in a small pool
        dict(name="compact small pool", op="compact", layers=4, pages=301, B=12, longest=500, live=0.6, kv_heads=4, dim=96, page=16, lot=9),
        # half of a large pool's sequences have ended
        dict(name="compact pool", op="compact", layers=16, pages=1024, B=64, longest=1024, live=0.5, kv_heads=8, dim=128, page=16, lot=10),
    ]


def spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "copy", "branch", "compact"])
    dtype = rng.choice(["f16", "bf16"])
    page, lot = rng.choice([16, 32, 64, 128]), rng.randrange(1 << 30)
    hk, dim = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 80, 96, 128, 192, 256])
    if op in ("append", "attend"):
        new = 1 if rng.random() < 0.5 else spread(rng, 2, 2048)
        B = spread(rng, 1, 512 if new == 1 else 16)
        longest = min(spread(rng, new, 32768), (1 << 30) // (B * hk * dim) + new) if op == "attend" else spread(rng, new, 1024)
        case = dict(op=op, dtype=dtype, B=B, new=new, longest=longest, even=rng.random() < 0.3, kv_heads=hk, dim=dim, page=page, lot=lot)
        if op == "attend":
            case["q_heads"] = hk * min(rng.choice([1, 2, 4, 5, 7, 8, 16]), max(1, 4096 // (hk * dim)))
            case["window"] = spread(rng, 16, 4096) if rng.random() < 0.3 else 0
            if new > 1:  # at most the largest listed case's products
                case["new"] = max(2, min(new, (1 << 38) // (B * longest * case["q_heads"] * dim), (1 << 25) // longest))
        return case
    layers = spread(rng, 1, 32)
    pages = max(8, min(spread(rng, 16, 4096), (1 << 29) // (2 * layers * hk * page * dim)))
    case = dict(op=op, layers=layers, pages=pages, kv_heads=hk, dim=dim, page=page)
    if op == "copy":
        case["n"] = spread(rng, 1, pages // 2)
        return case
    case["lot"] = lot
    case["B"] = spread(rng, 4, 256)
    case["longest"] = spread(rng, 8, 1024)
    if op == "branch":
        case["sources"] = rng.randint(1, case["B"] // 2)
        case["n"] = rng.randint(1, case["B"] - case["sources"])
        case["longest"] = min(case["longest"], max(1, (pages - case["n"]) // case["sources"]) * page)
        case["n"] = min(case["n"], pages - 1)
        case["sources"] = min(case["sources"], pages - case["n"])
        del case["pages"]
    else:
        case["live"] = rng.uniform(0.1, 0.9)
    return case


# ---------------------------------------------------------------- the inputs

def up(n, m):
    return -(-n // m)


def lengths_of(case):
    """Each sequence's tokens, new ones with them, and its new tokens: plain lists, by the case alone."""
    rng, lens, news = random.Random(case["lot"]), [], []
    for i in range(case["B"]):
        if case["even"]:
            n, length = case["new"], case["longest"]
        else:
            n = 1 if case["new"] == 1 or rng.random() < 0.3 else spread(rng, 1, case["new"])
            length = max(n, spread(rng, 1, case["longest"]))
            if i % 16 == 9:  # a row of the batch that holds no sequence
                length, n = 0, 1 if case["new"] == 1 else 0
        lens.append(length)
        news.append(n)
    return lens, news


def branches(case):
    """Lengths of all rows (the sources' first, then empty ones), and the pairs (source, branch)."""
    rng = random.Random(case["lot"])
    lens = [spread(rng, 1, case["longest"]) for _ in range(case["sources"])] + [0] * (case["B"] - case["sources"])
    return lens, [rng.randrange(case["sources"]) for _ in range(case["n"])], rng.sample(range(case["sources"], case["B"]), case["n"])


def pool(case):
    """Sequences until the live share of the pool is theirs; the rest of the rows are empty."""
    rng, lens, left = random.Random(case["lot"]), [], int(case["pages"] * case["live"])
    for _ in range(case["B"]):
        n = min(spread(rng, 1, case["longest"]), left * case["page"])
        left -= up(n, case["page"])
        lens.append(n)
    return lens


def fp8_normal(g, shape, chunk=1 << 26):
    """Normal values of about 100 in e4m3."""
    out = torch.empty(shape, dtype=FP8, device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), chunk):
        part = flat[i:i + chunk]
        part.copy_((torch.randn(part.numel(), generator=g, device="cuda") * 100).clamp_(-448, 448))
    return out


def powers(g, shape):
    """Scales of the sizes that keys and values have."""
    return torch.exp2(torch.randint(-9, -5, shape, generator=g, device="cuda").float())


def lay_out(g, lens, page, P, M, B):
    """Tables with ceil(length / page) pages for each sequence, from a shuffled pool of P pages; the pages' use counts."""
    order = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    tables = torch.full((B, M), -1, dtype=torch.int32, device="cuda")
    refs, at = torch.zeros(P, dtype=torch.int32, device="cuda"), 0
    for b, n in enumerate(lens):
        k = up(n, page)
        tables[b, :k] = order[at:at + k]
        at += k
    refs[order[:at].long()] = 1
    return tables, refs


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, page, hk, dim = case["op"], case["page"], case["kv_heads"], case["dim"]
    s = dict(op=op, page=page)
    if op in ("append", "attend"):
        dtype = TYPES[case["dtype"]]
        lens, news = lengths_of(case)
        B, T, M = case["B"], sum(news), up(max(max(lens), 1), page) + 1
        total = sum(up(n, page) for n in lens)
        P = total + max(4, total // 16)
        s["lens"], s["news"] = lens, news
        s["lengths"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["starts"] = None
        if case["new"] > 1:
            s["starts"] = torch.tensor([sum(news[:b]) for b in range(B + 1)], dtype=torch.int32, device="cuda")
        # a fused projection's rows: q heads, k heads, v heads
        hq = case.get("q_heads", hk)
        rows = torch.randn(T, (hq + 2 * hk) * dim, generator=g, device="cuda")
        rows = (rows * torch.exp(0.3 * torch.randn(rows.shape[1], generator=g, device="cuda"))).to(dtype)
        s["q"], s["k"], s["v"] = rows[:, :hq * dim], rows[:, hq * dim:(hq + hk) * dim], rows[:, (hq + hk) * dim:]
        held = lens if op == "attend" else [n - m for n, m in zip(lens, news)] if case["new"] > 1 else [max(n - 1, 0) for n in lens]
        s["tables"], s["refs"] = lay_out(g, held, page, P, M, B)
        if op == "attend":
            s["y"] = torch.empty(T, hq * dim, dtype=dtype, device="cuda")
            s["window"], s["softmax_scale"] = case["window"], dim ** -0.5
        # the sequences whose first new token goes to a page begun before, and where it goes
        heads = [(b, n - m) for b, (n, m) in enumerate(zip(lens, news)) if n >= m > 0 and (n - m) % page > 0]
        s["heads"] = torch.tensor(heads, dtype=torch.long, device="cuda").view(-1, 2)
        s["cache"] = fp8_normal(g, (P, 2, hk, page, dim))
        s["scale"] = powers(g, (P, 2, hk))
    else:
        L = case["layers"]
        if op == "branch":
            lens, src, dst = branches(case)
            P = sum(up(n, page) for n in lens) + case["n"] + 4
            s["src"], s["dst"] = [torch.tensor(v, dtype=torch.int32, device="cuda") for v in (src, dst)]
            s["begun"] = torch.tensor([i for i, b in enumerate(src) if lens[b] % page], dtype=torch.long, device="cuda")
        else:
            P = case["pages"]
        if op == "compact":
            lens = pool(case)
        if op != "copy":
            B, M = case["B"], up(case["longest"], page) + 1
            s["tables"], s["refs"] = lay_out(g, lens, page, P, M, B)
            s["lengths"], s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda"), lens
        if op == "compact":
            s["out_tables"], s["out_refs"] = torch.empty_like(s["tables"]), torch.empty_like(s["refs"])
            s["n_live"] = torch.empty(1, dtype=torch.int32, device="cuda")
            used = s["refs"] > 0
            s["moves"] = int(used[int(used.sum()):].sum())  # a host that keeps the counts knows it
        if op == "copy":
            order = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
            s["src"], s["dst"] = order[:case["n"]].contiguous(), order[case["n"]:2 * case["n"]].contiguous()
        s["cache"] = fp8_normal(g, (L, P, 2, hk, page, dim))
        s["scale"] = powers(g, (L, P, 2, hk))
    s["work"] = None
    if own:
        from gather_matmul_b200 import ops
        s["work"] = ops.cache_workspace(s["cache"].shape[-5], dim)
    return s


# ---------------------------------------------------------------- one pass

def plain_extend(s):
    tables, lengths, refs = s["tables"], s["lengths"], s["refs"]
    place = torch.arange(tables.shape[1], device="cuda")
    need = (lengths + s["page"] - 1) // s["page"]
    inside = place < need[:, None]
    held = torch.where(inside & (tables >= 0), place + 1, 0).amax(1)
    missing = inside & (place >= held[:, None])
    rank = torch.cumsum(missing.flatten().long(), 0).view_as(missing) - 1
    free = torch.argsort((refs != 0).to(torch.int8), stable=True).to(torch.int32)
    tables.copy_(torch.where(missing, free[rank.clamp(0, refs.numel() - 1)], tables))
    refs.index_add_(0, torch.where(missing, tables, 0).flatten().long(), missing.flatten().to(torch.int32))


def token_places(s):
    """Of each new token: sequence and position."""
    new = torch.tensor(s["news"], device="cuda")
    seq = torch.repeat_interleave(torch.arange(len(s["news"]), device="cuda"), new, output_size=sum(s["news"]))
    first = torch.cumsum(new, 0) - new
    return seq, s["lengths"][seq] - new[seq] + torch.arange(seq.numel(), device="cuda") - first[seq]


def plain_write(s):
    cache, scale, page = s["cache"], s["scale"], s["page"]
    P, _, hk, _, dim = cache.shape
    seq, pos = token_places(s)
    x = torch.stack([s["k"], s["v"]], 1).float().view(-1, 2, hk, dim)
    live = pos >= 0
    pg = torch.where(live, s["tables"][seq, pos.clamp_min(0) // page].long(), P)  # a row without a sequence goes to a page past the last
    most = torch.zeros(P + 1, 2, hk, device="cuda")
    most.index_reduce_(0, pg, x.abs().amax(-1), "amax")
    touched = torch.zeros(P + 1, device="cuda").index_add_(0, pg, torch.ones_like(pg, dtype=torch.float32))[:P] > 0
    # the page's first new place: 0 for a fresh page
    begun = torch.full((P + 1,), page, device="cuda").index_reduce_(0, pg, pos.clamp_min(0) % page, "amin")[:P]
    m, e = torch.frexp(most[:P] / 448)
    e = torch.where(m == 0.5, e - 1, e).clamp(-32, 32)  # least e with most <= 448 * 2 ** e
    e = torch.where(most[:P] == 0, torch.full_like(e, -32), e)
    new = torch.exp2(e.float())
    old = begun > 0
    new = torch.where(old[:, None, None], torch.maximum(scale, new), new)
    ids = (touched & old)
    ratio = torch.where(ids[:, None, None], scale / new, 1.0)
    kept = torch.arange(page, device="cuda")[None] < begun[:, None]
    redo = s["tables"][s["heads"][:, 0], s["heads"][:, 1] // page].long()  # the pages begun before
    again = (cache[redo].float() * ratio[redo][..., None, None]).to(FP8)
    cache[redo] = torch.where(kept[redo][:, None, None, :, None], again, cache[redo])
    scale.copy_(torch.where(touched[:, None, None], new, scale))
    to = torch.where(live, pg, 0)
    q = (x / scale[to][..., None]).clamp(-448, 448).to(FP8)
    at = (pos.clamp_min(0) % page)
    q = torch.where(live[:, None, None, None], q, cache[to, :, :, at])
    cache.index_put_((to[:, None, None], torch.arange(2, device="cuda")[:, None], torch.arange(hk, device="cuda"), at[:, None, None]), q)


def plain_attend(s):
    cache, page, c, w = s["cache"], s["page"], s["softmax_scale"], s["window"]
    hk, dim = cache.shape[2], cache.shape[4]
    group, t = s["q"].shape[1] // (hk * dim), 0
    y = s["y"]
    for b, (length, n) in enumerate(zip(s["lens"], s["news"])):
        if n == 0:
            continue
        first = max(0, length - n - w + 1) // page if w else 0
        pages = s["tables"][b, first:up(length, page)].long()
        kv = (cache[pages].float() * s["scale"][pages][..., None, None]).permute(1, 2, 0, 3, 4).reshape(2, hk, -1, dim)
        q = s["q"][t:t + n].float().view(n, hk, group, dim).permute(1, 2, 0, 3)
        j = first * page + torch.arange(kv.shape[2], device="cuda")
        i = length - n + torch.arange(n, device="cuda")[:, None]
        seen = (j <= i) & (j > i - w) if w else j <= i
        for h in range(hk):
            a = torch.matmul(q[h].reshape(group * n, dim), kv[0, h].t()).view(group, n, -1) * c
            a = a.masked_fill(~seen, -math.inf)
            top = a.amax(-1, keepdim=True) if a.shape[-1] else a.new_full((group, n, 1), -math.inf)
            p = torch.exp(a - torch.where(top == -math.inf, 0.0, top))
            o = torch.matmul(p.view(group * n, -1), kv[1, h]).view(group, n, dim) / p.sum(-1, keepdim=True).clamp_min(1e-30)
            y[t:t + n].view(n, hk, group, dim)[:, h] = o.transpose(0, 1).to(y.dtype)
        t += n
    return y


def plain_copy(cache, scale, src, dst):
    words = cache.view(torch.int64)
    words.index_copy_(1, dst, words.index_select(1, src))
    scale.index_copy_(1, dst, scale.index_select(1, src))


def plain_branch(s):
    tables, lengths, refs, page = s["tables"], s["lengths"], s["refs"], s["page"]
    src, dst = s["src"].long(), s["dst"].long()
    rows = tables[dst]
    refs.index_add_(0, rows.clamp_min(0).flatten().long(), -(rows >= 0).flatten().to(torch.int32))
    place = torch.arange(tables.shape[1], device="cuda")
    n = lengths[src]
    full, begun = n // page, n % page > 0
    free = torch.argsort((refs != 0).to(torch.int8), stable=True).to(torch.int32)
    fresh = free[torch.cumsum(begun.long(), 0) - 1]
    rows = torch.where(place < full[:, None], tables[src], -1)
    refs.index_add_(0, rows.clamp_min(0).flatten().long(), (rows >= 0).flatten().to(torch.int32))
    last = (place == full[:, None]) & begun[:, None]
    tables[dst] = torch.where(last, fresh[:, None], rows)
    lengths[dst] = n
    refs.index_add_(0, torch.where(begun, fresh, 0).long(), begun.to(torch.int32))
    i = s["begun"]
    plain_copy(s["cache"], s["scale"], tables[src[i], full[i].long()].long(), fresh[i].long())


def plain_compact(s):
    refs, tables = s["refs"], s["tables"]
    P = refs.numel()
    live = refs > 0
    n, page = live.sum(), torch.arange(P, device="cuda")
    # holes below n, lowest first; live pages from n on, highest first; both at the front of an order of all pages
    hole, high = ~live & (page < n), live & (page >= n)
    to = torch.argsort((~hole).to(torch.int8), stable=True)
    of = P - 1 - torch.argsort((~high.flip(0)).to(torch.int8), stable=True)
    moved = page < hole.sum()
    names = page.clone()
    names[of] = torch.where(moved, to, names[of])
    s["out_tables"].copy_(torch.where(tables >= 0, names[tables.clamp_min(0).long()].to(torch.int32), tables))
    out = torch.where(page < n, refs, 0)
    out[to] = torch.where(moved, refs[of], out[to])
    s["out_refs"].copy_(out)
    s["n_live"].copy_(n)
    k = s["moves"]
    plain_copy(s["cache"], s["scale"], of[:k], to[:k])


def run(s):
    op = s["op"]
    if own:
        from gather_matmul_b200 import ops
        if op == "append":
            ops.pages_extend(s["tables"], s["lengths"], s["refs"], s["page"], s["work"])
            ops.cache_write(s["k"], s["v"], s["cache"], s["scale"], s["tables"], s["lengths"], s["work"], starts=s["starts"])
        elif op == "attend":
            return ops.cache_attention(s["q"], s["cache"], s["scale"], s["tables"], s["lengths"], s["y"], s["work"],
                                       starts=s["starts"], softmax_scale=s["softmax_scale"], window=s["window"])
        elif op == "copy":
            ops.pages_copy(s["cache"], s["scale"], s["src"], s["dst"], s["work"])
        elif op == "branch":
            ops.pages_free(s["tables"], s["lengths"], s["refs"], s["dst"], s["work"])
            ops.pages_fork(s["tables"], s["lengths"], s["refs"], s["src"], s["dst"], s["cache"], s["scale"], s["work"])
        else:
            ops.pages_compact(s["tables"], s["refs"], s["cache"], s["scale"], s["work"], out_tables=s["out_tables"],
                              out_refs=s["out_refs"], n_live=s["n_live"])
    elif op == "append":
        plain_extend(s)
        plain_write(s)
    elif op == "attend":
        return plain_attend(s)
    elif op == "copy":
        plain_copy(s["cache"], s["scale"], s["src"].long(), s["dst"].long())
    elif op == "branch":
        plain_branch(s)
    else:
        plain_compact(s)
    if op == "append":
        return s["tables"], s["refs"], s["cache"], s["scale"]
    if op == "copy":
        return s["cache"], s["scale"]
    if op == "branch":
        return s["tables"], s["lengths"], s["refs"], s["cache"], s["scale"]
    return s["out_tables"], s["out_refs"], s["n_live"], s["cache"], s["scale"]


def work(case):
    op, page, hk, dim = case["op"], case["page"], case["kv_heads"], case["dim"]
    one = 2 * hk * (page * dim + 4)  # a page of a layer, with its scales
    if op in ("append", "attend"):
        lens, news = lengths_of(case)
        T = sum(news)
    if op == "append":
        return {"bytes": 6 * T * hk * dim + 8 * T, "flops": 4 * T * hk * dim}
    if op == "attend":
        hq, w, tokens, pairs = case["q_heads"], case["window"], 0, 0
        for length, n in zip(lens, news):
            if length == 0 or n == 0:
                continue
            tokens += length - (max(0, length - n - w + 1) if w else 0)
            pairs += sum(min(p + 1, w) if w else p + 1 for p in range(length - n, length))
        return {"bytes": 2 * tokens * hk * dim + 8 * up(tokens, page) * hk + 4 * T * hq * dim, "flops": 4 * pairs * hq * dim}
    if op == "copy":
        return {"bytes": 2 * case["n"] * case["layers"] * one, "flops": 0}
    if op == "branch":
        lens, src, _ = branches(case)
        begun = sum(lens[i] % page > 0 for i in src)
        return {"bytes": 2 * begun * case["layers"] * one + 12 * sum(up(lens[i], page) for i in src), "flops": 0}
    # of a shuffled pool's first n pages, n live ones in all, this share is free
    n = sum(up(v, page) for v in pool(case))
    return {"bytes": 2 * (n * (case["pages"] - n) // case["pages"]) * case["layers"] * one + 8 * case["pages"], "flops": 0}


# ---------------------------------------------------------------- in 64 bits

def exact_e4m3(v):
    """v (64 bits) to the nearest e4m3 value, ties to the even code."""
    grid = torch.tensor([m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1],
                        dtype=torch.float64, device=v.device)
    middle = (grid[1:] + grid[:-1]) / 2
    below, above = torch.bucketize(v.abs(), middle), torch.bucketize(v.abs(), middle, right=True)
    code = torch.where(below != above, below + below % 2, below)
    return torch.copysign(grid[code], v)


def exact_append(case, s):
    """Sequence by sequence and page by page; the free pages are taken lowest first."""
    page, hk, dim = case["page"], case["kv_heads"], case["dim"]
    tables, refs = s["tables"].tolist(), s["refs"].tolist()
    cache, scale = s["cache"].double(), s["scale"].double()
    free, t = iter([p for p, r in enumerate(refs) if r == 0]), 0
    steps = torch.exp2(torch.arange(-32, 33, dtype=torch.float64, device="cuda"))
    for b, (length, n) in enumerate(zip(s["lens"], s["news"])):
        done = max(0, length - n)
        if length:
            for place in range(up(done, page), up(length, page)):
                tables[b][place] = next(free)
        while done < length:
            first, m = done % page, min(page - done % page, length - done)
            x = torch.stack([s["k"][t:t + m], s["v"][t:t + m]]).double().view(2, m, hk, dim).transpose(1, 2)
            fits = x.abs().amax((2, 3))[..., None] <= 448 * steps
            new = torch.where(fits.any(-1), steps[fits.to(torch.int8).argmax(-1)], steps[-1])
            p = tables[b][done // page]
            if first:
                new = torch.maximum(new, scale[p])
                cache[p, :, :, :first] = exact_e4m3(cache[p, :, :, :first] * (scale[p] / new)[..., None, None])
            scale[p] = new
            cache[p, :, :, first:first + m] = exact_e4m3(x / new[..., None, None])
            done, t = done + m, t + m
        if not length:
            t += n
    return None, None, cache, scale


def exact_attend(case, s):
    page, hk, dim, w = case["page"], case["kv_heads"], case["dim"], case["window"]
    group, t = case["q_heads"] // hk, 0
    y = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, (length, n) in enumerate(zip(s["lens"], s["news"])):
        if n and length:
            ids = s["tables"][b, :up(length, page)].long()
            i = torch.arange(length - n, length, device="cuda")[:, None]
            j = torch.arange(length, device="cuda")[None]
            hidden = (j > i) | (j <= i - w) if w else j > i
            for h in range(hk):
                k, v = [(s["cache"][ids, a, h].double() * s["scale"][ids, a, h].double()[:, None, None]).reshape(-1, dim)[:length] for a in (0, 1)]
                for r in range(h * group, (h + 1) * group):
                    q = s["q"][t:t + n, r * dim:(r + 1) * dim].double() / math.sqrt(dim)
                    logits = (q @ k.t()).masked_fill_(hidden, -math.inf)
                    y[t:t + n, r * dim:(r + 1) * dim] = torch.softmax(logits, 1) @ v
        t += n
    return y


def exact(case, seed):
    if case["op"] == "append":
        return exact_append(case, prepare(case, seed))
    if case["op"] == "attend":
        return exact_attend(case, prepare(case, seed))
    return None
