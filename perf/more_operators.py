"""Rotary positions, attention over a paged latent cache, and a cache's pages: the cases that are measured, and the
operators in plain form.

* rope: queries or keys rotated by their positions, and gradients rotated back;
* append: a token's latent vector and its rotated key part into the pages of a latent cache, its query parts rotated;
* attend: causal attention of new tokens over cached latents, which are the keys and (without the rotated part) the values
  of all query heads;
* pages: sequences that share pages are forked and grow, shared last pages copied; a pool is compacted.

Sequences are ragged: sequence b has rows q_start[b] .. q_start[b + 1] of the call, kv_len[b] cached tokens (the new ones
included) and its pages in page_table[b]. Lengths follow from the case alone, values and the order of pages from the seed.
"""

import math

import torch

own = False

ROPE = 64          # width of a latent cache's rotated part


# ---------------------------------------------------------------- cases

def _rope_case(name, B, H, N, d, rope_dim, interleaved, rows, backward, far, factor):
    return dict(name=name, op="rope", B=B, H=H, N=N, d=d, rope_dim=rope_dim, interleaved=interleaved, rows=rows,
                backward=backward, far=far, factor=factor)


def _latent_case(name, op, B, heads, rank, page, len_min, len_max, new_min, new_max, interleaved=False):
    return dict(name=name, op=op, B=B, heads=heads, rank=rank, page=page, len_min=len_min, len_max=len_max,
                new_min=new_min, new_max=new_max, interleaved=interleaved)


def _pages_case(name, what, cache, B, children, kv_heads, width, page, len_min, len_max, grow, slack):
    return dict(name=name, op="pages", what=what, cache=cache, B=B, children=children, kv_heads=kv_heads, width=width,
                page=page, len_min=len_min, len_max=len_max, grow=grow, slack=slack)


def listed():
    return [
        # the queries of a training step, [B, H, N, d]
        _rope_case("rotate queries", 2, 32, 4096, 128, 128, False, False, False, 0, 1.0),
        # gradients of a few rows' query parts (64 of 192 columns), neighbouring pairs, positions of a stretched context
        _rope_case("rotate gradients", 1, 20, 333, 64, 64, True, True, True, 120000, 8.0),
        # the step of a serving batch: one token for each of 32 sequences
        _latent_case("append tokens", "append", 32, 24, 512, 64, 200, 4000, 1, 1),
        # whole prompts into fresh pages
        _latent_case("append prompts", "append", 3, 64, 512, 64, 3500, 4096, 4096, 4096, interleaved=True),
        # one user, one token: latency counts
        _latent_case("attend one token", "attend", 1, 16, 512, 64, 1000, 1000, 1, 1),
        # a full serving batch of very different lengths, many heads
        _latent_case("attend token batch", "attend", 64, 128, 512, 64, 500, 8000, 1, 1),
        # few users with long contexts
        _latent_case("attend long context", "attend", 3, 32, 512, 128, 100003, 131071, 1, 1),
        # up to five drafted tokens of each sequence at once, a smaller latent
        _latent_case("attend drafts", "attend", 32, 40, 256, 32, 1000, 4000, 1, 5),
        # a piece of a prompt behind what is cached
        _latent_case("attend prompt piece", "attend", 2, 16, 512, 64, 7000, 8192, 1024, 1024),
        # three more samples of each of 6 prompts, one token further: last pages are copied
        _pages_case("fork a few", "fork", "latent", 6, 3, 1, 576, 64, 300, 4000, 1, 0.2),
        # the same for a large batch on the 8-bit cache, and room for a piece of text
        _pages_case("fork a batch", "fork", "fp8", 192, 3, 8, 128, 64, 500, 2000, 100, 0.1),
        # a pool with holes is moved together
        _pages_case("compact a pool", "compact", "latent", 96, 0, 1, 576, 64, 1000, 6000, 0, 0.6),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "attend", "pages"])
    while True:
        if op == "rope":
            d = rng.choice([64, 128])
            rows = rng.random() < 0.5
            case = _rope_case("", 1 if rows else _log_int(rng, 1, 6), _log_int(rng, 1, 64), _log_int(rng, 1, 8192), d,
                              rng.choice([16, d // 2, d, d]), rng.random() < 0.5, rows, rng.random() < 0.5,
                              rng.choice([0, 1000, 120000]), rng.choice([1.0, 1.0, 4.0, 8.0]))
        elif op == "pages":
            what = rng.choice(["fork", "fork", "compact"])
            cache = rng.choice(["latent", "fp8"])
            heads = 1 if cache == "latent" else rng.choice([1, 2, 4, 8])
            width = rng.choice([320, 576]) if cache == "latent" else rng.choice([64, 128])
            len_max = _log_int(rng, 20, 6000)
            case = _pages_case("", what, cache, _log_int(rng, 1, 192), rng.randint(1, 4) if what == "fork" else 0, heads,
                               width, rng.choice([32, 64, 128]), rng.randint(1, len_max), len_max,
                               _log_int(rng, 1, 300) if what == "fork" else 0, rng.choice([0.1, 0.3, 0.6]))
        else:
            kind = rng.choice(["token", "drafts", "chunk"])
            new_min = new_max = 1
            if kind == "drafts":
                new_max = rng.randint(2, 8)
            elif kind == "chunk":
                new_max = _log_int(rng, 16, 2048)
                new_min = rng.randint(1, new_max)
            len_max = _log_int(rng, 64, 120000)
            if op == "append":
                len_max = min(len_max, 8192)
            case = _latent_case("", op, _log_int(rng, 1, 96), rng.choice([1, 5, 8, 16, 16, 20, 32, 40, 64, 96, 128]),
                                rng.choice([256, 512, 512]), rng.choice([32, 64, 128]),
                                rng.randint(max(1, len_max // 8), len_max), len_max, new_min, new_max, rng.random() < 0.5)
        del case["name"]
        w = work(case)
        if case["op"] == "pages" and (w["bytes"] > 6e8 or _pool_bytes(case) > 1e9):
            continue
        if case["op"] in ("append", "attend"):
            lens, news = _lengths(case)
            padded = case["B"] * max(news) * case["heads"] * max(lens)
            gathered = case["B"] * max(lens) * (case["rank"] + ROPE)
            if w["bytes"] > 4.5e8 or w["flops"] > 5.5e11 or padded > 6e8 or gathered > 3e8:
                continue
        return case


def _lengths(case):
    """kv_len (new tokens included) and new tokens of each sequence, from the case alone."""
    lens, news = [], []
    for b in range(case["B"]):
        f = ((b + 1) * 0.6180339887498949) % 1.0
        g = ((b + 1) * 0.7548776662466927) % 1.0
        t = case["len_min"] + int((case["len_max"] - case["len_min"]) * f)
        if case["B"] == 1:
            t = case["len_max"]
        n = case.get("new_min", 0)
        n = min(n + int((case.get("new_max", 0) - n + 1) * g), max(case.get("new_max", 0), n))
        lens.append(t)
        news.append(min(n, t))
    return lens, news


def _page_bytes(case):
    if case["cache"] == "latent":
        return case["page"] * case["width"] * 2
    return case["kv_heads"] * (2 * case["page"] * case["width"] + 8 + 2 * case["width"])


def _pool(case):
    """Pages held by the sequences, pages of the pool, and pages a compaction moves."""
    lens, _ = _lengths(case)
    ps = case["page"]
    held = sum(-(-t // ps) for t in lens)
    if case["what"] == "fork":
        rows = case["B"] * (1 + case["children"])
        return held, held + rows * (2 + case["grow"] // ps) + 1 + int(case["slack"] * held), 0
    pool = held + 1 + int(case["slack"] * held)
    return held, pool, held * (pool - held) // pool


def _pool_bytes(case):
    return _pool(case)[1] * _page_bytes(case)


def work(case):
    if case["op"] == "rope":
        n = case["B"] * case["H"] * case["N"]
        table = 4 * case["rope_dim"] * case["N"] * (case["B"] if case["far"] else 1)
        return {"bytes": 4 * n * case["d"] + table, "flops": 3 * n * case["rope_dim"]}
    lens, news = _lengths(case)
    if case["op"] == "pages":
        ps = case["page"]
        if case["what"] == "compact":
            held, pool, moved = _pool(case)
            return {"bytes": 2 * moved * _page_bytes(case) + 8 * pool + 8 * held, "flops": 0}
        # of a parent and its children that share a last page all but one get a copy
        copies = case["children"] * sum(1 for t in lens if t % ps)
        entries = case["children"] * sum(-(-t // ps) for t in lens)
        return {"bytes": 2 * copies * _page_bytes(case) + 12 * entries + 4 * _pool(case)[1], "flops": 0}
    T, heads, rank = sum(news), case["heads"], case["rank"]
    if case["op"] == "append":
        return {"bytes": T * 4 * (rank + ROPE) + T * heads * ROPE * 4 + T * ROPE * 4, "flops": 3 * T * (heads + 1) * ROPE}
    seen = sum(n * (t - n) + n * (n + 1) // 2 for t, n in zip(lens, news))     # visible (token, key) pairs
    cached = sum(t for t, n in zip(lens, news) if n)
    return {"bytes": T * heads * (2 * (rank + ROPE) + 2 * rank + 4) + cached * 2 * (rank + ROPE),
            "flops": 2 * (2 * rank + ROPE) * heads * seen}


# ---------------------------------------------------------------- inputs

def _frequencies(rope_dim, factor, dev):
    """Angle per position of each pair, 64 bits. A stretched context (factor > 1) divides those that turn less than once in
    4096 positions by the factor, leaves those that turn 32 times or more, and goes over linearly between; cosines and sines
    grow by 0.1 ln(factor) + 1."""
    inv = 10000.0 ** (-torch.arange(0, rope_dim, 2, dtype=torch.float64, device=dev) / rope_dim)
    if factor == 1.0:
        return inv, 1.0
    keep = ((4096 * inv / (2 * math.pi) - 1.0) / 31.0).clamp(0.0, 1.0)
    return inv * (keep + (1.0 - keep) / factor), 0.1 * math.log(factor) + 1.0


def _table(positions, rope_dim, factor, dev):
    inv, grow = _frequencies(rope_dim, factor, dev)
    ang = torch.arange(positions, dtype=torch.float64, device=dev)[:, None] * inv
    return (torch.cat([ang.cos(), ang.sin()], dim=1) * grow).float()


def _prepare_rope(case, gen, dev):
    B, H, N, d = case["B"], case["H"], case["N"], case["d"]
    s = dict(case=case)
    if case["rows"]:
        # rows of a projection whose heads are 2 d wider: [T, H, d] slices
        s["x"] = torch.randn(N, H, 3 * d, generator=gen, device=dev).to(torch.bfloat16)[:, :, 2 * d:]
    else:
        s["x"] = torch.randn(B, H, N, d, generator=gen, device=dev).to(torch.bfloat16)
    s["positions"] = None
    last = N
    if case["far"]:
        last = case["far"] + N
        shape = (N,) if case["rows"] else (B, N)
        s["positions"] = torch.randint(0, last, shape, generator=gen, device=dev, dtype=torch.int32)
    s["rope"] = _table(last, case["rope_dim"], case["factor"], dev)
    return s


def _prepare_pages(case, gen, dev):
    lens, _ = _lengths(case)
    B, ps, width, heads = case["B"], case["page"], case["width"], case["kv_heads"]
    held, pool, moved = _pool(case)
    n_pages = [-(-t // ps) for t in lens]
    rows = B * (1 + case["children"])
    max_pages = max(n_pages) + 1 + case["grow"] // ps
    s = dict(case=case, page=ps, pool=pool, rows=rows, max_pages=max_pages)
    # one buffer of table, lengths and reference counts, and the state it is taken back to before every pass
    s["start"] = torch.full((rows * max_pages + rows + pool,), -1, dtype=torch.int32, device=dev)
    s["meta"] = torch.empty_like(s["start"])
    table, kv_len, refs = _meta(s, s["start"])
    if case["what"] == "fork":
        used = torch.randperm(pool, generator=gen, device=dev)[:held]
        s["parents"] = torch.arange(B, dtype=torch.int32, device=dev).repeat_interleave(case["children"])
        s["children"] = torch.arange(B, rows, dtype=torch.int32, device=dev)
    else:
        # held pages with `moved` holes among the first and as many behind
        low = torch.randperm(held, generator=gen, device=dev)[: held - moved]
        high = held + torch.randperm(pool - held, generator=gen, device=dev)[:moved]
        used = torch.cat([low, high])[torch.randperm(held, generator=gen, device=dev)]
    slot = torch.arange(max_pages, device=dev)[None, :] < torch.tensor(n_pages + [0] * (rows - B), device=dev)[:, None]
    table[slot] = used.to(torch.int32)
    kv_len.zero_()
    kv_len[:B] = torch.tensor(lens, dtype=torch.int32, device=dev)
    refs.zero_()
    refs[used] = 1
    s["meta"].copy_(s["start"])
    if case["cache"] == "latent":
        s["data"] = torch.randn(pool, ps, width, generator=gen, device=dev).to(torch.bfloat16)
        return s
    for name in ("k", "v"):
        x = torch.randn(pool, heads, ps, width, generator=gen, device=dev) * 100.0
        s[name] = x.to(torch.float8_e4m3fn).view(torch.uint8)
        s[name + "_scale"] = torch.exp2(torch.randint(-9, -5, (pool, heads), generator=gen, device=dev).float())
    s["k_bounds"] = torch.randint(-127, 128, (pool, heads, 2, width), generator=gen, device=dev).to(torch.int8)
    return s


def _meta(s, buffer):
    n = s["rows"] * s["max_pages"]
    return buffer[:n].view(s["rows"], s["max_pages"]), buffer[n: n + s["rows"]], buffer[n + s["rows"]:]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    if case["op"] == "rope":
        return _prepare_rope(case, gen, dev)
    if case["op"] == "pages":
        return _prepare_pages(case, gen, dev)
    lens, news = _lengths(case)
    B, heads, rank, ps = case["B"], case["heads"], case["rank"], case["page"]
    T = sum(news)
    n_pages = [-(-t // ps) for t in lens]
    total, max_pages = sum(n_pages), max(n_pages)
    pages = total + 3
    # the scale of heads of 128 columns and the rotated ones before their projections were absorbed
    s = dict(case=case, rank=rank, page=ps, heads=heads, scale=1.0 / math.sqrt(128 + ROPE))
    s["kv_len"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    starts = [0]
    for n in news:
        starts.append(starts[-1] + n)
    s["q_start"] = torch.tensor(starts, dtype=torch.int32, device=dev)
    perm = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)[:total]
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device=dev)
    held = torch.arange(max_pages, device=dev)[None, :] < torch.tensor(n_pages, device=dev)[:, None]
    table[held] = perm
    s["page_table"] = table
    # latents of normed rows with a few strong channels, key parts with a slow drift
    channel = 0.5 + torch.rand(rank + ROPE, generator=gen, device=dev)
    channel[:: 64] *= 2.5
    data = torch.randn(pages, ps, rank + ROPE, generator=gen, device=dev) * channel
    data[..., rank:] += 0.3 * torch.randn(pages, 1, ROPE, generator=gen, device=dev)
    s["data"] = data.to(torch.bfloat16)
    if case["op"] == "append":
        # one projection's rows: latent and key part side by side; query heads of 128 plain and 64 rotated columns
        new = (torch.randn(T, rank + ROPE, generator=gen, device=dev) * channel).to(torch.bfloat16)
        s["latent"], s["k_rope"] = new[:, :rank], new[:, rank:]
        s["q_rope"] = torch.randn(T, heads, 128 + ROPE, generator=gen, device=dev).to(torch.bfloat16)[:, :, 128:]
        s["q"] = torch.zeros(T, heads, rank + ROPE, dtype=torch.bfloat16, device=dev)
        s["rope"] = _table(max(lens), ROPE, 1.0, dev)
    else:
        s["q"] = torch.randn(T, heads, rank + ROPE, generator=gen, device=dev).to(torch.bfloat16)
    return s


# ---------------------------------------------------------------- plain forms

def _rotate(x, cos, sin, interleaved):
    """x [..., d] in fp32, cos and sin [..., pairs]; the first 2 * pairs columns are rotated."""
    h = cos.shape[-1]
    if interleaved:
        a, b = x[..., 0: 2 * h: 2], x[..., 1: 2 * h: 2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = x[..., :h], x[..., h: 2 * h]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([y, x[..., 2 * h:]], dim=-1)


def _rope(s):
    c, x = s["case"], s["x"].float()
    h = c["rope_dim"] // 2
    at = torch.arange(c["N"], device=x.device) if s["positions"] is None else s["positions"].long()
    rows = s["rope"][at]                                  # [N or B, N, rope_dim]
    if c["rows"]:
        rows = rows[:, None]                              # [T, 1, .]: heads share a row
    elif rows.dim() == 3:
        rows = rows[:, None]                              # [B, 1, N, .]
    cos, sin = rows[..., :h], rows[..., h:]
    return _rotate(x, cos, -sin if c["backward"] else sin, c["interleaved"]).to(torch.bfloat16)


def _rows(s):
    """Sequence and position of each row of the call."""
    q_start, kv_len = s["q_start"].long(), s["kv_len"].long()
    row = torch.arange(s["q"].shape[0], device=q_start.device)
    b = torch.searchsorted(q_start, row, right=True) - 1
    return b, kv_len[b] - (q_start[b + 1] - q_start[b]) + row - q_start[b]


def _append(s):
    b, pos = _rows(s)
    ps, rank, inter = s["page"], s["rank"], s["case"]["interleaved"]
    h = ROPE // 2
    cos, sin = s["rope"][pos][:, :h], s["rope"][pos][:, h:]
    page, slot = s["page_table"].long()[b, pos // ps], pos % ps
    key = _rotate(s["k_rope"].float(), cos, sin, inter)
    s["data"][page, slot] = torch.cat([s["latent"].float(), key], dim=1).to(torch.bfloat16)
    s["q"][:, :, rank:] = _rotate(s["q_rope"].float(), cos[:, None], sin[:, None], inter).to(torch.bfloat16)


def _attend(s):
    b, pos = _rows(s)
    T, heads, width = s["q"].shape
    B, max_pages = s["page_table"].shape
    keys = max_pages * s["page"]
    k = s["data"][s["page_table"].long().clamp(min=0)].float().flatten(1, 2)          # [B, keys, width]
    key = torch.arange(keys, device=k.device)
    k = k.masked_fill(key[None, :, None] >= s["kv_len"][:, None, None], 0.0)
    n = max(_lengths(s["case"])[1])
    at = torch.arange(T, device=b.device) - s["q_start"].long()[b]
    q = torch.zeros(B, n, heads, width, device=k.device)
    q[b, at] = s["q"].float()
    limit = torch.zeros(B, n, dtype=torch.long, device=k.device)
    limit[b, at] = pos + 1
    x = torch.matmul(q.view(B, n * heads, width), k.transpose(1, 2)) * s["scale"]
    x = x.masked_fill(key >= limit.repeat_interleave(heads, dim=1)[:, :, None], -math.inf)
    m = x.amax(dim=-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    l = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p, k[:, :, : s["rank"]]) / torch.where(l == 0, torch.ones_like(l), l)
    lse = (m + torch.log(l))[..., 0]
    o = o.view(B, n, heads, s["rank"])[b, at]
    return o.to(torch.bfloat16), lse.view(B, n, heads)[b, at]


def _planes(s):
    return [s["data"]] if "data" in s else [s["k"], s["v"], s["k_scale"], s["v_scale"], s["k_bounds"]]


def _held(kv_len, ps):
    return (kv_len.long() + ps - 1) // ps


def _fork(s, table, kv_len, refs):
    p, c = s["parents"].long(), s["children"].long()
    rows = table[p]
    live = torch.arange(table.shape[1], device=table.device)[None, :] < _held(kv_len[p], s["page"])[:, None]
    table[c] = torch.where(live, rows, table[c])
    refs.scatter_add_(0, rows.clamp(min=0).long().flatten(), live.flatten().to(torch.int32))
    kv_len[c] = kv_len[p]


def _extend(s, table, old, new, refs):
    ps, B = s["page"], table.shape[0]
    row, slot = torch.arange(B, device=table.device), torch.arange(table.shape[1], device=table.device)
    first, last = _held(old, ps), _held(new, ps)
    at = (old.long() // ps).clamp(max=table.shape[1] - 1)
    tail = table[row, at].long()
    writes = (old % ps != 0) & (new > old)
    # sequences are served in order, so the last one that shares a page keeps it
    before = writes[None, :] & (tail[:, None] == tail[None, :]) & (row[None, :] < row[:, None])
    copy = writes & (refs[tail.clamp(min=0)] - before.sum(dim=1) >= 2)
    need = copy.long() + (last - first).clamp(min=0)
    start = need.cumsum(0) - need
    free = torch.sort(torch.where(refs == 0, torch.arange(refs.shape[0], device=refs.device), refs.shape[0]))[0]
    to, what = free[start[copy]], tail[copy]
    for plane in _planes(s):
        plane[to] = plane[what]
    refs.scatter_add_(0, what, torch.full_like(what, -1, dtype=torch.int32))
    table[row[copy], at[copy]] = to.to(torch.int32)
    grown = (slot[None, :] >= first[:, None]) & (slot[None, :] < last[:, None])
    pick = (start + copy.long() - first)[:, None] + slot[None, :]
    table.copy_(torch.where(grown, free[pick.clamp(0, refs.shape[0] - 1)].to(torch.int32), table))
    refs[free[: need.sum()]] = 1


def _compact(s, table, kv_len, refs):
    page = torch.arange(refs.shape[0], device=refs.device)
    used = refs > 0
    total = used.sum()
    src, dst = page[used & (page >= total)], page[~used & (page < total)]
    where = page.clone()
    where[src] = dst
    for plane in _planes(s):
        plane[dst] = plane[src]
    refs[dst] = refs[src]
    refs[src] = 0
    live = torch.arange(table.shape[1], device=table.device)[None, :] < _held(kv_len, s["page"])[:, None]
    table.copy_(torch.where(live, where[table.clamp(min=0).long()].to(torch.int32), table))


def _pages_out(s, table, kv_len, refs):
    out = {"table": table, "refs": refs, "kv_len": kv_len}
    if "data" in s:
        return {**out, "data": s["data"]}
    return {**out, "k": s["k"].view(torch.float8_e4m3fn), "v": s["v"].view(torch.float8_e4m3fn),
            "k_scale": s["k_scale"], "v_scale": s["v_scale"], "k_bounds": s["k_bounds"]}


def _pages(s):
    c = s["case"]
    s["meta"].copy_(s["start"])          # a pass begins where the last one began
    table, kv_len, refs = _meta(s, s["meta"])
    if own:
        from exact_attention_fattn_gb300 import (Fp8Cache, LatentCache, PagePool, fattn_pages_compact,
                                                 fattn_pages_extend, fattn_pages_fork)

        pool = PagePool(refs)
        cache = LatentCache(s["data"], c["width"] - ROPE) if "data" in s else Fp8Cache(*_planes(s))
        if c["what"] == "compact":
            fattn_pages_compact(pool, cache, table, kv_len)
        else:
            fattn_pages_fork(pool, cache, table, kv_len, s["parents"], s["children"])
            fattn_pages_extend(pool, cache, table, kv_len, kv_len + c["grow"])
    elif c["what"] == "compact":
        _compact(s, table, kv_len, refs)
    else:
        _fork(s, table, kv_len, refs)
        _extend(s, table, kv_len, kv_len + c["grow"], refs)
    return _pages_out(s, table, kv_len, refs)


def run(state):
    s, c = state, state["case"]
    if c["op"] == "pages":
        return _pages(s)
    if own:
        from exact_attention_fattn_gb300 import (LatentCache, fattn_latent_append, fattn_latent_fwd, fattn_rope,
                                                 fattn_rope_bwd)

        if c["op"] == "rope":
            turn = fattn_rope_bwd if c["backward"] else fattn_rope
            return {"y": turn(s["x"], s["rope"], positions=s["positions"], interleaved=c["interleaved"])}
        cache = LatentCache(s["data"], s["rank"])
        where = (s["page_table"], s["q_start"], s["kv_len"])
        if c["op"] == "append":
            fattn_latent_append(s["latent"], s["k_rope"], cache, *where, rope=s["rope"], q_rope=s["q_rope"], q=s["q"],
                                interleaved=c["interleaved"])
            return {"q": s["q"], "data": s["data"]}
        o, lse = fattn_latent_fwd(s["q"], cache, *where, scale=s["scale"])
        return {"o": o, "lse": lse}
    if c["op"] == "rope":
        return {"y": _rope(s)}
    if c["op"] == "append":
        _append(s)
        return {"q": s["q"], "data": s["data"]}
    o, lse = _attend(s)
    return {"o": o, "lse": lse}


# ---------------------------------------------------------------- 64 bits

def _turned(x, position, rope_dim, factor, interleaved, back=False):
    """x [..., d] rotated in 64 bits by the angles of `position` (of a shape that broadcasts to x's without its last)."""
    x = x.double()
    i = torch.arange(rope_dim // 2, device=x.device)
    inv, grow = _frequencies(rope_dim, factor, x.device)
    z = torch.polar(torch.full_like(position, grow, dtype=torch.float64)[..., None].expand(*position.shape, len(i)),
                    position.double()[..., None] * inv)
    if back:
        z = z.conj()
    i0, i1 = (2 * i, 2 * i + 1) if interleaved else (i, i + rope_dim // 2)
    w = torch.complex(x[..., i0], x[..., i1]) * z
    y = x.clone()
    y[..., i0], y[..., i1] = w.real, w.imag
    return y


def exact(case, seed):
    if case["op"] == "pages" or work(case)["flops"] > 1.2e12:
        return None
    s = prepare(case, seed)
    if case["op"] == "rope":
        N = case["N"]
        at = torch.arange(N, device=s["x"].device) if s["positions"] is None else s["positions"]
        if case["rows"] or at.dim() == 2:
            at = at.unsqueeze(1)
        return {"y": _turned(s["x"], at, case["rope_dim"], case["factor"], case["interleaved"], case["backward"])}
    lens, news = _lengths(case)
    ps, rank, heads = case["page"], case["rank"], case["heads"]
    row = 0
    if case["op"] == "append":
        data, q = s["data"].double(), s["q"].double()
        for b, (t, n) in enumerate(zip(lens, news)):
            at = torch.arange(t - n, t, device=data.device)
            page = s["page_table"][b].long()[at // ps]
            data[page, at % ps, :rank] = s["latent"][row: row + n].double()
            data[page, at % ps, rank:] = _turned(s["k_rope"][row: row + n], at, ROPE, 1.0, case["interleaved"])
            q[row: row + n, :, rank:] = _turned(s["q_rope"][row: row + n], at[:, None], ROPE, 1.0, case["interleaved"])
            row += n
        return {"q": q, "data": data}
    outs, lses = [], []
    for b, (t, n) in enumerate(zip(lens, news)):
        if not n:
            continue
        k = s["data"][s["page_table"][b, : -(-t // ps)].long()].double().reshape(-1, rank + ROPE)[:t]
        key = torch.arange(t, device=k.device)
        for i0 in range(0, n, 128):
            i = torch.arange(i0, min(n, i0 + 128), device=k.device)
            x = torch.einsum("rhd,kd->rhk", s["q"][row + i].double(), k) * s["scale"]
            x = x.masked_fill((key[None, :] > (t - n + i)[:, None])[:, None], -math.inf)
            lse = torch.logsumexp(x, dim=2)
            outs.append(torch.einsum("rhk,kd->rhd", torch.exp(x - lse[..., None]), k[:, :rank]))
            lses.append(lse)
        row += n
    return {"o": torch.cat(outs), "lse": torch.cat(lses)}
