"""Attention over a paged 8-bit cache: the cases that are measured, and the operators in plain form.

Three operators share the cache (e4m3 codes [pages, kv heads, page, d], one power-of-two scale per page and head):

* append: rotate new queries and keys by their positions, quantise keys and values into the cache's pages;
* attend: causal attention of new tokens over their sequences' cached tokens, from one token to prompt chunks;
* sparse: pages selected for each token and kv head by a score from per-page bounds of the keys, then attention over
  the selected pages only.

Sequences are ragged: sequence b has rows q_start[b] .. q_start[b + 1] of the call, kv_len[b] cached tokens (the new ones
included) and its pages in page_table[b]. Lengths follow from the case alone, values and the order of pages from the seed.
"""

import math

import torch

own = False

E4M3_MAX = 448.0
E_MIN, E_MAX = -48, 48          # range of the scales' exponents


# ---------------------------------------------------------------- cases

def _case(name, op, B, kv_heads, group, d, page, len_min, len_max, new_min, new_max, rope_dim=0, interleaved=False,
          n_selected=0, n_first=0, n_recent=0):
    return dict(name=name, op=op, B=B, kv_heads=kv_heads, group=group, d=d, page=page, len_min=len_min, len_max=len_max,
                new_min=new_min, new_max=new_max, rope_dim=rope_dim, interleaved=interleaved, n_selected=n_selected,
                n_first=n_first, n_recent=n_recent)


def listed():
    return [
        # the step of a serving batch: one token for each of 32 sequences
        _case("append tokens", "append", 32, 8, 4, 128, 64, 200, 4000, 1, 1, rope_dim=128),
        # four whole prompts into fresh pages
        _case("append prompts", "append", 4, 8, 4, 128, 128, 3000, 4096, 4096, 4096, rope_dim=128),
        # prompts in pieces behind what is cached, small heads, neighbouring pairs rotated, half of the head
        _case("append pieces", "append", 7, 2, 7, 64, 32, 900, 3001, 1, 701, rope_dim=32, interleaved=True),
        # one user, one token: latency counts
        _case("attend one token", "attend", 1, 8, 4, 128, 64, 1000, 1000, 1, 1),
        # a full serving batch of very different lengths
        _case("attend token batch", "attend", 64, 8, 8, 128, 64, 500, 8000, 1, 1),
        # few users with long contexts
        _case("attend long context", "attend", 2, 8, 4, 128, 128, 100003, 131071, 1, 1),
        # heads that share nothing, d = 64, short contexts
        _case("attend unshared heads", "attend", 32, 16, 1, 64, 32, 100, 2500, 1, 1),
        # five drafted tokens of each sequence at once
        _case("attend drafts", "attend", 32, 8, 8, 128, 64, 1000, 4000, 5, 5),
        # a piece of a long prompt behind what is cached
        _case("attend prompt piece", "attend", 2, 8, 4, 128, 64, 14336, 16384, 2048, 2048),
        # long contexts in a batch, 2048 tokens attended of each
        _case("sparse batch", "sparse", 16, 8, 4, 128, 64, 20000, 65536, 1, 1, n_selected=32, n_first=1, n_recent=2),
        # one user with a long context and three drafted tokens
        _case("sparse one user", "sparse", 1, 4, 8, 128, 32, 30011, 30011, 3, 3, n_selected=48, n_first=1, n_recent=1),
        # small heads, one page out of eight
        _case("sparse small heads", "sparse", 24, 4, 2, 64, 128, 4000, 16000, 1, 1, n_selected=16, n_first=0, n_recent=1),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "sparse"])
    while True:
        kv_heads = rng.choice([1, 2, 3, 4, 8, 16])
        group = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
        d = rng.choice([64, 128, 128])
        page = rng.choice([32, 64, 128])
        B = _log_int(rng, 1, 96)
        kind = rng.choice(["token", "drafts", "chunk"])
        rope_dim, interleaved, sel = 0, False, (0, 0, 0)
        if kind == "token":
            new_min = new_max = 1
        elif kind == "drafts":
            new_min, new_max = 1, rng.randint(2, 9)
        else:
            new_max = _log_int(rng, 16, 4096)
            new_min = rng.randint(1, new_max)
        len_max = _log_int(rng, 64, 120000)
        len_min = rng.randint(max(1, len_max // 8), len_max)
        if op == "append":
            rope_dim = rng.choice([0, d // 2, d, d])
            interleaved = rng.random() < 0.5
            len_max = min(len_max, 8192)
            len_min = min(len_min, len_max)
        if op == "sparse":
            new_max = min(new_max, 8)
            new_min = min(new_min, new_max)
            k = _log_int(rng, 4, 96)
            n_first, n_recent = rng.randint(0, 2), rng.randint(0, 2)
            sel = (k, n_first, n_recent)
        case = _case("", op, B, kv_heads, group, d, page, len_min, len_max, new_min, new_max, rope_dim, interleaved, *sel)
        del case["name"]
        w = work(case)
        lens, news = _lengths(case)
        cached = sum(lens) * kv_heads * d * 2
        padded = B * max(news) * max(lens) * kv_heads * group
        if cached <= 5e8 and w["flops"] <= 1e12 and w["bytes"] <= 4e8 and padded <= 2.1e9 and B * max(lens) * kv_heads * d <= 4e8:
            return case


def _lengths(case):
    """kv_len (new tokens included) and new tokens of each sequence, from the case alone."""
    lens, news = [], []
    for b in range(case["B"]):
        f = ((b + 1) * 0.6180339887498949) % 1.0
        g = ((b + 1) * 0.7548776662466927) % 1.0
        n = case["new_min"] + int((case["new_max"] - case["new_min"] + 1) * g)
        n = min(n, case["new_max"])
        t = case["len_min"] + int((case["len_max"] - case["len_min"]) * f)
        if case["B"] == 1:
            t = case["len_max"]
        lens.append(t)
        news.append(min(n, t))
    return lens, news


def work(case):
    lens, news = _lengths(case)
    T, kvh, g, d = sum(news), case["kv_heads"], case["group"], case["d"]
    hq = kvh * g
    if case["op"] == "append":
        rows = T * d * (2 * hq * 2 + 2 * kvh * 2 + 2 * kvh)       # q in and out, k and v in, codes out
        table = 4 * T * case["rope_dim"]
        return {"bytes": rows + table, "flops": 3 * T * (hq + kvh) * case["rope_dim"] + 4 * T * kvh * d}
    q_and_o = T * hq * (4 * d + 4)
    if case["op"] == "attend":
        seen = sum(n * (t - n) + n * (n + 1) // 2 for t, n in zip(lens, news))     # visible (token, key) pairs
        cached = sum(t for t, n in zip(lens, news) if n)
        scales = 8 * kvh * sum(-(-t // case["page"]) for t in lens)
        return {"bytes": q_and_o + 2 * cached * kvh * d + scales, "flops": 4 * d * hq * seen}
    pages = [-(-t // case["page"]) for t in lens]
    bounds = sum(pages) * kvh * (2 * d + 4)
    k, ps = case["n_selected"], case["page"]
    seen = sum(n * min(t, k * ps) for t, n in zip(lens, news))
    # one sequence's tokens may share pages: at least the largest set of one token is read
    codes = sum(min(t, k * ps) for t, n in zip(lens, news) if n) * kvh * 2 * d
    return {"bytes": q_and_o + bounds + codes + 4 * T * kvh * k,
            "flops": 4 * d * hq * seen + 4 * d * kvh * sum(n * p for n, p in zip(news, pages))}


# ---------------------------------------------------------------- inputs

def _exponent(amax):
    """The smallest e in [E_MIN, E_MAX] with amax <= 448 * 2^e (448 = 0.875 * 2^9)."""
    m, x = torch.frexp(amax)
    e = torch.where(m > 0.875, x - 8, x - 9)
    return torch.where(amax > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)


def _bounds_of(codes):
    """floor and ceil of 127 / 448 times the codes' values, [..., page, d] -> [..., page, d] each (as floats).

    On a GPU a division by a number is a product with its rounded reciprocal, which takes 448 to just above 127."""
    t = codes * 127.0 / E4M3_MAX
    return torch.floor(t).clamp(min=-127.0), torch.ceil(t).clamp(max=127.0)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    lens, news = _lengths(case)
    B, kvh, d, ps = case["B"], case["kv_heads"], case["d"], case["page"]
    hq = kvh * case["group"]
    T = sum(news)
    n_pages = [-(-t // ps) for t in lens]
    total, spare = sum(n_pages), 3
    max_pages = max(n_pages)
    pages = total + spare

    s = dict(case=case, d=d, page=ps, kv_heads=kvh, q_heads=hq, scale=1.0 / math.sqrt(d))
    s["kv_len"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    starts = [0]
    for n in news:
        starts.append(starts[-1] + n)
    s["q_start"] = torch.tensor(starts, dtype=torch.int32, device=dev)
    perm = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)[:total]
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device=dev)
    slot = torch.arange(max_pages, device=dev)[None, :]
    held = slot < torch.tensor(n_pages, device=dev)[:, None]
    table[held] = perm
    s["page_table"] = table

    # What the cache holds: keys with a few strong channels and a slow drift from page to page, values of varying size.
    channel = 0.5 + torch.rand(kvh, 1, d, generator=gen, device=dev)
    channel[:, :, :: max(1, d // 4)] *= 3.0

    def filled(spread, per_channel):
        x = torch.randn(pages, kvh, ps, d, generator=gen, device=dev)
        x *= torch.exp(spread * torch.randn(pages, kvh, 1, 1, generator=gen, device=dev))
        if per_channel:
            x *= channel
            x += 0.5 * torch.randn(pages, kvh, 1, d, generator=gen, device=dev)
        scale = torch.exp2(_exponent(x.abs().amax(dim=(2, 3))).float())
        codes = (x / scale[:, :, None, None]).to(torch.float8_e4m3fn)
        return codes, scale

    k, k_scale = filled(0.2, True)
    v, v_scale = filled(0.5, False)
    lo, hi = torch.zeros(pages, kvh, d, device=dev), torch.zeros(pages, kvh, d, device=dev)
    if case["op"] != "attend":
        lo, hi = _bounds_of(k.float())
        lo, hi = lo.amin(dim=2), hi.amax(dim=2)
    s["k"], s["v"] = k.view(torch.uint8), v.view(torch.uint8)
    s["k_scale"], s["v_scale"] = k_scale, v_scale
    s["k_bounds"] = torch.stack([lo, hi], dim=2).to(torch.int8).contiguous()
    if case["op"] == "append":
        # rows of one fused projection: q, k and v of a token side by side
        qkv = torch.randn(T, (hq + 2 * kvh) * d, generator=gen, device=dev)
        qkv = qkv.to(torch.bfloat16)
        s["q"] = qkv[:, : hq * d].unflatten(1, (hq, d))
        s["k_new"] = qkv[:, hq * d: (hq + kvh) * d].unflatten(1, (kvh, d))
        s["v_new"] = qkv[:, (hq + kvh) * d:].unflatten(1, (kvh, d))
        rd = case["rope_dim"]
        s["rope"] = None
        if rd:
            # angles of far positions need 64 bits
            inv = 10000.0 ** (-torch.arange(0, rd, 2, dtype=torch.float64, device=dev) / rd)
            ang = torch.arange(max(lens), dtype=torch.float64, device=dev)[:, None] * inv
            s["rope"] = torch.cat([ang.cos(), ang.sin()], dim=1).float()
    else:
        s["q"] = torch.randn(T, hq, d, generator=gen, device=dev).to(torch.bfloat16)
    return s


# ---------------------------------------------------------------- plain forms

def _rows(s):
    """Sequence, position and table slot of each row of the call."""
    q_start, kv_len = s["q_start"].long(), s["kv_len"].long()
    T = s["q"].shape[0]
    row = torch.arange(T, device=q_start.device)
    b = torch.searchsorted(q_start, row, right=True) - 1
    pos = kv_len[b] - (q_start[b + 1] - q_start[b]) + row - q_start[b]
    return b, pos


def _rotate(x, cos, sin, interleaved):
    """x [T, heads, d] in fp32; the first 2 * cos.shape[1] columns are rotated."""
    h = cos.shape[1]
    cos, sin = cos[:, None, :], sin[:, None, :]
    if interleaved:
        a, b = x[..., 0: 2 * h: 2], x[..., 1: 2 * h: 2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = x[..., :h], x[..., h: 2 * h]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([y, x[..., 2 * h:]], dim=-1)


def _append_one(codes, scales, page, slot, fresh, first, x, bounds):
    """Quantise x [T, heads, d] into the pages; `first`: the first new slot of each page (page size where none is new)."""
    touched = first < codes.shape[2]
    amax = torch.zeros(codes.shape[:2], device=x.device)
    amax.scatter_reduce_(0, page[:, None].expand(-1, x.shape[1]), x.abs().amax(dim=2), "amax")
    e_new = _exponent(amax)
    e_old = _exponent(scales * E4M3_MAX)
    e = torch.where(fresh[:, None], e_new, torch.maximum(e_old, e_new))
    e = torch.where(touched[:, None], e, e_old)
    down = torch.exp2((e_old - e).float())
    # what the pages that receive tokens held: rounded again where their scale grew
    at = touched.nonzero()[:, 0]
    held = codes[at].view(torch.float8_e4m3fn).float()
    keep = torch.arange(codes.shape[2], device=x.device)[None, :] < first[at][:, None]
    again = torch.where(keep[:, None, :, None], held * down[at][:, :, None, None], held)
    codes[at] = again.to(torch.float8_e4m3fn).view(torch.uint8)
    scales.copy_(torch.exp2(e.float()))
    new = (x * torch.exp2(-e.float())[page][:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    codes[page, :, slot] = new.view(torch.uint8)
    if bounds is not None:
        lo, hi = _bounds_of(new.float())
        old = bounds.float() * torch.where(fresh, torch.zeros(()).to(x.device), torch.ones(()).to(x.device))[:, None, None, None]
        none = torch.where(fresh, torch.full((), 1e9, device=x.device), torch.zeros((), device=x.device))[:, None, None]
        low = torch.floor(old[:, :, 0] * down[:, :, None]) + none
        high = torch.ceil(old[:, :, 1] * down[:, :, None]) - none
        where = page[:, None, None].expand_as(lo)
        low.scatter_reduce_(0, where, lo, "amin")
        high.scatter_reduce_(0, where, hi, "amax")
        bounds.copy_(torch.where(touched[:, None, None, None], torch.stack([low, high], dim=2), bounds.float()).to(torch.int8))


def _append(s):
    b, pos = _rows(s)
    ps = s["page"]
    page = s["page_table"].long()[b, pos // ps]
    slot = pos % ps
    q, k, v = s["q"].float(), s["k_new"].float(), s["v_new"].float()
    if s["rope"] is not None:
        h = s["rope"].shape[1] // 2
        cos, sin = s["rope"][pos][:, :h], s["rope"][pos][:, h:]
        q = _rotate(q, cos, sin, s["case"]["interleaved"])
        k = _rotate(k, cos, sin, s["case"]["interleaved"])
    first = torch.full((s["k"].shape[0],), ps, dtype=torch.long, device=page.device)
    first.scatter_reduce_(0, page, slot, "amin")
    fresh = first == 0
    _append_one(s["k"], s["k_scale"], page, slot, fresh, first, k, s["k_bounds"])
    _append_one(s["v"], s["v_scale"], page, slot, fresh, first, v, None)
    return q.to(torch.bfloat16)


def _values(codes, scale):
    return codes.view(torch.float8_e4m3fn).float() * scale[..., None, None]


def _softmax_v(x, see, v):
    """x: scores [..., rows, keys]; see: visible; v [..., keys, d]. Rows that see nothing give 0 and -inf."""
    x = x.masked_fill(~see, -math.inf)
    m = x.amax(dim=-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    l = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(l == 0, torch.ones_like(l), l)
    return o, (m + torch.log(l))[..., 0]


def _attend(s):
    b, pos = _rows(s)
    T, hq, d = s["q"].shape
    kvh, ps = s["kv_heads"], s["page"]
    g = hq // kvh
    B, max_pages = s["page_table"].shape
    table = s["page_table"].long().clamp(min=0)
    k = _values(s["k"][table], s["k_scale"][table]).transpose(1, 2).flatten(2, 3)       # [B, kv heads, keys, d]
    v = _values(s["v"][table], s["v_scale"][table]).transpose(1, 2).flatten(2, 3)
    v = v.masked_fill(torch.arange(max_pages * ps, device=v.device)[None, None, :, None] >= s["kv_len"][:, None, None, None], 0.0)
    n = max(_lengths(s["case"])[1])
    at = torch.arange(T, device=b.device) - s["q_start"].long()[b]
    q = torch.zeros(B, n, hq, d, device=k.device)
    q[b, at] = s["q"].float()
    limit = torch.zeros(B, n, dtype=torch.long, device=k.device)
    limit[b, at] = pos + 1
    q = q.view(B, n, kvh, g, d).transpose(1, 2).reshape(B, kvh, n * g, d)
    x = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    see = torch.arange(max_pages * ps, device=k.device) < limit.repeat_interleave(g, dim=1)[:, None, :, None]
    o, lse = _softmax_v(x, see, v)
    o = o.view(B, kvh, n, g, d).transpose(1, 2).reshape(B, n, hq, d)[b, at]
    lse = lse.view(B, kvh, n, g).transpose(1, 2).reshape(B, n, hq)[b, at]
    return o.to(torch.bfloat16), lse


def _select(s):
    b, pos = _rows(s)
    T, hq, d = s["q"].shape
    kvh, ps, c = s["kv_heads"], s["page"], s["case"]
    q = s["q"].float().view(T, kvh, hq // kvh, d)
    amax = q.abs().amax(dim=(2, 3), keepdim=True)
    q8 = torch.round(q * torch.where(amax > 0, 127.0 / amax, torch.zeros_like(amax)))
    up, down = q8.clamp(min=0).sum(dim=2), q8.clamp(max=0).sum(dim=2)                   # [T, kv heads, d], whole numbers
    table = s["page_table"].long().clamp(min=0)[b]                                      # [T, max pages]
    bounds = s["k_bounds"][table]                                                       # [T, max pages, kv heads, 2, d]
    # sums of whole numbers up to 2^27: exact in 64 bits
    whole = (up[:, None].double() * bounds[:, :, :, 1] + down[:, None].double() * bounds[:, :, :, 0]).sum(dim=3)
    score = (whole.float() * s["k_scale"][table]).transpose(1, 2)                       # [T, kv heads, max pages]
    at = torch.arange(table.shape[1], device=q.device)
    pages = ((pos + ps) // ps)[:, None, None]
    score = torch.where((at < c["n_first"]) | (at >= pages - c["n_recent"]), math.inf, score)
    score = torch.where(at < pages, score, -math.inf)
    k = c["n_selected"]
    top = torch.sort(score, dim=2, descending=True, stable=True)[1][:, :, :k]
    top = torch.where(top < pages, top, table.shape[1])
    top = torch.sort(top, dim=2)[0]
    top = torch.where(top < pages, top, -1)
    top = torch.cat([top, top.new_full((T, kvh, k - top.shape[2]), -1)], dim=2)
    return top.to(torch.int32)


def _attend_selected(s, selected):
    b, pos = _rows(s)
    T, hq, d = s["q"].shape
    kvh, ps = s["kv_heads"], s["page"]
    g = hq // kvh
    sel = selected.long()
    page = torch.gather(s["page_table"].long().clamp(min=0)[b][:, None].expand(-1, kvh, -1), 2, sel.clamp(min=0))
    head = torch.arange(kvh, device=page.device)[None, :, None]
    k = _values(s["k"][page, head], s["k_scale"][page, head]).flatten(2, 3)             # [T, kv heads, keys, d]
    v = _values(s["v"][page, head], s["v_scale"][page, head]).flatten(2, 3)
    key = (sel[..., None] * ps + torch.arange(ps, device=page.device)).flatten(2)
    see = (sel >= 0).repeat_interleave(ps, dim=2) & (key <= pos[:, None, None])
    v = v.masked_fill(~see[..., None], 0.0)
    q = s["q"].float().view(T, kvh, g, d)
    x = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    o, lse = _softmax_v(x, see[:, :, None, :], v)
    return o.reshape(T, hq, d).to(torch.bfloat16), lse.reshape(T, hq)


def _cache_out(s):
    return {"k": s["k"].view(torch.float8_e4m3fn), "v": s["v"].view(torch.float8_e4m3fn), "k_scale": s["k_scale"],
            "v_scale": s["v_scale"], "k_bounds": s["k_bounds"]}


def run(state):
    s, c = state, state["case"]
    if own:
        from exact_attention_fattn_gb300 import (Fp8Cache, fattn_cache_append, fattn_cache_fwd, fattn_cache_select)

        cache = Fp8Cache(s["k"], s["v"], s["k_scale"], s["v_scale"], s["k_bounds"])
        where = (s["page_table"], s["q_start"], s["kv_len"])
        if c["op"] == "append":
            q = fattn_cache_append(s["k_new"], s["v_new"], cache, *where, rope=s["rope"], q=s["q"],
                                   interleaved=c["interleaved"])
            return {"q": q, **_cache_out(s)}
        if c["op"] == "attend":
            o, lse = fattn_cache_fwd(s["q"], cache, *where, causal=True)
            return {"o": o, "lse": lse}
        selected = fattn_cache_select(s["q"], cache, *where, c["n_selected"], n_first=c["n_first"], n_recent=c["n_recent"])
        o, lse = fattn_cache_fwd(s["q"], cache, *where, causal=True, selected=selected)
        return {"selected": selected, "o": o, "lse": lse}
    if c["op"] == "append":
        return {"q": _append(s), **_cache_out(s)}
    if c["op"] == "attend":
        o, lse = _attend(s)
        return {"o": o, "lse": lse}
    selected = _select(s)
    o, lse = _attend_selected(s, selected)
    return {"selected": selected, "o": o, "lse": lse}


# ---------------------------------------------------------------- 64 bits

def _decode64(codes):
    """Values of e4m3 codes from their bit fields, in 64 bits."""
    c = codes.to(torch.int64)
    e, m = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e == 0, m * 2.0 ** -9, (8.0 + m) * torch.exp2((e - 10).double()))
    return torch.where(c >= 128, -mag, mag)


def _nearest64(x):
    """x rounded to the nearest e4m3 value, ties to even, saturated."""
    e = torch.frexp(x)[1].clamp(min=-5) - 1
    step = torch.exp2((e - 3).double())
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _exact_append(case, s):
    lens, news = _lengths(case)
    ps, d, rd = case["page"], case["d"], case["rope_dim"]
    codes = {n: _decode64(s[n]) for n in ("k", "v")}
    scales = {n: s[n + "_scale"].double() for n in ("k", "v")}
    q_out, row = [], 0
    theta = 10000.0 ** (-torch.arange(rd // 2, dtype=torch.float64, device=s["q"].device) * 2 / max(rd, 1))

    def turned(x, p):
        x = x.double()
        if not rd:
            return x
        a = p[:, None, None] * theta
        y = x.clone()
        i = torch.arange(rd // 2, device=x.device)
        i0, i1 = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rd // 2)
        y[..., i0] = x[..., i0] * a.cos() - x[..., i1] * a.sin()
        y[..., i1] = x[..., i0] * a.sin() + x[..., i1] * a.cos()
        return y

    for b, (t, n) in enumerate(zip(lens, news)):
        p = torch.arange(t - n, t, device=s["q"].device).double()
        q_out.append(turned(s["q"][row: row + n], p))
        new = {"k": turned(s["k_new"][row: row + n], p), "v": s["v_new"][row: row + n].double()}
        for j in range((t - n) // ps, -(-t // ps)):
            at = int(s["page_table"][b, j])
            lo, hi = max(t - n, j * ps), min(t, j * ps + ps)
            for m in ("k", "v"):
                x = new[m][lo - (t - n): hi - (t - n)].transpose(0, 1)
                amax = x.abs().amax(dim=(1, 2))
                unit = torch.exp2(torch.ceil(torch.log2(amax / 448.0)).clamp(-48, 48))
                if lo > j * ps:
                    unit = torch.maximum(unit, scales[m][at])
                    kept = codes[m][at][:, : lo - j * ps] * (scales[m][at] / unit)[:, None, None]
                    codes[m][at][:, : lo - j * ps] = _nearest64(kept)
                codes[m][at][:, lo - j * ps: hi - j * ps] = _nearest64(x / unit[:, None, None])
                scales[m][at] = unit
        row += n
    return {"q": torch.cat(q_out), "k": codes["k"], "v": codes["v"], "k_scale": scales["k"], "v_scale": scales["v"],
            "k_bounds": None}


def _exact_rows(q, k, v, limit, scale):
    """Attention of q [rows, heads, d] over k, v [heads, keys, d]; row i sees the keys that limit [rows, keys] says."""
    x = torch.einsum("rhd,hkd->hrk", q, k) * scale
    x = x.masked_fill(~limit[None], -math.inf)
    lse = torch.logsumexp(x, dim=2)
    p = torch.exp(x - lse[..., None]).nan_to_num(nan=0.0)
    return torch.einsum("hrk,hkd->rhd", p, v), lse.t()


def exact(case, seed):
    if work(case)["flops"] > 1.5e12:
        return None
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(case, s)
    lens, news = _lengths(case)
    ps, g, kvh, d = case["page"], case["group"], case["kv_heads"], case["d"]
    outs, lses, row = [], [], 0
    chosen = _select(s) if case["op"] == "sparse" else None       # whole numbers: what is attended is part of the input here
    scale = 1.0 / math.sqrt(d)
    for b, (t, n) in enumerate(zip(lens, news)):
        if not n:
            continue
        held = s["page_table"][b, : -(-t // ps)].long()
        k, v = ((_decode64(s[m][held]) * s[m + "_scale"][held].double()[..., None, None]).transpose(0, 1).reshape(kvh, -1, d)[:, :t]
                for m in ("k", "v"))
        key = torch.arange(t, device=k.device)
        for i0 in range(0, n, 512):
            i = torch.arange(i0, min(n, i0 + 512), device=k.device)
            see = key[None, :] <= (t - n + i)[:, None]
            q = s["q"][row + i].double()
            os_, ls_ = [], []
            for h in range(kvh):
                seen = see
                if chosen is not None:
                    pick = torch.zeros(len(i), len(held) + 1, dtype=torch.bool, device=k.device)
                    pick.scatter_(1, torch.where(chosen[row + i, h] < 0, len(held), chosen[row + i, h]).long(), True)
                    seen = see & pick[:, key // ps]
                qh = q[:, h * g: (h + 1) * g]
                o, l = _exact_rows(qh, k[h: h + 1].expand(g, -1, -1), v[h: h + 1].expand(g, -1, -1), seen, scale)
                os_.append(o)
                ls_.append(l)
            outs.append(torch.cat(os_, dim=1))
            lses.append(torch.cat(ls_, dim=1))
        row += n
    out = {"o": torch.cat(outs), "lse": torch.cat(lses)}
    return {"selected": None, **out} if chosen is not None else out
