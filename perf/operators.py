"""Cases of the 4-bit key/value cache operators: block tables, cache rows, attention.

``run`` computes them in plain torch operations, or (``own``) through the
library's entry points.  A case is a dict of plain values; ``op`` names the
operator:

* ``tables``: ``kq_block_tables``, the pages, slots and lengths of one step;
* ``rows``: ``kq_kv_store`` of new key and value rows, then ``kq_kv_load`` of
  the same rows (what the 4-bit rows stand for);
* ``attn``: ``kq_kv_attention`` over cached rows, for single tokens and prompts.
"""

import math

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step of a batch: every request grows by one token
        {"name": "tables_decode_64", "op": "tables", "requests": 64, "page": 16, "width": 512, "max_ctx": 8000,
         "max_new": 1, "pad": 0},
        # a step that admits prompts beside running requests, in a padded token buffer
        {"name": "tables_mixed_500", "op": "tables", "requests": 500, "page": 64, "width": 160, "max_ctx": 9000,
         "max_new": 65, "pad": 77},
        # new rows of one decode step, 64 requests of 8 key/value heads
        {"name": "rows_decode_64", "op": "rows", "tokens": 64, "heads": 8, "d": 128, "page": 16, "dtype": "f16",
         "out": "f16", "packed": True, "pad": 0},
        # rows of a long prompt in bfloat16, slices of a fused projection
        {"name": "rows_prompt_8192", "op": "rows", "tokens": 8192, "heads": 8, "d": 128, "page": 64, "dtype": "bf16",
         "out": "bf16", "packed": True, "pad": 0},
        # odd counts, float32 rows, a padded tail, a head size that is no power of two
        {"name": "rows_odd_1031_d96", "op": "rows", "tokens": 1031, "heads": 5, "d": 96, "page": 32, "dtype": "f32",
         "out": "f32", "packed": False, "pad": 6},
        # one short chat: the smallest call, where latency counts
        {"name": "attn_decode_1x330", "op": "attn", "requests": 1, "q_heads": 32, "kv_heads": 8, "d": 128,
         "page": 16, "min_len": 330, "max_len": 330, "min_new": 1, "max_new": 1, "window": 0, "dtype": "f16",
         "packed": True, "empty": 0},
        # a serving batch of ragged lengths
        {"name": "attn_decode_64x8k", "op": "attn", "requests": 64, "q_heads": 32, "kv_heads": 8, "d": 128,
         "page": 64, "min_len": 200, "max_len": 8192, "min_new": 1, "max_new": 1, "window": 0, "dtype": "f16",
         "packed": True, "empty": 0},
        # long documents: few rows over a long axis
        {"name": "attn_decode_4x128k", "op": "attn", "requests": 4, "q_heads": 32, "kv_heads": 8, "d": 128,
         "page": 256, "min_len": 120000, "max_len": 131072, "min_new": 1, "max_new": 1, "window": 0, "dtype": "bf16",
         "packed": True, "empty": 0},
        # no shared heads, head size 64, a sliding window, an idle slot of the batch
        {"name": "attn_decode_19_mha_d64_window", "op": "attn", "requests": 19, "q_heads": 16, "kv_heads": 16, "d": 64,
         "page": 32, "min_len": 1, "max_len": 5000, "min_new": 1, "max_new": 1, "window": 1000, "dtype": "bf16",
         "packed": False, "empty": 1},
        # a prompt from its first token
        {"name": "attn_prompt_4096", "op": "attn", "requests": 1, "q_heads": 32, "kv_heads": 8, "d": 128,
         "page": 64, "min_len": 4096, "max_len": 4096, "min_new": 4096, "max_new": 4096, "window": 0, "dtype": "f16",
         "packed": True, "empty": 0},
        # chunks of several prompts on top of cached tokens, single tokens among them
        {"name": "attn_chunks_9_mixed", "op": "attn", "requests": 9, "q_heads": 32, "kv_heads": 8, "d": 128,
         "page": 16, "min_len": 100, "max_len": 9000, "min_new": 1, "max_new": 700, "window": 0, "dtype": "bf16",
         "packed": True, "empty": 1},
        # a wide head with a sliding window, odd length
        {"name": "attn_prompt_1777_d256_window", "op": "attn", "requests": 1, "q_heads": 16, "kv_heads": 4, "d": 256,
         "page": 64, "min_len": 1777, "max_len": 1777, "min_new": 1777, "max_new": 1777, "window": 1024,
         "dtype": "f16", "packed": False, "empty": 0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["tables", "rows", "rows", "attn", "attn", "attn", "attn"])
    if kind == "tables":
        page = rng.choice([16, 32, 64, 128, 256])
        ctx = _log_int(rng, 100, 9000)
        new = rng.choice([1, 1, _log_int(rng, 2, 65)])
        return {"op": "tables", "requests": _log_int(rng, 1, 500), "page": page, "max_ctx": ctx, "max_new": new,
                "width": (ctx + new + page - 1) // page + rng.randrange(9), "pad": rng.choice([0, rng.randrange(100)])}
    if kind == "rows":
        tokens = _log_int(rng, 1, 8000)
        return {"op": "rows", "tokens": tokens, "heads": rng.randint(1, 8), "d": rng.choice([64, 96, 128]),
                "page": rng.choice([16, 32, 64, 128, 256]), "dtype": rng.choice(["f16", "bf16", "f32"]),
                "out": rng.choice(["f16", "bf16", "f32"]), "packed": rng.random() < 0.5,
                "pad": min(tokens - 1, rng.choice([0, 0, 3, 50]))}
    kv, group = rng.choice([(8, 4), (8, 1), (4, 8), (2, 7), (16, 1), (1, 16), (5, 3)])
    case = {"op": "attn", "q_heads": kv * group, "kv_heads": kv, "d": rng.choice([64, 64, 96, 128, 128, 128, 256]),
            "page": rng.choice([16, 32, 64, 128, 256]), "dtype": rng.choice(["f16", "bf16"]),
            "window": rng.choice([0, 0, 0, _log_int(rng, 64, 4000)]), "packed": rng.random() < 0.5}
    if rng.random() < 0.6:  # single tokens (or a few, as a verified draft has)
        n = _log_int(rng, 1, 64)
        hi = _log_int(rng, 16, max(64, min(100000, 400000 // n)))
        new = rng.choice([1, 1, 1, rng.randint(2, 6)])
        case.update(requests=n, min_len=max(new, hi // rng.choice([1, 2, 30])), max_len=max(new, hi), min_new=1,
                    max_new=new, empty=rng.choice([0, 0, 1]) if n > 1 else 0)
    else:  # prompts, or chunks of them
        n = _log_int(rng, 1, 8)
        new = _log_int(rng, 20, 2048 // n)
        ctx = rng.choice([0, _log_int(rng, 10, 3000)])
        case.update(requests=n, min_len=new, max_len=new + ctx, min_new=max(1, new // rng.choice([1, 3])), max_new=new,
                    empty=rng.choice([0, 0, 1]) if n > 1 else 0)
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed, device="cpu"):
    return torch.Generator(device=device).manual_seed(1000003 * (seed % 1000000) + 17)


def _ints(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g)


def _mix(case):
    """A generator of the case's own: its requests' lengths are the case's, their order and all values the seed's."""
    return _gen(sum((i + 1) * v for i, v in enumerate(case.values()) if type(v) is int))


def _tables_lengths(case):
    """Tokens held and tokens added of each request."""
    g, n = _mix(case), case["requests"]
    ctx, new = _ints(g, 0, case["max_ctx"], n), _ints(g, 1, case["max_new"], n)
    new[torch.rand(n, generator=g) < 0.03] = 0  # a few requests pause this step
    return ctx, new


def _attn_lengths(case):
    """New tokens and length (new ones included) of each request."""
    g, n = _mix(case), case["requests"]
    new = _ints(g, case["min_new"], case["max_new"], n)
    new[0] = case["max_new"]
    lens = torch.maximum(_ints(g, case["min_len"], case["max_len"], n), new)
    lens[0] = max(case["max_len"], case["max_new"])
    if case["empty"]:  # an idle slot of the batch: a row of queries with nothing to attend
        lens[-1] = 0
    return new, lens


def _dev(t):
    return t.to(dtype=torch.int32, device="cuda")


def _page_bytes(page, d):
    return page * (d // 2 + d // 16)


def _quantize(x):
    """float32 [..., 32 n] -> codes (int32, 0..15) [..., n, 32] and float16 scales [..., n] of q4_0 blocks."""
    x = torch.nan_to_num(x, nan=0.0, posinf=65504.0, neginf=-65504.0).clamp(-65504.0, 65504.0)
    x = x.unflatten(-1, (-1, 32))
    d = (x.abs().amax(-1).double() / 7).float().clamp(max=8188.0).half()
    df = d.float().unsqueeze(-1)
    q = torch.round(torch.where(df > 0, x / df, torch.zeros_like(x))).clamp(-8, 7)
    r = x - q * df  # exact: both terms have few bits and lie within a factor of each other
    q = torch.where(r > df / 2, q + 1, q)
    q = torch.where((r < -df / 2) | ((r == -df / 2) & (df > 0)), q - 1, q)
    return (q.clamp(-8, 7) + 8).int(), d


def _pack(codes, d, cache, page, dim, slots):
    """Rows' codes [rows, heads, n, 32] and scales [rows, heads, n] into the cache's slots."""
    pages, heads = cache.shape[:2]
    c = codes.flatten(-2)
    by = (c[..., 0::2] | (c[..., 1::2] << 4)).to(torch.uint8)
    codes_view = cache[:, :, :page * dim // 2].unflatten(-1, (page, dim // 2))
    scale_view = cache[:, :, page * dim // 2:].unflatten(-1, (page, dim // 16))
    pg, off = slots // page, slots % page
    codes_view[pg, :, off] = by
    scale_view[pg, :, off] = d.contiguous().view(torch.uint8).reshape(d.shape[0], heads, dim // 16)


def _unpack(cache, page, dim, pages=None):
    """float32 values [pages, heads, page, dim] of (the chosen pages of) the cache."""
    c = cache if pages is None else cache[pages]
    codes = c[:, :, :page * dim // 2].unflatten(-1, (page, dim // 2))
    q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float() - 8
    d = c[:, :, page * dim // 2:].contiguous().view(torch.float16).unflatten(-1, (page, dim // 32)).float()
    return (q.unflatten(-1, (-1, 32)) * d.unsqueeze(-1)).flatten(-2)


def _rows(g, shape, spread=True):
    """Rows as projections give them: normal, some channels larger than others."""
    x = torch.randn(shape, generator=g, device="cuda")
    if spread:
        x *= 0.5 + 1.5 * torch.rand(shape[-1], generator=g, device="cuda")
    return x


def _prepare_tables(case, seed):
    g = _gen(seed)
    n, page, width = case["requests"], case["page"], case["width"]
    order = torch.randperm(n, generator=g)
    ctx, new = (t[order] for t in _tables_lengths(case))
    held = -(-ctx // page)
    pool = int(held.sum())
    need = int((-(-(ctx + new) // page) - held).sum())
    ids = torch.randperm(pool + need + 40, generator=g)
    table = torch.full((n, width), -1, dtype=torch.int64)
    at = 0
    for s in range(n):
        table[s, :held[s]] = ids[at:at + int(held[s])]
        at += int(held[s])
    used = int(_ints(g, 0, 5, 1))
    free = torch.cat((torch.zeros(used, dtype=torch.int64), ids[at:]))
    tokens = int(new.sum()) + case["pad"]
    e = lambda *shape: torch.empty(shape, dtype=torch.int32, device="cuda")
    return {"case": case, "ctx": _dev(ctx), "new": _dev(new), "free": _dev(free),
            "head": torch.tensor([used], dtype=torch.int32, device="cuda"), "table": _dev(table),
            "slots": e(tokens), "cu": e(n + 1), "lens": e(n), "head_out": e(1), "status": e(1)}


def _prepare_rows(case, seed):
    g, gd = _gen(seed), _gen(seed, "cuda")
    n, heads, d, page = case["tokens"], case["heads"], case["d"], case["page"]
    dt, od = DT[case["dtype"]], DT[case["out"]]
    if case["packed"]:  # slices of a fused query/key/value projection with twice as many query heads
        qkv = _rows(gd, (n, 4 * heads, d)).to(dt)
        k, v = qkv[:, 2 * heads:3 * heads], qkv[:, 3 * heads:]
    else:
        k, v = _rows(gd, (n, heads, d)).to(dt), _rows(gd, (n, heads, d)).to(dt)
    pages = (n + page - 1) // page + 3
    perm = torch.randperm(pages, generator=g)
    pos = torch.arange(n) + page // 2
    slots = perm[pos // page] * page + pos % page  # a prompt that starts inside a page
    if case["pad"]:
        slots[-case["pad"]:] = -1
    pb = _page_bytes(page, d)
    zeros = lambda: torch.zeros((pages, heads, pb), dtype=torch.uint8, device="cuda")
    out = lambda: torch.zeros((n, heads, d), dtype=od, device="cuda")
    return {"case": case, "k": k, "v": v, "slots": _dev(slots), "k_cache": zeros(), "v_cache": zeros(),
            "k_out": out(), "v_out": out()}


def _prepare_attn(case, seed):
    g, gd = _gen(seed), _gen(seed, "cuda")
    n, page, d, kv, hq = case["requests"], case["page"], case["d"], case["kv_heads"], case["q_heads"]
    order = torch.randperm(n, generator=g)
    new, lens = (t[order] for t in _attn_lengths(case))
    tokens = int(new.sum())
    cu = torch.cat((torch.zeros(1, dtype=torch.int64), new.cumsum(0)))
    width = -(-int(lens.max()) // page)
    held = -(-lens // page)
    pages = int(held.sum()) + 5
    perm = torch.randperm(pages, generator=g)
    table = torch.full((n, width), -1, dtype=torch.int64)
    at = 0
    for s in range(n):
        table[s, :held[s]] = perm[at:at + int(held[s])]
        at += int(held[s])
    caches = []
    for _ in range(2):
        cache = torch.empty((pages, kv, _page_bytes(page, d)), dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 26) // (kv * page * d))
        channels = 0.5 + 1.5 * torch.rand(d, generator=gd, device="cuda")
        for p in range(0, pages, step):
            c = min(step, pages - p)
            codes, sc = _quantize(torch.randn((c, kv, page, d), generator=gd, device="cuda") * channels)
            codes = codes.flatten(-2)
            cache[p:p + c, :, :page * d // 2] = (codes[..., 0::2] | (codes[..., 1::2] << 4)).to(torch.uint8).flatten(2)
            cache[p:p + c, :, page * d // 2:] = sc.contiguous().view(torch.uint8).reshape(c, kv, -1)
        caches.append(cache)
    heads = hq + 2 * kv if case["packed"] else hq
    q = _rows(gd, (tokens, heads, d), False).to(DT[case["dtype"]])[:, :hq]
    state = {"case": case, "q": q, "cu": _dev(cu), "lens": _dev(lens), "table": _dev(table), "k_cache": caches[0],
             "v_cache": caches[1], "out": torch.empty((tokens, hq, d), dtype=q.dtype, device="cuda"),
             "scale": d ** -0.5, "max_new": int(new.max()), "max_kv": max(1, int(lens.max())),
             "host_cu": cu.tolist(), "host_lens": lens.tolist()}
    if own:  # the scratch memory that a serving program keeps from step to step
        from gguf_quant_matmul_amd import kq

        need = kq.kq_kv_attention_workspace(tokens, n, hq, kv, d, state["max_new"], state["max_kv"])
        state["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    return state


def prepare(case, seed):
    return {"tables": _prepare_tables, "rows": _prepare_rows, "attn": _prepare_attn}[case["op"]](case, seed)


# ---------------------------------------------------------------------------
# the operators
# ---------------------------------------------------------------------------

def _own(st):
    from gguf_quant_matmul_amd import kq

    case = st["case"]
    if case["op"] == "tables":
        kq.kq_block_tables(st["ctx"], st["new"], st["free"], st["head"], case["page"], st["table"], st["slots"],
                           st["cu"], st["lens"], st["head_out"], st["status"])
        return st["table"], st["slots"], st["cu"], st["lens"], st["head_out"], st["status"]
    if case["op"] == "rows":
        kq.kq_kv_store("q4_0", st["k"], st["v"], st["slots"], st["k_cache"], st["v_cache"], case["page"])
        kq.kq_kv_load("q4_0", st["k_cache"], st["v_cache"], st["slots"], case["page"], st["k_out"], st["v_out"])
        return st["k_out"], st["v_out"]
    kq.kq_kv_attention("q4_0", st["q"], st["cu"], st["lens"], st["table"], st["k_cache"], st["v_cache"], case["page"],
                       st["out"], scale=st["scale"], window=case["window"], max_new=st["max_new"],
                       max_kv=st["max_kv"], workspace=st["workspace"])
    return st["out"]


def _plain_tables(st):
    page = st["case"]["page"]
    ctx, new, table = st["ctx"].long(), st["new"].long(), st["table"]
    n, width = table.shape
    tokens = st["slots"].numel()
    head = st["head"].long()
    ends = new.cumsum(0)
    held, total = (ctx + page - 1) // page, (ctx + new + page - 1) // page
    wide, late = total > width, ends > tokens
    valid = ~(wide | late)
    need = torch.where(valid, total - held, 0)
    cum = need.cumsum(0)
    fit = valid & ((need == 0) | (cum <= st["free"].numel() - head))
    taken = torch.where(fit & (need > 0), cum, 0).max()
    # every new page of every request: its column in the request's table row, its place in the free list
    col = torch.arange(width, device="cuda").unsqueeze(0)
    fresh = fit.unsqueeze(1) & (col >= held.unsqueeze(1)) & (col < total.unsqueeze(1))
    place = head + (cum - need).unsqueeze(1) + col - held.unsqueeze(1)
    ids = st["free"][place.clamp(0, st["free"].numel() - 1)]
    table.copy_(torch.where(fresh, ids, table))
    t = torch.arange(tokens, device="cuda")
    s = torch.searchsorted(ends, t, right=True).clamp(max=n - 1)
    pos = ctx[s] + t - (ends - new)[s]
    pid = table[s, (pos // page).clamp(0, width - 1)].long()
    live = (t < ends[-1]) & fit[s] & (pid >= 0)
    slots = torch.where(live, pid * page + pos % page, -1).int()
    cu = torch.cat((torch.zeros(1, dtype=torch.long, device="cuda"), ends)).clamp(max=tokens).int()
    lens = torch.where(fit, ctx + new, 0).int()
    status = (valid & ~fit).any().int() + 2 * wide.any().int() + 4 * late.any().int()
    return table, slots, cu, lens, (head + taken).int(), status.reshape(1).int()


def _plain_rows(st):
    case = st["case"]
    page, d = case["page"], case["d"]
    live = st["slots"] >= 0
    slots = st["slots"][live].long()
    for x, cache, out in ((st["k"], st["k_cache"], st["k_out"]), (st["v"], st["v_cache"], st["v_out"])):
        codes, sc = _quantize(x[live].float())
        _pack(codes, sc, cache, page, d, slots)
        codes_view = cache[:, :, :page * d // 2].unflatten(-1, (page, d // 2))
        scale_view = cache[:, :, page * d // 2:].unflatten(-1, (page, d // 16))
        by = codes_view[slots // page, :, slots % page]
        q = torch.stack((by & 15, by >> 4), -1).flatten(-2).float() - 8
        f = scale_view[slots // page, :, slots % page].contiguous().view(torch.float16).float()
        out[live] = (q.unflatten(-1, (-1, 32)) * f.unsqueeze(-1)).flatten(-2).to(out.dtype)
    return st["k_out"], st["v_out"]


def _plain_attn(st):
    case = st["case"]
    page, d, kv, hq = case["page"], case["d"], case["kv_heads"], case["q_heads"]
    group = hq // kv
    out = st["out"]
    for s, length in enumerate(st["host_lens"]):
        a, b = st["host_cu"][s], st["host_cu"][s + 1]
        if length == 0:
            out[a:b] = 0
            continue
        pages = st["table"][s, :(length + page - 1) // page].long()
        k = _unpack(st["k_cache"], page, d, pages).transpose(0, 1).flatten(1, 2)[:, :length]
        v = _unpack(st["v_cache"], page, d, pages).transpose(0, 1).flatten(1, 2)[:, :length]
        kt = k.transpose(1, 2).contiguous()
        keys = torch.arange(length, device="cuda")
        for t in range(a, b, 1024):
            e = min(b, t + 1024)
            q = st["q"][t:e].float().unflatten(1, (kv, group)).permute(1, 2, 0, 3).reshape(kv, group * (e - t), d)
            w = torch.matmul(q, kt).unflatten(1, (group, e - t)) * st["scale"]
            p = torch.arange(t - b + length, e - b + length, device="cuda").unsqueeze(1)
            seen = keys <= p
            if case["window"]:
                seen &= keys > p - case["window"]
            w = torch.where(seen, w, -torch.inf)
            w = torch.exp(w - w.amax(-1, keepdim=True))
            w = w / w.sum(-1, keepdim=True)
            o = torch.matmul(w.flatten(1, 2), v).unflatten(1, (group, e - t))
            out[t:e] = o.permute(2, 0, 1, 3).flatten(1, 2).to(out.dtype)
    return out


def run(state):
    if own:
        return _own(state)
    return {"tables": _plain_tables, "rows": _plain_rows, "attn": _plain_attn}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without, and its result in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "tables":
        ctx, new = _tables_lengths(case)
        n, page, tokens = case["requests"], case["page"], int(new.sum())
        pages = int(((ctx + new + page - 1) // page - (ctx + page - 1) // page).sum())
        # lengths in; slots, offsets and lengths out; new pages' ids read and written; the last held page's id read
        return {"bytes": 8 * n + 4 * (tokens + case["pad"]) + 8 * n + 8 * pages + 4 * n, "flops": 0}
    size = {"f16": 2, "bf16": 2, "f32": 4}
    if case["op"] == "rows":
        values = 2 * (case["tokens"] - case["pad"]) * case["heads"] * case["d"]
        # rows in, the cache's bytes, rows out
        return {"bytes": int(values * (size[case["dtype"]] + 9 / 16 + size[case["out"]])), "flops": 0}
    keys = pairs = 0
    new, lens = (t.tolist() for t in _attn_lengths(case))
    window = case["window"] or 1 << 40
    for m, length in zip(new, lens):
        if length:
            keys += min(length, window + m - 1)  # keys that some query of the request sees
            full = max(0, min(m, length - window))  # queries that see a whole window
            pairs += full * window + sum(range(length - m + 1, length - full + 1))
    q = 2 * sum(new) * case["q_heads"] * case["d"]
    return {"bytes": int(keys * case["kv_heads"] * case["d"] * 9 / 8 + 2 * q),
            "flops": 4 * case["d"] * case["q_heads"] * pairs}


def _exact_tables(st):
    page = st["case"]["page"]
    ctx, new = st["ctx"].tolist(), st["new"].tolist()
    free, head = st["free"].tolist(), st["head"].item()
    table = st["table"].tolist()
    width, room = len(table[0]), st["slots"].numel()
    slots, cu, lens, status, at, asked = [], [0], [], 0, 0, 0
    for s, (c, m) in enumerate(zip(ctx, new)):
        at += m
        cu.append(min(at, room))
        held, total = math.ceil(c / page), math.ceil((c + m) / page)
        ok = True
        if total > width:
            ok, status = False, status | 2
        if at > room:
            ok, status = False, status | 4
        if ok and total > held:
            asked += total - held
            if asked > len(free) - st["head"].item():
                ok, status = False, status | 1
            else:
                table[s][held:total] = free[st["head"].item() + asked - (total - held):st["head"].item() + asked]
                head = st["head"].item() + asked
        lens.append(c + m if ok else 0)
        for i in range(m):
            if len(slots) < room:
                slots.append(table[s][(c + i) // page] * page + (c + i) % page if ok else -1)
    slots += [-1] * (room - len(slots))
    t = lambda a: torch.tensor(a, dtype=torch.int32)
    return t(table), t(slots), t(cu), t(lens), t([head]), t([status])


def _exact_rows(st):
    live = (st["slots"] >= 0).cpu()
    res = []
    for x in (st["k"], st["v"]):
        x = x.cpu().double()
        blocks = x.reshape(x.shape[0], x.shape[1], -1, 32).clamp(-65504, 65504)
        # the scale is what 16 bits hold of the float32 quotient
        d = (blocks.abs().max(-1, keepdim=True).values / 7).to(torch.float32).clamp(max=8188).to(torch.float16).double()
        best = torch.full_like(blocks, -8) * d
        for code in range(-7, 8):  # the nearest of the sixteen values; the lower of two at the same distance
            here = code * d
            best = torch.where((blocks - here).abs() < (blocks - best).abs(), here, best)
        best = torch.where(d > 0, best, torch.zeros_like(best))
        best = best.reshape(x.shape)
        best[~live] = 0
        res.append(best)
    return tuple(res)


def _exact_attn(st):
    case = st["case"]
    page, d, kv, hq = case["page"], case["d"], case["kv_heads"], case["q_heads"]
    group = hq // kv
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    codes_at = page * d // 2

    def values(cache, ids, h):
        raw = cache[ids, h]
        by = raw[:, :codes_at].reshape(-1, d // 2)
        row = torch.empty((by.shape[0], d), dtype=torch.float64, device="cuda")
        row[:, 0::2] = (by % 16).double() - 8
        row[:, 1::2] = (by // 16).double() - 8
        d16 = raw[:, codes_at:].contiguous().view(torch.float16).reshape(-1, d // 32).double()
        return row * d16.repeat_interleave(32, 1)

    for s, length in enumerate(st["host_lens"]):
        a, b = st["host_cu"][s], st["host_cu"][s + 1]
        if length == 0:
            continue
        ids = st["table"][s, :math.ceil(length / page)].long()
        place = torch.arange(length, device="cuda")
        for h in range(kv):
            k, v = values(st["k_cache"], ids, h)[:length], values(st["v_cache"], ids, h)[:length]
            for j in range(group):
                for t in range(a, b, 2048):
                    e = min(b, t + 2048)
                    logits = st["q"][t:e, h * group + j].double() @ k.T * st["scale"]
                    pos = (length - b + torch.arange(t, e, device="cuda"))[:, None]
                    hidden = place[None, :] > pos
                    if case["window"]:
                        hidden |= place[None, :] <= pos - case["window"]
                    logits.masked_fill_(hidden, -math.inf)
                    out[t:e, h * group + j] = torch.softmax(logits, -1) @ v
    return out


def exact(case, seed):
    st = prepare(case, seed)
    return {"tables": _exact_tables, "rows": _exact_rows, "attn": _exact_attn}[case["op"]](st)
