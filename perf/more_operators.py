"""Cases of the serving step's operators around the paged key/value cache: rotary positions, pages shared and moved,
attention with sinks, attention over a shared prefix.

``run`` computes them in plain torch operations, or (``own``) through the library's entry points.  A case is a dict of
plain values; ``op`` names the operator:

* ``rope``: ``kq_rope``, the queries and keys of one step rotated to their positions;
* ``fork``: ``kq_kv_fork`` of requests, then ``kq_kv_copy_pages`` of the pages that their lengths end in;
* ``free``: ``kq_kv_free``, pages given back by requests that end or whose window moved on;
* ``compact``: ``kq_kv_compact`` and ``kq_kv_copy_pages``, the held pages brought to the front of the cache;
* ``sinks``: ``kq_kv_attention_sinks``, a sliding window beside a few first tokens that stay visible;
* ``prefix``: ``kq_kv_attention_prefix``, requests that share their first pages.
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
        # one decode step of a batch, every head rotated whole, a context stretched eightfold
        {"name": "rope_decode_64", "op": "rope", "requests": 64, "q_heads": 32, "kv_heads": 8, "d": 128, "rot": 128,
         "layout": "half", "scaling": "yarn", "factor": 8.0, "base": 500000.0, "max_ctx": 60000, "min_new": 1,
         "max_new": 1, "pad": 0, "dtype": "f16", "packed": True},
        # chunks of three prompts, half of each head rotated in pairs, a padded tail
        {"name": "rope_chunks_3x2700_pairs", "op": "rope", "requests": 3, "q_heads": 32, "kv_heads": 8, "d": 128,
         "rot": 64, "layout": "pairs", "scaling": "none", "factor": 1.0, "base": 10000.0, "max_ctx": 4000,
         "min_new": 2500, "max_new": 2731, "pad": 5, "dtype": "bf16", "packed": True},
        # eight samples of one chat
        {"name": "fork_8_of_1", "op": "fork", "parents": 1, "forks": 8, "page": 16, "kv_heads": 8, "d": 128,
         "min_len": 330, "max_len": 330, "whole": True},
        # a beam step of a batch: requests continue from places of others
        {"name": "fork_256_of_64", "op": "fork", "parents": 64, "forks": 256, "page": 64, "kv_heads": 8, "d": 128,
         "min_len": 100, "max_len": 8000, "whole": False},
        # requests of a batch that end, others whose window moved past a page
        {"name": "free_5_of_64", "op": "free", "requests": 64, "ending": 5, "page": 16, "max_len": 8000, "shared": 20,
         "sliding": True},
        # a batch that ends as a whole, half of it on a shared prefix
        {"name": "free_500_of_500", "op": "free", "requests": 500, "ending": 500, "page": 64, "max_len": 9000,
         "shared": 31, "sliding": False},
        # a small cache a fifth of whose pages are free
        {"name": "compact_500", "op": "compact", "pages": 500, "held": 0.8, "requests": 7, "page": 16, "kv_heads": 2,
         "d": 64},
        # a large one, a third free
        {"name": "compact_12000", "op": "compact", "pages": 12000, "held": 0.67, "requests": 120, "page": 64,
         "kv_heads": 8, "d": 128},
        # a decode step of long chats that keep their first tokens and a window
        {"name": "sinks_decode_64", "op": "sinks", "requests": 64, "q_heads": 32, "kv_heads": 8, "d": 128, "page": 64,
         "min_len": 200, "max_len": 30000, "min_new": 1, "max_new": 1, "window": 2000, "sinks": 4, "dtype": "f16",
         "packed": True, "empty": 1},
        # a prompt from its first token
        {"name": "sinks_prompt_4096", "op": "sinks", "requests": 1, "q_heads": 32, "kv_heads": 8, "d": 128, "page": 16,
         "min_len": 4096, "max_len": 4096, "min_new": 4096, "max_new": 4096, "window": 1024, "sinks": 4,
         "dtype": "bf16", "packed": True, "empty": 0},
        # drafts of up to five tokens on a short instruction, no shared heads, an idle slot
        {"name": "prefix_drafts_6x1000_mha_d64", "op": "prefix", "requests": 6, "q_heads": 16, "kv_heads": 16, "d": 64,
         "page": 16, "prefix": 1008, "max_own": 300, "min_new": 1, "max_new": 5, "dtype": "bf16", "packed": False,
         "empty": 1},
        # a batch of questions about one long document
        {"name": "prefix_decode_64x16k", "op": "prefix", "requests": 64, "q_heads": 32, "kv_heads": 8, "d": 128,
         "page": 64, "prefix": 16384, "max_own": 900, "min_new": 1, "max_new": 1, "dtype": "f16", "packed": True,
         "empty": 0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "fork", "free", "compact", "sinks", "sinks", "prefix", "prefix", "prefix"])
    page = rng.choice([16, 32, 64, 128, 256])
    kv, group = rng.choice([(8, 4), (8, 1), (4, 8), (2, 7), (16, 1), (1, 16), (5, 3)])
    if op == "rope":
        d = rng.choice([64, 96, 128, 128, 256])
        n = _log_int(rng, 1, 64)
        new = rng.choice([1, 1, _log_int(rng, 2, max(3, min(4000, 8000 * 40 * 128 // (n * kv * (group + 1) * d))))])
        return {"op": "rope", "requests": n, "q_heads": kv * group, "kv_heads": kv, "d": d,
                "rot": rng.choice([d, d, d // 2, d // 4]), "layout": rng.choice(["half", "pairs"]),
                "scaling": rng.choice(["none", "linear", "yarn"]), "factor": rng.choice([2.0, 4.0, 16.0]),
                "base": rng.choice([10000.0, 500000.0, 1000000.0]), "max_ctx": _log_int(rng, 1, 120000),
                "min_new": max(1, new // rng.choice([1, 2, 5])), "max_new": new, "pad": rng.choice([0, 0, 3, 50]),
                "dtype": rng.choice(["f16", "bf16", "f32"]), "packed": rng.random() < 0.5}
    if op == "fork":
        parents = _log_int(rng, 1, 64)
        hi = _log_int(rng, 20, 8000)
        return {"op": "fork", "parents": parents, "forks": _log_int(rng, 1, 256), "page": page, "kv_heads": kv,
                "d": rng.choice([64, 96, 128]), "min_len": max(1, hi // rng.choice([1, 4, 40])), "max_len": hi,
                "whole": rng.random() < 0.5}
    if op == "free":
        n = _log_int(rng, 1, 500)
        return {"op": "free", "requests": n, "ending": rng.choice([n, rng.randint(1, n)]), "page": page,
                "max_len": _log_int(rng, 50, 9000), "shared": rng.choice([0, rng.randint(1, 40)]),
                "sliding": rng.random() < 0.5}
    if op == "compact":
        d = rng.choice([64, 96, 128])
        return {"op": "compact", "pages": _log_int(rng, 50, min(200000, 12000 * 64 * 8 * 128 // (page * kv * d))),
                "held": rng.choice([0.3, 0.6, 0.9, 0.97]), "requests": _log_int(rng, 1, 300), "page": page,
                "kv_heads": kv, "d": d}
    d = rng.choice([64, 64, 96, 128, 128, 128, 256])
    case = {"op": op, "q_heads": kv * group, "kv_heads": kv, "d": d, "page": page, "dtype": rng.choice(["f16", "bf16"]),
            "packed": rng.random() < 0.5}
    if op == "sinks":
        case.update(window=_log_int(rng, 60, 2000), sinks=rng.choice([1, 4, 4, 16, 70, 200]))
        if rng.random() < 0.6:  # single tokens, or a few
            n = _log_int(rng, 1, 64)
            hi = _log_int(rng, 16, 30000)
            new = rng.choice([1, 1, 1, rng.randint(2, 6)])
            lo = max(new, hi // rng.choice([1, 2, 30]))
            case.update(requests=n, min_len=lo, max_len=max(lo, hi), min_new=1, max_new=new)
        else:
            n = _log_int(rng, 1, 8)
            new = _log_int(rng, 20, 2048 // n)
            case.update(requests=n, min_len=new, max_len=new + rng.choice([0, _log_int(rng, 10, 4000)]),
                        min_new=max(1, new // rng.choice([1, 3])), max_new=new)
    else:
        n = _log_int(rng, 1, 64)
        length = _log_int(rng, 256, 16384)
        new = rng.choice([1, 1, 1, rng.randint(2, 6), max(1, 300 // n)])
        case.update(requests=n, prefix=length // page * page or page, max_own=_log_int(rng, new + 1, 900),
                    min_new=max(1, new // 2), max_new=new)
    case["empty"] = rng.choice([0, 0, 1]) if case["requests"] > 1 else 0
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed, device="cpu"):
    return torch.Generator(device=device).manual_seed(1000003 * (seed % 1000000) + 29)


def _mix(case):
    """A generator of the case's own: what sizes its work is the case's, orders and values are the seed's."""
    return _gen(sum((i + 1) * int(v) for i, v in enumerate(case.values()) if type(v) is int))


def _ints(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g)


def _dev(t):
    return t.to(dtype=torch.int32, device="cuda")


def _e(*shape):
    return torch.empty(shape, dtype=torch.int32, device="cuda")


def _page_bytes(case):
    return case["page"] * (case["d"] // 2 + case["d"] // 16)


def _lengths(case):
    """New tokens and length (new ones included) of each request of a rope, sinks or prefix case."""
    g, n = _mix(case), case["requests"]
    new = _ints(g, case["min_new"], case["max_new"], n)
    new[0] = case["max_new"]
    if case["op"] == "rope":
        return new, new + _ints(g, 0, case["max_ctx"], n)
    if case["op"] == "prefix":
        lens = case["prefix"] + torch.maximum(_ints(g, 1, case["max_own"], n), new)
    else:
        lens = torch.maximum(_ints(g, case["min_len"], case["max_len"], n), new)
        lens[0] = max(case["max_len"], case["max_new"])
    if case["empty"]:  # an idle slot of the batch: queries with nothing to attend
        lens[-1] = 0
    return new, lens


def _inv_freq(case):
    """Frequencies of the rotated pairs in float64, and the factor on the rotated values."""
    rot, base, factor = case["rot"], case["base"], case["factor"]
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if case["scaling"] == "linear":
        return f / factor, 1.0
    if case["scaling"] == "yarn":  # high frequencies as they are, low ones stretched, a ramp over the pairs between
        at = lambda turns: rot * math.log(8192 / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(0, math.floor(at(32))), min(rot - 1, math.ceil(at(1)))
        ramp = ((torch.arange(rot // 2, dtype=torch.float64) - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1
    return f, 1.0


def _starts(new):
    return torch.cat((torch.zeros(1, dtype=torch.int64), new.cumsum(0)))


def _prepare_rope(case, seed):
    g, gd = _gen(seed), _gen(seed, "cuda")
    order = torch.randperm(case["requests"], generator=g)
    new, lens = (t[order] for t in _lengths(case))
    hq, kv, d = case["q_heads"], case["kv_heads"], case["d"]
    tokens = int(new.sum()) + case["pad"]
    rows = lambda heads: torch.randn((tokens, heads, d), generator=gd, device="cuda").to(DT[case["dtype"]])
    if case["packed"]:  # slices of a fused query/key/value projection
        qkv = rows(hq + 2 * kv)
        q, k = qkv[:, :hq], qkv[:, hq:hq + kv]
    else:
        q, k = rows(hq), rows(kv)
    freq, mscale = _inv_freq(case)
    # (rows behind the last request stay zero)
    out = lambda heads: torch.zeros((tokens, heads, d), dtype=q.dtype, device="cuda")
    return {"case": case, "q": q, "k": k, "cu": _dev(_starts(new)), "lens": _dev(lens),
            "freq": freq.to(device="cuda", dtype=torch.float32), "mscale": mscale, "q_out": out(hq), "k_out": out(kv)}


def _fork_lengths(case):
    """Length of each parent, and how many of its tokens each fork takes."""
    g = _mix(case)
    lens = _ints(g, case["min_len"], case["max_len"], case["parents"])
    taken = lens[torch.arange(case["forks"]) % case["parents"]]
    if not case["whole"]:
        taken = (taken * torch.rand(case["forks"], generator=g)).long() + 1
    return lens, taken


def _bytes(case, pages, seed):
    g = _gen(seed + 3, "cuda")
    shape = (pages, case["kv_heads"], _page_bytes(case))
    return [torch.randint(0, 256, shape, dtype=torch.uint8, generator=g, device="cuda") for _ in range(2)]


def _prepare_fork(case, seed):
    g = _gen(seed)
    page, n, forks = case["page"], case["parents"], case["forks"]
    lens, taken = _fork_lengths(case)
    parent = torch.arange(forks) % n
    order = torch.randperm(forks, generator=g)
    parent, taken = parent[order], taken[order]
    held = -(-lens // page)
    pool = int(held.sum())
    pages = pool + forks + 20
    ids = torch.randperm(pages, generator=g)
    table = torch.full((n + forks, int(held.max()) + 2), -1, dtype=torch.int64)
    at = 0
    for s in range(n):
        table[s, :held[s]] = ids[at:at + int(held[s])]
        at += int(held[s])
    k_cache, v_cache = _bytes(case, pages, seed)
    return {"case": case, "parent": _dev(parent), "child": _dev(n + torch.randperm(forks, generator=g)),
            "take": _dev(taken), "table": _dev(table), "refs": torch.zeros(pages, dtype=torch.int32, device="cuda"),
            "free": _dev(ids), "head": _dev(torch.tensor([pool])), "src": _e(forks), "dst": _e(forks),
            "head_out": _e(1), "status": _e(1), "k_cache": k_cache, "v_cache": v_cache}


def _free_ranges(case):
    """Columns that each request holds, and those it gives back."""
    g, n = _mix(case), case["requests"]
    held = -(-_ints(g, 1, case["max_len"], n) // case["page"])
    first, last = torch.zeros(n, dtype=torch.int64), held.clone()
    slide = (held * torch.rand(n, generator=g)).long()  # the column that a running request's window has passed
    run = torch.arange(n) >= case["ending"]
    first[run] = slide[run]
    last[run] = slide[run] + (1 if case["sliding"] else 0)
    return held, first, last


def _prepare_free(case, seed):
    g, n = _gen(seed), case["requests"]
    order = torch.randperm(n, generator=g)
    held, first, last = (t[order] for t in _free_ranges(case))
    shares = (torch.arange(n)[order] % 2 == 0) & (held >= case["shared"]) & (case["shared"] > 0)
    need = int(held.sum() - shares.sum() * case["shared"]) + case["shared"]
    pages = need + 30
    ids = torch.randperm(pages, generator=g)
    common, at = ids[:case["shared"]], case["shared"]
    table = torch.full((n, int(held.max()) + 3), -1, dtype=torch.int64)
    for s in range(n):
        c = case["shared"] if shares[s] else 0
        table[s, :c] = common[:c]
        table[s, c:held[s]] = ids[at:at + int(held[s]) - c]
        at += int(held[s]) - c
    refs = torch.zeros(pages, dtype=torch.int64)
    refs[common] = (shares.sum() - 1).clamp(min=0)
    return {"case": case, "first": _dev(first), "last": _dev(last), "table": _dev(table), "refs": _dev(refs),
            "free": _dev(ids), "head": _dev(torch.tensor([at])), "head_out": _e(1), "status": _e(1)}


def _compact_held(case):
    """Which pages are held (the order of their ids is the case's, so that as many move whatever the seed)."""
    return torch.rand(case["pages"], generator=_mix(case)) < case["held"]


def _prepare_compact(case, seed):
    g, pages, n = _gen(seed), case["pages"], case["requests"]
    held = _compact_held(case)
    ids = held.nonzero().flatten()
    ids = ids[torch.randperm(len(ids), generator=g)]
    free = (~held).nonzero().flatten()
    free = torch.cat((ids, free[torch.randperm(len(free), generator=g)]))  # (what is in front of the head was taken)
    width = -(-len(ids) // n) + 2
    table = torch.full((n, width), -1, dtype=torch.int64)
    table.view(-1)[torch.randperm(n * width, generator=g)[:len(ids)]] = ids
    refs = torch.where(held & (torch.rand(pages, generator=g) < 0.1), _ints(g, 1, 9, pages), 0)
    k_cache, v_cache = _bytes(case, pages, seed)
    most = pages // 2
    return {"case": case, "free": _dev(free), "head": _dev(torch.tensor([len(ids)])), "table": _dev(table),
            "refs": _dev(refs), "table_out": _e(n, width), "refs_out": _e(pages), "free_out": _e(pages),
            "remap": _e(pages), "src": _e(most), "dst": _e(most), "head_out": _e(1), "status": _e(1),
            "k_cache": k_cache, "v_cache": v_cache}


def _caches(case, pages, gd):
    """Key and value rows as projections give them (some channels larger than others) in q4_0 blocks."""
    page, d, kv = case["page"], case["d"], case["kv_heads"]
    caches = []
    for _ in range(2):
        cache = torch.empty((pages, kv, _page_bytes(case)), dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 26) // (kv * page * d))
        channels = 0.5 + 1.5 * torch.rand(d, generator=gd, device="cuda")
        for p in range(0, pages, step):
            c = min(step, pages - p)
            x = torch.randn((c, kv, page, d), generator=gd, device="cuda") * channels
            x = x.unflatten(-1, (-1, 32))
            sc = (x.abs().amax(-1) / 7).half()
            codes = (torch.round(x / sc.float().unsqueeze(-1)).clamp(-8, 7) + 8).to(torch.uint8).flatten(-2)
            cache[p:p + c, :, :page * d // 2] = (codes[..., 0::2] | (codes[..., 1::2] << 4)).flatten(2)
            cache[p:p + c, :, page * d // 2:] = sc.contiguous().view(torch.uint8).reshape(c, kv, -1)
        caches.append(cache)
    return caches


def _prepare_attn(case, seed):
    g, gd = _gen(seed), _gen(seed, "cuda")
    n, page, d, kv, hq = case["requests"], case["page"], case["d"], case["kv_heads"], case["q_heads"]
    order = torch.randperm(n, generator=g)
    new, lens = (t[order] for t in _lengths(case))
    tokens = int(new.sum())
    shared = case.get("prefix", 0) // page
    held = -(-lens // page)
    common = torch.where(held > 0, shared, 0)
    pages = int((held - common).sum()) + shared + 5
    perm = torch.randperm(pages, generator=g)
    prefix, at = perm[:shared], shared
    table = torch.full((n, int(held.max())), -1, dtype=torch.int64)
    for s in range(n):
        c = int(common[s])
        table[s, :c] = prefix[:c]
        table[s, c:held[s]] = perm[at:at + int(held[s]) - c]
        at += int(held[s]) - c
    k_cache, v_cache = _caches(case, pages, gd)
    heads = hq + 2 * kv if case["packed"] else hq
    q = torch.randn((tokens, heads, d), generator=gd, device="cuda").to(DT[case["dtype"]])[:, :hq]
    state = {"case": case, "q": q, "cu": _dev(_starts(new)), "lens": _dev(lens), "table": _dev(table),
             "prefix": _dev(prefix), "k_cache": k_cache, "v_cache": v_cache, "scale": d ** -0.5,
             "out": torch.empty((tokens, hq, d), dtype=q.dtype, device="cuda"), "max_new": int(new.max()),
             "max_kv": max(1, int(lens.max())), "host_lens": lens.tolist()}
    if own:  # the scratch memory that a serving program keeps from step to step
        from gguf_quant_matmul_amd import kq

        sizes = tokens, n, hq, kv, d
        if case["op"] == "sinks":
            need = kq.kq_kv_attention_workspace(*sizes, state["max_new"], state["max_kv"])
        else:
            need = kq.kq_kv_attention_prefix_workspace(*sizes, case["prefix"], state["max_new"], state["max_kv"])
        state["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    return state


_PREPARE = {"rope": _prepare_rope, "fork": _prepare_fork, "free": _prepare_free, "compact": _prepare_compact,
            "sinks": _prepare_attn, "prefix": _prepare_attn}


def prepare(case, seed):
    return _PREPARE[case["op"]](case, seed)


# ---------------------------------------------------------------------------
# the operators through the library
# ---------------------------------------------------------------------------

def _own(st):
    from gguf_quant_matmul_amd import kq

    case = st["case"]
    op = case["op"]
    if op == "rope":
        kq.kq_rope(st["q"], st["k"], st["cu"], st["lens"], st["freq"], st["q_out"], st["k_out"], layout=case["layout"],
                   mscale=st["mscale"])
        return st["q_out"], st["k_out"]
    if op == "fork":
        kq.kq_kv_fork(st["parent"], st["child"], st["take"], case["page"], st["table"], st["refs"], st["free"],
                      st["head"], st["src"], st["dst"], st["head_out"], st["status"])
        kq.kq_kv_copy_pages(st["src"], st["dst"], st["k_cache"], st["v_cache"])
        return tuple(st[x] for x in ("table", "refs", "src", "dst", "head_out", "status", "k_cache", "v_cache"))
    if op == "free":
        kq.kq_kv_free(st["first"], st["last"], st["table"], st["refs"], st["free"], st["head"], st["head_out"],
                      st["status"])
        return st["refs"], st["free"], st["head_out"], st["status"]
    if op == "compact":
        kq.kq_kv_compact(st["free"], st["head"], st["table"], st["refs"], st["table_out"], st["refs_out"],
                         st["free_out"], st["remap"], st["src"], st["dst"], st["head_out"], st["status"])
        kq.kq_kv_copy_pages(st["src"], st["dst"], st["k_cache"], st["v_cache"])
        return tuple(st[x] for x in ("table_out", "refs_out", "free_out", "remap", "src", "dst", "head_out", "status",
                                     "k_cache", "v_cache"))
    if op == "sinks":
        kq.kq_kv_attention_sinks("q4_0", st["q"], st["cu"], st["lens"], st["table"], st["k_cache"], st["v_cache"],
                                 case["page"], st["out"], case["window"], case["sinks"], scale=st["scale"],
                                 max_new=st["max_new"], max_kv=st["max_kv"], workspace=st["workspace"])
    else:
        kq.kq_kv_attention_prefix("q4_0", st["q"], st["cu"], st["lens"], st["table"], st["prefix"], st["k_cache"],
                                  st["v_cache"], case["page"], st["out"], scale=st["scale"], max_new=st["max_new"],
                                  max_kv=st["max_kv"], workspace=st["workspace"])
    return st["out"]


# ---------------------------------------------------------------------------
# their plain forms
# ---------------------------------------------------------------------------

def _place(st):
    """Request, position and presence of every token row."""
    cu, lens = st["cu"].long(), st["lens"].long()
    t = torch.arange(st["q"].shape[0], device="cuda")
    s = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=lens.numel() - 1)
    return s, lens[s] - cu[s + 1] + t, t < cu[-1]


def _plain_rope(st):
    case = st["case"]
    rot = case["rot"]
    _, pos, live = _place(st)
    a = pos.double().unsqueeze(1) * st["freq"].double()  # (32 bits lose the angles of far positions)
    c, s = ((f(a) * st["mscale"]).float().unsqueeze(1) for f in (torch.cos, torch.sin))
    for x, out in ((st["q"], st["q_out"]), (st["k"], st["k_out"])):
        y = x.float()
        if case["layout"] == "half":
            u, v = y[..., :rot // 2], y[..., rot // 2:rot]
            r = torch.cat((u * c - v * s, v * c + u * s), -1)
        else:
            u, v = y[..., 0:rot:2], y[..., 1:rot:2]
            r = torch.stack((u * c - v * s, v * c + u * s), -1).flatten(-2)
        y = torch.cat((r, y[..., rot:]), -1).to(out.dtype)
        torch.where(live[:, None, None], y, out, out=out)
    return st["q_out"], st["k_out"]


def _copy(st):
    live = st["dst"] >= 0
    src, dst = st["src"][live].long(), st["dst"][live].long()
    st["k_cache"][dst] = st["k_cache"][src]
    st["v_cache"][dst] = st["v_cache"][src]


def _plain_fork(st):
    page = st["case"]["page"]
    table, refs = st["table"], st["refs"]
    parent, child, take = st["parent"].long(), st["child"].long(), st["take"].long()
    n_free, width = st["free"].numel(), table.shape[1]
    head = st["head"].long()
    whole, part = take // page, take % page > 0
    cum = part.cumsum(0)
    fit = ~part | (cum <= n_free - head)
    fresh = st["free"][(head + cum - 1).clamp(0, n_free - 1)]
    col = torch.arange(width, device="cuda").unsqueeze(0)
    old, rows = table[child], table[parent]
    share = fit.unsqueeze(1) & (col < whole.unsqueeze(1))
    new = (fit & part).unsqueeze(1) & (col == whole.unsqueeze(1))
    table[child] = torch.where(share, rows, torch.where(new, fresh.unsqueeze(1), old))
    refs.index_add_(0, rows.clamp(min=0).flatten().long(), share.flatten().int())
    made = fit & part
    st["src"].copy_(torch.where(made, rows.gather(1, whole.clamp(max=width - 1).unsqueeze(1)).squeeze(1), -1))
    st["dst"].copy_(torch.where(made, fresh, -1))
    st["head_out"].copy_(head + torch.where(made, cum, 0).max())
    st["status"].copy_((~fit).any().int())
    _copy(st)
    return tuple(st[x] for x in ("table", "refs", "src", "dst", "head_out", "status", "k_cache", "v_cache"))


def _plain_free(st):
    table, refs, free = st["table"], st["refs"], st["free"]
    pages = refs.numel()
    col = torch.arange(table.shape[1], device="cuda").unsqueeze(0)
    given = (col >= st["first"].unsqueeze(1)) & (col < st["last"].unsqueeze(1))
    given &= (table >= 0) & (table < pages)
    refs.index_add_(0, table.clamp(0, pages - 1).flatten().long(), -given.flatten().int())
    dead = refs < 0
    rank = dead.long().cumsum(0)
    count, head = rank[-1], st["head"].long()
    place = head - count + rank - 1
    status = (refs < -1).any().int() + 2 * (count > head).any().int()
    refs.clamp_(min=0)
    # (one place more takes what is not written)
    room = torch.cat((free, free[:1]))
    room[torch.where(dead & (place >= 0), place, free.numel())] = torch.arange(pages, dtype=torch.int32, device="cuda")
    free.copy_(room[:-1])
    st["head_out"].copy_((head - count).clamp(min=0))
    st["status"].copy_(status)
    return refs, free, st["head_out"], st["status"]


def _plain_compact(st):
    pages, n_free, most = st["refs"].numel(), st["free"].numel(), st["src"].numel()
    at = torch.arange(n_free, device="cuda")
    listed = (at >= st["head"]) & (st["free"] >= 0) & (st["free"] < pages)
    held = torch.ones(pages + 1, dtype=torch.bool, device="cuda")
    held[torch.where(listed, st["free"].long(), pages)] = False
    held = held[:pages]
    count = held.sum()
    ids = torch.arange(pages, device="cuda")
    movers, holes = held & (ids >= count), ~held & (ids < count)
    lists = []
    for mask in (movers, holes):
        x = torch.full((most + 1,), -1, dtype=torch.int64, device="cuda")
        x[torch.where(mask, mask.long().cumsum(0) - 1, most)] = ids
        moved = mask.sum()
        lists.append(torch.where(torch.arange(most, device="cuda") < moved, x[:most], -1))
    st["src"].copy_(lists[0])
    st["dst"].copy_(lists[1])
    to = torch.where(movers, lists[1][(movers.long().cumsum(0) - 1).clamp(0, most - 1)], ids)
    remap = torch.where(held, to, -1)
    st["remap"].copy_(remap)
    inside = (st["table"] >= 0) & (st["table"] < pages)
    st["table_out"].copy_(torch.where(inside, remap[st["table"].clamp(0, pages - 1).long()], -1))
    refs = torch.zeros(pages + 1, dtype=torch.int32, device="cuda")
    refs[torch.where(held, remap, pages)] = st["refs"]
    st["refs_out"].copy_(refs[:pages])
    head = n_free - (pages - count)
    st["free_out"].copy_(torch.where(at >= head, count + at - head, st["free"].long()))
    st["head_out"].copy_(head)
    st["status"].copy_(head != st["head"])
    _copy(st)
    return tuple(st[x] for x in ("table_out", "refs_out", "free_out", "remap", "src", "dst", "head_out", "status",
                                 "k_cache", "v_cache"))


def _unpack(cache, page, d, ids, off):
    """float32 rows [..., kv, d] at offsets off of pages ids."""
    codes = cache[:, :, :page * d // 2].unflatten(-1, (page, d // 2))[ids, :, off]
    scales = cache.view(torch.float16)[:, :, page * d // 4:].unflatten(-1, (page, d // 32))[ids, :, off]
    x = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float() - 8
    return (x.unflatten(-1, (-1, 32)) * scales.float().unsqueeze(-1)).flatten(-2)


def _part(q, k, v, seen, scale):
    """Maximum, sum and weighted values of the softmax over some of a row's keys.  q [n, kv, g, m, d], k and v
    [n, l, kv, d], seen [n, m, l]; keys of no weight leave a maximum of -inf and sums of 0."""
    n, kv, g, m, d = q.shape
    w = torch.matmul(q.flatten(2, 3), k.permute(0, 2, 3, 1).contiguous()).unflatten(2, (g, m)) * scale
    w = torch.where(seen[:, None, None], w, -torch.inf)
    top = w.amax(-1)
    w = torch.exp(w - torch.where(top == -torch.inf, 0.0, top).unsqueeze(-1))
    o = torch.matmul(w.flatten(2, 3), v.permute(0, 2, 1, 3).contiguous()).unflatten(2, (g, m))
    return top, w.sum(-1), o


def _padded(st):
    """Row of each request's i-th token [n, m] and whether it has one."""
    cu = st["cu"].long()
    i = torch.arange(st["max_new"], device="cuda")
    rows = cu[:-1, None] + i
    return rows.clamp(max=st["q"].shape[0] - 1), rows < cu[1:, None], i


def _columns(st, first, most, rest=None):
    """Keys and values of positions first + 0 .. most - 1 of every request (behind positions `rest`), and those
    positions; past a request's table they are any page's."""
    case = st["case"]
    page = case["page"]
    pos = first[:, None] + torch.arange(most, device="cuda")
    if rest is not None:
        pos = torch.cat((rest, pos), 1)
    table = st["table"].long()
    ids = table.gather(1, (pos // page).clamp(max=table.shape[1] - 1)).clamp(min=0)
    return pos, *(_unpack(st[c], page, case["d"], ids, pos % page) for c in ("k_cache", "v_cache"))


def _plain_sinks(st):
    case = st["case"]
    kv, hq, window, sinks = case["kv_heads"], case["q_heads"], case["window"], case["sinks"]
    rows, there, i = _padded(st)
    cu, lens = st["cu"].long(), st["lens"].long()
    before = lens - (cu[1:] - cu[:-1])  # position of the first new token
    p = before[:, None] + i
    q = st["q"][rows].float().unflatten(2, (kv, hq // kv)).permute(0, 2, 3, 1, 4)
    # the sinks, then what the first row's window begins with
    first = (before - window + 1).clamp(min=sinks)
    most = min(window + st["max_new"], st["max_kv"])
    few = torch.arange(min(sinks, st["max_kv"]), device="cuda").expand(lens.numel(), -1)
    pos, k, v = _columns(st, first, most, few)
    at, p = pos[:, None, :], p[:, :, None]
    seen = (at <= p) & ((at > p - window) | (at < sinks)) & (at < lens[:, None, None])
    _, total, o = _part(q, k, v, seen, st["scale"])
    o = o / torch.where(total == 0, 1.0, total).unsqueeze(-1)
    st["out"][rows[there]] = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[there].to(st["out"].dtype)
    return st["out"]


def _plain_prefix(st):
    case = st["case"]
    kv, hq, page, d, length = case["kv_heads"], case["q_heads"], case["page"], case["d"], case["prefix"]
    rows, there, i = _padded(st)
    cu, lens = st["cu"].long(), st["lens"].long()
    p = (lens - (cu[1:] - cu[:-1]))[:, None] + i
    # all rows over the prefix at once
    ids = st["prefix"].long().repeat_interleave(page)
    off = torch.arange(length, device="cuda") % page
    k, v = (_unpack(st[c], page, d, ids, off).unsqueeze(0) for c in ("k_cache", "v_cache"))
    every = st["q"].float().unflatten(1, (kv, hq // kv)).permute(1, 2, 0, 3).unsqueeze(0)
    has = (lens > 0)[_place(st)[0]]
    a = _part(every, k, v, has[None, :, None].expand(1, -1, length), st["scale"])
    a = [x[0].transpose(0, 2) for x in a]  # [tokens, g, kv, ...]
    a = [x[rows].transpose(1, 3) for x in a]  # [n, kv, g, m, ...]
    # each request over its own
    q = st["q"][rows].float().unflatten(2, (kv, hq // kv)).permute(0, 2, 3, 1, 4)
    pos, k, v = _columns(st, torch.full_like(lens, length), max(1, st["max_kv"] - length))
    seen = (pos[:, None, :] <= p[:, :, None]) & (pos[:, None, :] < lens[:, None, None])
    b = _part(q, k, v, seen, st["scale"])
    top = torch.maximum(a[0], b[0])
    top = torch.where(top == -torch.inf, 0.0, top)
    u, w = torch.exp(a[0] - top), torch.exp(b[0] - top)
    total = a[1] * u + b[1] * w
    o = (a[2] * u.unsqueeze(-1) + b[2] * w.unsqueeze(-1)) / torch.where(total == 0, 1.0, total).unsqueeze(-1)
    st["out"][rows[there]] = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[there].to(st["out"].dtype)
    return st["out"]


_PLAIN = {"rope": _plain_rope, "fork": _plain_fork, "free": _plain_free, "compact": _plain_compact,
          "sinks": _plain_sinks, "prefix": _plain_prefix}


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without, and its result in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "rope":
        new, _ = _lengths(case)
        values = int(new.sum()) * (case["q_heads"] + case["kv_heads"])
        return {"bytes": 2 * values * case["d"] * (4 if case["dtype"] == "f32" else 2), "flops": 3 * values * case["rot"]}
    if op == "fork":
        _, take = _fork_lengths(case)
        whole, part = int((take // case["page"]).sum()), int((take % case["page"] > 0).sum())
        # entries read and written, holders counted; copied pages of both caches
        return {"bytes": 16 * whole + 12 * case["forks"] + part * (20 + 4 * case["kv_heads"] * _page_bytes(case)),
                "flops": 0}
    if op == "free":
        held, first, last = _free_ranges(case)
        return {"bytes": 8 * case["requests"] + 16 * int((last - first).sum()), "flops": 0}
    if op == "compact":
        held = _compact_held(case)
        pages, count = case["pages"], int(held.sum())
        moved = int(held[count:].sum())
        # the free list and the table read and written, holders and new ids written; copied pages of both caches
        return {"bytes": 8 * (pages - count) + 8 * count + 8 * pages + 4 * pages + 8 * moved
                + 4 * moved * case["kv_heads"] * _page_bytes(case), "flops": 0}
    new, lens = _lengths(case)
    keys = pairs = 0
    if op == "prefix":
        keys = case["prefix"]
        for m, length in zip(new.tolist(), lens.tolist()):
            if length:
                keys += length - case["prefix"]
                pairs += m * (length - m) + m * (m + 1) // 2
    else:
        window, sinks = case["window"], case["sinks"]
        for m, length in zip(new.tolist(), lens.tolist()):
            if length:
                first = max(0, length - m - window + 1)
                keys += length - first + min(sinks, first)
                p = torch.arange(length - m, length)
                lo = (p - window + 1).clamp(min=0)
                pairs += int((p + 1 - lo + lo.clamp(max=sinks)).sum())
    q = 2 * int(new.sum()) * case["q_heads"] * case["d"]
    return {"bytes": int(keys * case["kv_heads"] * case["d"] * 9 / 8 + 2 * q), "flops": 4 * case["d"] * case["q_heads"] * pairs}


def _exact_rope(st):
    case = st["case"]
    cu, lens = st["cu"].tolist(), st["lens"].tolist()
    res = []
    for x in (st["q"], st["k"]):
        y = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
        for s, length in enumerate(lens):
            a, b = cu[s], cu[s + 1]
            pos = torch.arange(length - (b - a), length, dtype=torch.float64, device="cuda")
            turn = torch.polar(torch.tensor(st["mscale"], dtype=torch.float64, device="cuda").expand(b - a, case["rot"] // 2),
                               pos[:, None] * st["freq"].double()[None, :])
            z = x[a:b].double()
            y[a:b] = z
            if case["layout"] == "pairs":
                w = torch.view_as_complex(z[..., :case["rot"]].reshape(*z.shape[:2], -1, 2).contiguous()) * turn[:, None]
                y[a:b, :, :case["rot"]] = torch.view_as_real(w).reshape(*z.shape[:2], -1)
            else:
                h = case["rot"] // 2
                w = torch.complex(z[..., :h].contiguous(), z[..., h:2 * h].contiguous()) * turn[:, None]
                y[a:b, :, :h], y[a:b, :, h:2 * h] = w.real, w.imag
        res.append(y)
    return tuple(res)


def _exact_attn(st):
    case = st["case"]
    page, d, kv, hq = case["page"], case["d"], case["kv_heads"], case["q_heads"]
    group = hq // kv
    window, sinks = case.get("window", 1 << 40), case.get("sinks", 0)
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    codes_at = page * d // 2

    def values(cache, ids, h):
        raw = cache[ids, h]
        by = raw[:, :codes_at].reshape(-1, d // 2)
        row = torch.empty((by.shape[0], d), dtype=torch.float64, device="cuda")
        row[:, 0::2] = (by % 16).double() - 8
        row[:, 1::2] = (by // 16).double() - 8
        return row * raw[:, codes_at:].contiguous().view(torch.float16).reshape(-1, d // 32).double().repeat_interleave(32, 1)

    cu = st["cu"].tolist()
    for s, length in enumerate(st["host_lens"]):
        a, b = cu[s], cu[s + 1]
        if length:
            ids = st["table"][s, :math.ceil(length / page)].long()
            place = torch.arange(length, device="cuda")
            for h in range(kv):
                k, v = values(st["k_cache"], ids, h)[:length], values(st["v_cache"], ids, h)[:length]
                for j in range(group):
                    for t in range(a, b, 2048):
                        e = min(b, t + 2048)
                        logits = st["q"][t:e, h * group + j].double() @ k.T * st["scale"]
                        pos = (length - b + torch.arange(t, e, device="cuda"))[:, None]
                        hidden = (place[None, :] > pos) | ((place[None, :] <= pos - window) & (place[None, :] >= sinks))
                        logits.masked_fill_(hidden, -math.inf)
                        out[t:e, h * group + j] = torch.softmax(logits, -1) @ v
    return out


def exact(case, seed):
    """None for the page operators: their outputs are whole numbers and bytes carried over."""
    op = case["op"]
    if op in ("fork", "free", "compact"):
        return None
    st = prepare(case, seed)
    return _exact_rope(st) if op == "rope" else _exact_attn(st)
