"""GPU parity of the 4-bit cache operators: block tables, row store and load, attention.

Block tables, stored bytes and loaded values equal the oracle exactly.
Attention is held to a bound from its roundings (``_bound``): keys and values
enter as float16 (half a step, 2^-11 relative), so a logit is off by at most
E = (2^-11 + d 2^-23) scale sum |q| |k| (the second term the float32 sums), a
probability by a factor e^(2E), its own float16 rounding 2^-11 (an absolute
2^-25 of the largest below float16's normal range), float32 exponentials and
sums 2^-16, and the store by half a step of the output type.
"""

import numpy as np
import pytest

from _gpu import dev, host, say
from oracle import kvcache

pytestmark = pytest.mark.gpu

HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module")
def kq():
    from gguf_quant_matmul_amd import kq as mod

    return mod


def _tdt(name):
    import torch

    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def _i32(a):
    return dev(np.ascontiguousarray(a, dtype=np.int32))


def _f64(t):
    import torch

    return host(t.to(torch.float64))


def _close(got, ref, bound, what):
    assert np.isfinite(got).all(), f"{what}: non-finite output"
    use = np.abs(got - ref) / np.maximum(bound, 1e-300)
    use[(got == ref)] = 0
    i = np.unravel_index(int(use.argmax()), use.shape) if use.size else ()
    if use.size:
        assert use.max() <= 1, f"{what}: {got[i]!r} for {ref[i]!r} at {i}, bound {bound[i]:.3e}"
        say(f"  {what}: bound use {use.max():.3f}")


def _bound(ref, absv, mag, count, vmax, d, out):
    e = (2.0 ** -11 + d * 2.0 ** -23) * mag[..., None]
    p = absv * (np.expm1(2 * e) + 2 * 2.0 ** -11 + 2.0 ** -16) * 1.01
    small = count[..., None] * 2.0 ** -25 * vmax
    tiny = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}[out]
    return p + small + HALF_STEP[out] * (np.abs(ref) + p + small) + tiny


# ---------------------------------------------------------------------------
# rows
# ---------------------------------------------------------------------------

def _row_case(seed, tokens, heads, d, dtype, special=False):
    """Rows as a device tensor of `dtype` and the float32 values they hold."""
    import torch

    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((tokens, heads, d)) * np.exp2(rng.integers(-8, 5, (tokens, heads, 1)))).astype(np.float32)
    x[0, 0] = 0
    if special:
        x[-1, 0, :6] = [np.nan, np.inf, 1, -np.inf, 3, 0]
        x[-2, 0, :4] = [7, -6.5, 0.5, -0.5]
        x[-2, 0, 4:] = np.clip(x[-2, 0, 4:], -6, 6)
        x[-3, 0] *= 1e-8
        x[-4, 0] = np.nan
        x[-5, 0, 3] = 65000
    t = dev(x).to(_tdt(dtype))
    return t, host(t.to(torch.float32))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("tokens, heads, d, page", [(1, 1, 32, 16), (7, 2, 64, 32), (37, 5, 96, 16), (130, 8, 128, 64),
                                                     (40, 1, 224, 256), (65, 3, 256, 16)])
def test_store_and_load_equal_the_oracle(kq, dtype, tokens, heads, d, page):
    import torch

    special = tokens > 5
    k, kf = _row_case(1, tokens, heads, d, dtype, special)
    v, vf = _row_case(2, tokens, heads, d, dtype, special)
    rng = np.random.default_rng(3)
    pages = tokens // page + 3
    slots = rng.permutation(pages * page)[:tokens]
    if tokens > 5:
        slots[[1, 4]] = [-1, pages * page]
    # rows as slices of a wider buffer
    wide = torch.full((tokens, 2 * heads + 1, d), 9.0, dtype=k.dtype, device="cuda")
    wide[:, 1:heads + 1], wide[:, heads + 1:] = k, v
    kc, vc = (torch.full((pages, heads, kvcache.page_bytes(page, d)), 0xA5, dtype=torch.uint8, device="cuda")
              for _ in range(2))
    want = []
    for x in (kf, vf):
        c = np.full(tuple(kc.shape), 0xA5, np.uint8)
        kvcache.store(c, page, slots, *kvcache.encode(x))
        want.append(c)
    kq.kq_kv_store("q4_0", wide[:, 1:heads + 1], wide[:, heads + 1:], _i32(slots), kc, vc, page)
    assert np.array_equal(host(kc), want[0]) and np.array_equal(host(vc), want[1])

    live = (slots >= 0) & (slots < pages * page)
    for out in ("f32", "f16", "bf16"):
        ko, vo = (torch.full((tokens, heads, d), 5.0, dtype=_tdt(out), device="cuda") for _ in range(2))
        kq.kq_kv_load("q4_0", kc, vc, _i32(slots), page, ko, vo)
        for got, c in ((ko, want[0]), (vo, want[1])):
            ref = torch.full((tokens, heads, d), 5.0, dtype=torch.float64)
            ref[torch.from_numpy(live)] = torch.from_numpy(kvcache.load(c, page, d, slots[live]))
            # exact in float32; a narrower type rounds that once
            assert torch.equal(got.cpu(), ref.to(torch.float32).to(_tdt(out)))


def test_store_is_the_wire_encoder(kq):
    import torch

    rng = np.random.default_rng(11)
    x = dev((rng.standard_normal((50, 128)) * 3).astype(np.float32))
    wire = kq.quantize("q4_0", x)
    kc, vc = kq.kv_cache("q4_0", 4, 1, 16, 128)
    kq.kq_kv_store("q4_0", x.view(50, 1, 128), -x.view(50, 1, 128), _i32(np.arange(50)), kc, vc, 16)
    k, v = (torch.empty((50, 1, 128), dtype=torch.float32, device="cuda") for _ in range(2))
    kq.kq_kv_load("q4_0", kc, vc, _i32(np.arange(50)), 16, k, v)
    assert torch.equal(k.view(50, 128), kq.dequantize("q4_0", wire, 128, torch.float32))


# ---------------------------------------------------------------------------
# block tables
# ---------------------------------------------------------------------------

def _tables_case(rng, n, page, max_ctx, max_new, slack, width=None, short=0):
    ctx = rng.integers(0, max_ctx + 1, n)
    new = rng.integers(0, max_new + 1, n)
    held = -(-ctx // page)
    total = -(-(ctx + new) // page)
    width = int(total.max()) + 2 if width is None else width
    need = int((total - held).sum())
    ids = rng.permutation(int(held.sum()) + need + 9)
    table = np.full((n, width), -1)
    at = 0
    for s in range(n):
        h = min(int(held[s]), width)
        table[s, :h] = ids[at:at + h]
        at += h
    head = int(rng.integers(0, 4))
    free = np.concatenate((np.full(head, -7), ids[at:at + max(0, need + slack)]))
    tokens = max(0, int(new.sum()) + (0 if short else int(rng.integers(0, 5))) - short)
    return ctx, new, free, head, table, tokens


def _check_tables(kq, page, ctx, new, free, head, table, tokens, what):
    import torch

    want = kvcache.block_tables(ctx, new, page, free, head, table, tokens)
    t, n = _i32(table), len(ctx)
    fill = lambda m: torch.full((m,), -99, dtype=torch.int32, device="cuda")
    slots, cu, lens, ho, status = fill(tokens), fill(n + 1), fill(n), fill(1), fill(1)
    kq.kq_block_tables(_i32(ctx), _i32(new), _i32(free), _i32([head]), page, t, slots, cu, lens, ho, status)
    got = [host(x).tolist() for x in (t, slots, cu, lens, ho, status)]
    for name, g, w in zip(("table", "slots", "cu", "lens", "head", "status"), got,
                          want[:4] + ([want[4]], [want[5]])):
        assert g == w, f"{what}: {name}"


@pytest.mark.parametrize("n, page, max_ctx, max_new", [(1, 16, 0, 1), (1, 16, 40, 5000), (3, 16, 100, 50), (64, 64, 3000, 1),
                                                       (257, 32, 500, 9), (1500, 16, 200, 3), (5000, 128, 900, 2)])
def test_block_tables_equal_the_oracle(kq, n, page, max_ctx, max_new):
    rng = np.random.default_rng(n)
    for slack, short in ((2, 0), (-1, 0), (-3, 0), (1, 2)):
        _check_tables(kq, page, *_tables_case(rng, n, page, max_ctx, max_new, slack, short=short), f"slack {slack} short {short}")


def test_block_tables_odd_inputs(kq):
    rng = np.random.default_rng(4)
    # a table narrower than some requests need
    _check_tables(kq, 16, *_tables_case(rng, 40, 16, 300, 60, 5, width=12), "narrow")
    # negative lengths, a free list that is spent, a head out of range
    ctx, new, free, head, table, tokens = _tables_case(rng, 30, 16, 100, 20, 3)
    bad_ctx, bad_new = ctx.copy(), new.copy()
    bad_ctx[3], bad_new[7], bad_new[29] = -5, -1, 2 ** 31 - 1
    _check_tables(kq, 16, bad_ctx, bad_new, free, head, table, tokens, "negative")
    _check_tables(kq, 16, ctx, new, free, len(free), table, tokens, "spent")
    _check_tables(kq, 16, ctx, new, free, -2, table, tokens, "head before the list")
    _check_tables(kq, 16, ctx, new, free, len(free) + 3, table, tokens, "head behind the list")
    # ids that fit no slot
    _check_tables(kq, 4096, [0], [4097], [2 ** 31 - 1, 2 ** 19 - 1, -4], 0, [[-1, -1]], 4097, "large ids")
    # no request, no rows
    _check_tables(kq, 16, [], [], [4, 5], 1, np.zeros((0, 3), int), 6, "no request")
    _check_tables(kq, 16, [5], [0], [4, 5], 1, [[3, -1]], 0, "no rows")


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def _case(seed, new, lens, hq, kv, d, page, q_dtype="f16", q_scale=1.0, extra_tokens=0, garbage=0xFF):
    """Queries and caches of a batch; bytes of the caches that no row fills are `garbage` (NaN scales)."""
    rng = np.random.default_rng(seed)
    new, lens = np.asarray(new), np.asarray(lens)
    n = len(new)
    cu = np.concatenate(([0], np.cumsum(new)))
    tokens = int(cu[-1]) + extra_tokens
    width = max(1, int(-(-lens.max() // page)))
    held = -(-lens // page)
    pages = int(held.sum()) + 2
    ids = rng.permutation(pages)
    table = np.full((n, width), -1)
    caches = [np.full((pages, kv, kvcache.page_bytes(page, d)), garbage, np.uint8) for _ in range(2)]
    at = 0
    for s in range(n):
        table[s, :held[s]] = ids[at:at + held[s]]
        at += held[s]
        slots = table[s][np.arange(lens[s]) // page] * page + np.arange(lens[s]) % page
        for c in caches:
            kvcache.store(c, page, slots, *kvcache.encode(rng.standard_normal((lens[s], kv, d)).astype(np.float32)))
    q = dev((rng.standard_normal((tokens, hq, d)) * q_scale).astype(np.float32)).to(_tdt(q_dtype))
    return dict(q=q, cu=cu, lens=lens, table=table, kc=caches[0], vc=caches[1], page=page, d=d)


def _attn(kq, c, out="f16", scale=None, window=0, max_new=None, max_kv=None, **kw):
    import torch

    o = torch.full(c["q"].shape, 77.0, dtype=_tdt(out), device="cuda")
    kq.kq_kv_attention("q4_0", c["q"], _i32(c["cu"]), _i32(c["lens"]), _i32(c["table"]), dev(c["kc"]), dev(c["vc"]),
                       c["page"], o, scale=scale, window=window, max_new=max_new, max_kv=max_kv, **kw)
    return o


def _check(kq, c, what, out="f16", scale=None, window=0, **kw):
    sc = c["d"] ** -0.5 if scale is None else float(np.float32(scale))
    ref, absv, mag, count = kvcache.attention(_f64(c["q"]), c["cu"], c["lens"], c["table"], c["kc"], c["vc"], c["page"],
                                              sc, window, detail=True)
    got = _f64(_attn(kq, c, out, scale, window, **kw))
    none = np.isnan(ref)
    assert (got[none] == 77).all(), f"{what}: rows of no request were written"
    ref[none] = got[none]
    vmax = 0.0
    if c["lens"].max() > 0:
        vmax = np.nanmax(np.abs(kvcache.load(c["vc"], c["page"], c["d"], np.arange(c["vc"].shape[0] * c["page"]))))
    empty = (count == 0) & ~none.any(-1)
    assert not got[empty].any(), f"{what}: a row without keys is not zero"
    _close(got, ref, _bound(ref, absv, mag, count, vmax, c["d"], out), what)


HEADS = [(1, 1, 32, 16), (8, 2, 64, 16), (4, 4, 96, 32), (32, 8, 128, 64), (7, 1, 160, 16), (6, 2, 192, 16),
         (20, 1, 224, 32), (16, 4, 256, 128)]


@pytest.mark.parametrize("q_dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq, kv, d, page", HEADS)
def test_single_tokens(kq, hq, kv, d, page, q_dtype):
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 0, 129, 300]
    c = _case(d, [1] * len(lens), lens, hq, kv, d, page, q_dtype)
    _check(kq, c, "host bounds", q_dtype, max_new=1, max_kv=300)
    _check(kq, c, "no bounds", "f32")
    _check(kq, c, "window", q_dtype, window=33, max_new=1, max_kv=300)


@pytest.mark.parametrize("q_dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq, kv, d, page", HEADS)
def test_prompts(kq, hq, kv, d, page, q_dtype):
    new = [1, 37, 0, 64, 5, 3, 9]
    lens = [1, 37, 10, 130, 200, 0, 4]  # from the first token, on top of cached ones, none, fewer keys than queries
    c = _case(d + 1, new, lens, hq, kv, d, page, q_dtype, extra_tokens=3)
    _check(kq, c, "host bounds", q_dtype, max_new=64, max_kv=200)
    _check(kq, c, "no bounds", "bf16")
    _check(kq, c, "window", q_dtype, window=17, max_new=64, max_kv=200)


@pytest.mark.parametrize("q_dtype, hq, kv, d", [("f16", 8, 2, 128), ("bf16", 4, 4, 64)])
def test_uniform_weights_count_every_key_once(kq, q_dtype, hq, kv, d):
    # scale 0: the mean of the values; a key left out or taken twice is 1 / n
    # of a value, several times the bound at these lengths
    c = _case(50, [1, 1, 3, 70, 1], [330, 65, 66, 200, 511], hq, kv, d, 16, q_dtype)
    _check(kq, c, "mean", "f32", scale=0.0, max_new=70, max_kv=511)
    _check(kq, c, "mean, window", "f32", scale=0.0, window=100, max_new=70, max_kv=511)


@pytest.mark.parametrize("max_new", [1, 600])
def test_each_key_is_found(kq, max_new):
    # queries that are large multiples of one key each: the output is that key's value
    import torch

    hq, kv, d, page, n = 4, 2, 128, 32, 600
    c = _case(60, [n], [n], hq, kv, d, page)
    slots = c["table"][0][np.arange(n) // page] * page + np.arange(n) % page
    k, v = (kvcache.load(x, page, d, slots) for x in (c["kc"], c["vc"]))
    rng = np.random.default_rng(61)
    pick = np.array([rng.integers(0, t + 1) for t in range(n)])
    q = np.repeat(k[pick], hq // kv, axis=1)
    c["q"] = dev((8 * q).astype(np.float16))
    got = _f64(_attn(kq, c, "f32", scale=1.0, max_new=max_new, max_kv=n))
    # |k|^2 is near 128 and other products below 80: weights of other keys under e^-300
    ref = np.repeat(v[pick], hq // kv, axis=1)
    assert np.abs(got - ref).max() <= 2.0 ** -10 * np.abs(ref).max()
    assert torch.isfinite(torch.from_numpy(got)).all()


@pytest.mark.parametrize("n, length, max_kv", [(1, 5000, 5000), (2, 1000, 131072), (3, 9000, 512), (70, 700, 700)])
def test_split_keys(kq, n, length, max_kv):
    # rows whose keys are shared by several workgroups; bounds that are too wide and too narrow
    rng = np.random.default_rng(n)
    lens = rng.integers(1, length + 1, n)
    lens[0] = length
    c = _case(70 + n, [1] * n, lens, 4, 2, 64, 64)
    _check(kq, c, "split", "f16", max_new=1, max_kv=max_kv)
    _check(kq, c, "split, window", "f16", window=length // 2, max_new=1, max_kv=max_kv)


def test_drafts_and_bounds_that_do_not_hold(kq):
    new = [6, 1, 3, 40, 2]
    c = _case(80, new, [400, 1, 90, 300, 65], 8, 1, 64, 16)
    _check(kq, c, "drafts", "f16", max_new=6, max_kv=400)
    _check(kq, c, "bounds of one token and one key", "f16", max_new=1, max_kv=1)


@pytest.mark.parametrize("d, hq, kv, page", [(64, 4, 2, 16), (128, 8, 2, 128), (96, 3, 3, 64), (256, 4, 2, 4096)])
def test_shared_steps_of_many_requests(kq, d, hq, kv, page):
    # more than 64 requests whose steps are shared out evenly, idle ones among them, first and last included
    rng = np.random.default_rng(160 + d)
    n = 90
    lens = rng.integers(0, 300, n)
    lens[[0, 1, 40, 41, 42, 89]] = 0
    lens[[7, 50]] = [1500, 2300]
    c = _case(160 + d, rng.integers(0, 3, n), lens, hq, kv, d, page, "bf16" if d == 96 else "f16", extra_tokens=2)
    _check(kq, c, "shared", "f32", max_new=2, max_kv=2300)
    _check(kq, c, "bounds that do not hold", "f16", max_new=1, max_kv=1025)
    _check(kq, c, "uniform", "f32", scale=0.0, max_new=2, max_kv=100000)


def test_shared_steps_of_rows_past_the_bound(kq):
    c = _case(170, [40, 1, 70, 5], [1400, 30, 900, 5], 8, 2, 64, 16)
    _check(kq, c, "16-row tiles of long requests", "f16", max_new=1, max_kv=1400)
    _check(kq, c, "window", "f16", max_new=1, max_kv=1400, window=1100)


def test_more_requests_than_share_steps(kq):
    rng = np.random.default_rng(171)
    lens = rng.integers(0, 40, 1100)
    lens[5] = 1300
    _check(kq, _case(171, [1] * 1100, lens, 2, 1, 32, 16), "one workgroup to a request", "f16", max_new=1, max_kv=1300)


@pytest.mark.parametrize("d, hq, kv, q_dtype", [(128, 8, 1, "f16"), (64, 7, 1, "bf16"), (256, 4, 1, "f16"), (160, 3, 1, "bf16")])
def test_prompts_whose_keys_are_split(kq, d, hq, kv, q_dtype):
    # prompt tiles and 16-row tiles in one batch, both with shared keys
    c = _case(180 + d, [20, 1, 45, 2, 0, 33], [2500, 1700, 45, 2100, 10, 1300], hq, kv, d, 64, q_dtype, extra_tokens=1)
    _check(kq, c, "split", q_dtype, max_new=45, max_kv=2500)
    _check(kq, c, "split, wide bound", "f32", max_new=45, max_kv=200000)
    _check(kq, c, "window", q_dtype, max_new=45, max_kv=2500, window=700)
    _check(kq, c, "uniform", "f32", scale=0.0, max_new=45, max_kv=2500)


@pytest.mark.parametrize("d, hq, kv, q_dtype", [(32, 64, 32, "f16"), (128, 40, 40, "bf16"), (224, 48, 16, "f16")])
def test_prompts_in_even_shares(kq, d, hq, kv, q_dtype):
    # few workgroups to a head: each has a piece of one prompt's tile, several whole ones and a piece of another
    rng = np.random.default_rng(185 + d)
    new = np.concatenate((rng.integers(34, 150, 9), [0, 0, 35, 300, 1, 270]))
    lens = new + rng.integers(0, 200, len(new)) * (rng.random(len(new)) < 0.6)
    lens[3], lens[9], lens[12] = 20, 0, 333  # rows before the first key, an idle request, a longer one
    c = _case(185 + d, new, lens, hq, kv, d, 16, q_dtype, extra_tokens=3)
    for max_kv in (700, 300000):
        _check(kq, c, f"max_kv {max_kv}", "f16", max_new=300, max_kv=max_kv)
    _check(kq, c, "window", "f32", max_new=300, max_kv=300000, window=90)
    c = _case(186 + d, [301], [411], hq, kv, d, 32, q_dtype)
    _check(kq, c, "one request", "f16", max_new=301, max_kv=300000)


@pytest.mark.parametrize("d, hq, kv, n", [(128, 4, 1, 200), (128, 16, 2, 70), (192, 5, 1, 130), (32, 1, 1, 300)])
def test_prompts_over_several_tiles(kq, d, hq, kv, n):
    c = _case(190 + d + n, [n], [n + 77], hq, kv, d, 32)
    _check(kq, c, "prompt", "f16", max_new=n, max_kv=n + 77)
    _check(kq, c, "window", "f32", max_new=n, max_kv=n + 77, window=50)
    c = _case(191 + d + n, [n], [n], hq, kv, d, 32, "bf16")
    _check(kq, c, "from the first token", "bf16", max_new=n, max_kv=n)


def test_strided_queries_and_results_repeat(kq):
    import torch

    c = _case(200, [1, 60, 1, 4], [3000, 900, 1, 1200], 6, 3, 128, 16)
    wide = torch.full((66, 14, 128), 3.0, dtype=torch.float16, device="cuda")
    wide[:, 5:11] = c["q"]
    first = None
    for q in (c["q"], wide[:, 5:11]):
        for _ in range(3):
            got = _attn(kq, dict(c, q=q), "f16", max_new=60, max_kv=3000)
            first = got.clone() if first is None else first
            assert torch.equal(got, first)


def test_workspace_that_is_too_small(kq):
    import torch

    c = _case(210, [1, 1], [3000, 900], 4, 2, 64, 16)
    with pytest.raises(kq.KQError) as e:
        _attn(kq, c, "f16", max_new=1, max_kv=3000, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == kq.KQ_ERR_CAPACITY
    with pytest.raises(ValueError, match="cu_new has 2"):
        _attn(kq, dict(c, cu=c["cu"][:2]), "f16", max_new=1, max_kv=3000)


def test_signs_and_sizes_of_scale_and_queries(kq):
    for q_dtype, q_scale, scale in (("f16", 1.0, -0.2), ("bf16", 1e-20, 1e19), ("bf16", 1e20, 1e-21), ("bf16", 300.0, -1e-3),
                                    ("f16", 1e-3, 50.0), ("bf16", 1.0, 1e-38)):
        c = _case(90, [1, 30, 1], [100, 60, 1], 4, 2, 64, 16, q_dtype, q_scale)
        _check(kq, c, f"{q_dtype} queries of {q_scale}, scale {scale}", "f16" if q_dtype == "f16" else "bf16", scale=scale)


def test_lengths_and_offsets_are_bounded(kq):
    c = _case(100, [2, 4, 1], [40, 70, 33], 4, 2, 64, 16, extra_tokens=2)
    c["lens"] = np.array([-3, 1 << 29, 33])  # none; the table's width
    c["kc"][:], c["vc"][:] = 0x11, 0x22  # every byte a finite scale or code
    c["table"][1, :] = [0, 1, 2, 3, 4]
    _check(kq, c, "lengths", "f16", max_new=4, max_kv=70)
    c = _case(101, [2, 4, 1], [40, 70, 33], 4, 2, 64, 16, extra_tokens=2)
    for cu in ([0, 2, 6, 400], [-5, 2, 6, 7]):
        c["cu"] = np.array(cu)
        _check(kq, c, f"offsets {cu}", "f16", max_new=9, max_kv=70)


def test_pages_outside_the_cache_are_left_out(kq):
    c = _case(110, [1, 20, 1], [100, 90, 40], 8, 2, 64, 16)
    c["table"][0, 2], c["table"][0, 6], c["table"][1, 0], c["table"][1, 3] = -1, 1 << 30, c["kc"].shape[0], -9
    c["table"][2, :3] = -1  # no key at all
    _check(kq, c, "bad pages", "f16", max_new=20, max_kv=100)


def test_nan_queries_stay_in_their_row(kq):
    import torch

    for q_dtype in ("f16", "bf16"):
        c = _case(120, [1, 40], [100, 60], 4, 2, 64, 16, q_dtype)
        clean = _attn(kq, c, q_dtype, max_new=40, max_kv=100)
        c["q"][3, 1, 5] = float("nan")
        c["q"][0, 0, 0] = float("inf")
        got = _attn(kq, c, q_dtype, max_new=40, max_kv=100)
        assert torch.isnan(got[3, 1]).all() and torch.isnan(got[0, 0]).all()
        got[3, 1], got[0, 0] = clean[3, 1], clean[0, 0]
        assert torch.equal(got, clean)


def test_offsets_past_32_bits(kq):
    import torch

    page, kv, d, hq = 256, 8, 128, 8
    pb = kvcache.page_bytes(page, d)
    pages = (5 << 30) // (kv * pb)
    kc, vc = (torch.full((pages, kv, pb), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2))
    rng = np.random.default_rng(130)
    length = 700
    ids = np.array([pages - 1, pages - 7, pages // 2 + 1])
    slots = ids[np.arange(length) // page] * page + np.arange(length) % page
    k, v = ((rng.standard_normal((length, kv, d))).astype(np.float16) for _ in range(2))
    kq.kq_kv_store("q4_0", dev(k), dev(v), _i32(slots), kc, vc, page)
    ko, vo = (torch.empty((length, kv, d), dtype=torch.float32, device="cuda") for _ in range(2))
    kq.kq_kv_load("q4_0", kc, vc, _i32(slots), page, ko, vo)
    ck, cv = kvcache.encode(k.astype(np.float32)), kvcache.encode(v.astype(np.float32))
    assert np.array_equal(host(ko), kvcache.values(*ck)) and np.array_equal(host(vo), kvcache.values(*cv))
    q = rng.standard_normal((1, hq, d)).astype(np.float16)
    out = torch.zeros((1, hq, d), dtype=torch.float16, device="cuda")
    kq.kq_kv_attention("q4_0", dev(q), _i32([0, 1]), _i32([length]), _i32([ids]), kc, vc, page, out, max_new=1,
                       max_kv=length)
    small = [np.zeros((3, kv, pb), np.uint8) for _ in range(2)]
    for c, e in zip(small, (ck, cv)):
        kvcache.store(c, page, np.arange(length), *e)
    ref, absv, mag, count = kvcache.attention(q, [0, 1], [length], [[0, 1, 2]], *small, page, d ** -0.5, detail=True)
    _close(_f64(out), ref, _bound(ref, absv, mag, count, np.abs(kvcache.values(*cv)).max(), d, "f16"), "far pages")


# ---------------------------------------------------------------------------
# streams, graphs, a run of them together
# ---------------------------------------------------------------------------

def test_graphs_and_streams(kq):
    import torch

    c = _case(140, [1] * 6, [900, 3, 0, 64, 2000, 500], 16, 4, 128, 64)
    d = _case(141, [30, 50], [700, 50], 16, 4, 128, 64)
    args = []
    for x, mn in ((c, 1), (d, 50)):
        need = kq.kq_kv_attention_workspace(len(x["q"]), len(x["lens"]), 16, 4, 128, mn, 2000)
        args.append(dict(q=x["q"], cu=_i32(x["cu"]), lens=_i32(x["lens"]), table=_i32(x["table"]), kc=dev(x["kc"]),
                         vc=dev(x["vc"]), out=torch.zeros_like(x["q"]), mn=mn,
                         ws=torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")))

    def work(a, stream=None):
        kq.kq_kv_attention("q4_0", a["q"], a["cu"], a["lens"], a["table"], a["kc"], a["vc"], 64, a["out"],
                           max_new=a["mn"], max_kv=2000, workspace=a["ws"], stream=stream)

    for a in args:
        work(a)
    torch.cuda.synchronize()
    ref = [a["out"].clone() for a in args]
    graphs = []
    for a in args:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            work(a)
        graphs.append(g)
    for _ in range(4):
        for a in args:
            a["out"].zero_()
            a["ws"].fill_(0x7F)
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a["out"], r) for a, r in zip(args, ref))
    # two calls at once, on streams of their own with workspaces of their own
    streams = [torch.cuda.Stream() for _ in args]
    for a in args:
        a["out"].zero_()
    torch.cuda.synchronize()
    for a, s in zip(args, streams):
        work(a, s)
    torch.cuda.synchronize()
    assert all(torch.equal(a["out"], r) for a, r in zip(args, ref))
    with pytest.raises(ValueError, match="own workspace"):
        a = args[0]
        kq.kq_kv_attention("q4_0", a["q"], a["cu"], a["lens"], a["table"], a["kc"], a["vc"], 64, a["out"], max_new=1,
                           max_kv=100000, stream=streams[0])


def test_a_run_of_steps(kq):
    """Requests that are admitted, grow over page borders and finish: tables, store and attention each step, the
    queries, keys and values from one quantized projection."""
    import torch

    rng = np.random.default_rng(150)
    hq, kv, d, page, hidden, n, width = 8, 2, 64, 16, 256, 5, 6
    rows = (hq + 2 * kv) * d
    w = kq.quantize("q4_0", dev((rng.standard_normal((rows, hidden)) * 0.06).astype(np.float32)))
    pages = 24
    kc, vc = kq.kv_cache("q4_0", pages, kv, page, d)
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    free = _i32(rng.permutation(pages))
    head = _i32([0])
    ctx = np.zeros(n, int)
    mirror = [np.zeros(tuple(kc.shape), np.uint8) for _ in range(2)]
    for step, new in enumerate(([13, 16, 0, 1, 0], [1, 1, 33, 1, 0], [1, 1, 1, 1, 5], [3, 1, 1, 0, 1], [1, 1, 1, 1, 20])):
        tokens = sum(new) + 2
        x = dev(rng.standard_normal((tokens, hidden)).astype(np.float16))
        qkv = kq.quantized_matmul("q4_0", w, rows, hidden, x).view(tokens, hq + 2 * kv, d)
        before = host(table).tolist()
        slots, cu, lens, head2, status = kq.block_tables(_i32(ctx), _i32(new), free, head, page, table, tokens)
        want = kvcache.block_tables(ctx, new, page, host(free), int(head.item()), before, tokens)
        assert [host(t).tolist() for t in (table, slots, cu, lens)] == list(want[:4]) and status.item() == want[5] == 0
        k, v = qkv[:, hq:hq + kv], qkv[:, hq + kv:]
        kq.kq_kv_store("q4_0", k, v, slots, kc, vc, page)
        for c, y in zip(mirror, (k, v)):
            kvcache.store(c, page, want[1], *kvcache.encode(host(y.float())))
        assert np.array_equal(host(kc), mirror[0]) and np.array_equal(host(vc), mirror[1])
        out = kq.kv_attention("q4_0", qkv[:, :hq], cu, lens, table, kc, vc, page, max_new=max(new),
                              max_kv=int(max(ctx + new)))
        ref, absv, mag, count = kvcache.attention(_f64(qkv[:, :hq]), want[2], want[3], want[0], *mirror, page, d ** -0.5,
                                                  detail=True)
        ref[np.isnan(ref)] = 0
        _close(_f64(out), ref, _bound(ref, absv, mag, count, 20.0, d, "f16"), f"step {step}")
        ctx, head = ctx + np.array(new), head2
