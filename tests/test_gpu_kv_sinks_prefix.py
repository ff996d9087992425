"""GPU parity of attention with sinks and over a shared prefix, and serving steps of all cache operators together.

Bounds are those of ``test_gpu_kv``: the rows' sums over a prefix and over their
own keys are joined in float32, as those of workgroups that share a row are.
"""

import numpy as np
import pytest

from _gpu import dev, host
from oracle import kvcache
from test_gpu_kv import HEADS, _bound, _case, _close, _f64, _i32, _tdt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kq():
    from gguf_quant_matmul_amd import kq as mod

    return mod


def _hold(c, got, what, out, scale=None, window=0, sinks=0, prefix=None):
    sc = c["d"] ** -0.5 if scale is None else float(np.float32(scale))
    ref, absv, mag, count = kvcache.attention(_f64(c["q"]), c["cu"], c["lens"], c["table"], c["kc"], c["vc"], c["page"], sc,
                                              window, detail=True, sinks=sinks, prefix=prefix)
    got = _f64(got)
    none = np.isnan(ref)
    assert (got[none] == 77).all(), f"{what}: rows of no request were written"
    ref[none] = got[none]
    vmax = np.nanmax(np.abs(kvcache.load(c["vc"], c["page"], c["d"], np.arange(c["vc"].shape[0] * c["page"]))))
    assert not got[(count == 0) & ~none.any(-1)].any(), f"{what}: a row without keys is not zero"
    _close(got, ref, _bound(ref, absv, mag, count, vmax, c["d"], out), what)


def _args(c, out):
    import torch

    o = torch.full(c["q"].shape, 77.0, dtype=_tdt(out), device="cuda")
    return o, (c["q"], _i32(c["cu"]), _i32(c["lens"]), _i32(c["table"]))


# ---------------------------------------------------------------------------
# sinks
# ---------------------------------------------------------------------------

def _sinks(kq, c, window, sinks, out="f16", **kw):
    o, a = _args(c, out)
    kq.kq_kv_attention_sinks("q4_0", *a, dev(c["kc"]), dev(c["vc"]), c["page"], o, window, sinks, **kw)
    return o


@pytest.mark.parametrize("q_dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq, kv, d, page", HEADS)
def test_sinks_single_tokens(kq, hq, kv, d, page, q_dtype):
    lens = [1, 2, 15, 16, 64, 65, 0, 129, 300, 555]
    c = _case(d, [1] * len(lens), lens, hq, kv, d, page, q_dtype)
    for window, sinks in ((33, 4), (64, 70), (100, 1), (1, 1)):
        got = _sinks(kq, c, window, sinks, q_dtype, max_new=1, max_kv=555)
        _hold(c, got, f"window {window} sinks {sinks}", q_dtype, window=window, sinks=sinks)


@pytest.mark.parametrize("q_dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq, kv, d, page", HEADS)
def test_sinks_prompts(kq, hq, kv, d, page, q_dtype):
    new = [1, 37, 0, 64, 5, 3, 9, 150]
    lens = [1, 37, 10, 330, 400, 0, 4, 500]
    c = _case(d + 1, new, lens, hq, kv, d, page, q_dtype, extra_tokens=3)
    for window, sinks, bounds in ((17, 4, True), (40, 130, True), (90, 5, False)):
        kw = dict(max_new=150, max_kv=500) if bounds else {}
        _hold(c, _sinks(kq, c, window, sinks, "bf16", **kw), f"window {window} sinks {sinks}", "bf16", window=window, sinks=sinks)


@pytest.mark.parametrize("d, hq, kv, page", [(64, 4, 2, 16), (128, 8, 2, 128), (256, 4, 2, 64)])
@pytest.mark.parametrize("new, lens", [([1, 1, 1], [5000, 30, 4000]), ([2, 90, 1, 40], [3000, 2500, 7, 1500]), ([300], [4000])])
def test_sinks_split_keys(kq, new, lens, d, hq, kv, page):
    # rows whose keys are shared by workgroups, 16-row and prompt tiles
    c = _case(sum(lens) + d, new, lens, hq, kv, d, page)
    _hold(c, _sinks(kq, c, 2000, 100, "f32", max_new=max(new), max_kv=5000), "split", "f32", window=2000, sinks=100)


def test_no_sinks_no_window(kq):
    # where sinks change nothing the call is kq_kv_attention, bit for bit
    import torch

    c = _case(5, [1, 40, 3], [400, 700, 90], 8, 2, 128, 32)
    o, a = _args(c, "f16")
    caches = dev(c["kc"]), dev(c["vc"])
    for window, sinks in ((50, 0), (0, 9), (1 << 30, 4), (60, 1 << 30), (1 << 40, 1 << 40)):
        kq.kq_kv_attention_sinks("q4_0", *a, *caches, c["page"], o.fill_(77), window, sinks, max_new=40, max_kv=700)
        same = torch.full_like(o, 77.0)
        kq.kq_kv_attention("q4_0", *a, *caches, c["page"], same, window=window if sinks == 0 else 0, max_new=40, max_kv=700)
        assert torch.equal(o, same), (window, sinks)
    # sinks as far as the window: every key, by another path
    _hold(c, _sinks(kq, c, 300, 500, "f32", max_new=40, max_kv=700), "all keys", "f32", window=300, sinks=500)


@pytest.mark.parametrize("new, lens, max_kv", [([1, 1], [3000, 900], 3000), ([1, 1], [3000, 900], 500), ([70, 1], [2000, 500], 2000),
                                               ([70, 40], [2000, 1500], 1 << 20)])
@pytest.mark.parametrize("sinks", [4, 20, 64, 100])
def test_pages_between_sinks_and_window_are_not_read(kq, new, lens, max_kv, sinks):
    # their table entries name no pages, or one full of NaN
    page, window = 16, 203
    c = _case(8, new, lens, 4, 2, 64, page)
    want = _f64(_sinks(kq, c, window, sinks, max_new=max(new), max_kv=max_kv))
    _hold(c, _sinks(kq, c, window, sinks, "f32", max_new=max(new), max_kv=max_kv), "whole table", "f32", window=window, sinks=sinks)
    spare = np.nonzero(~np.isin(np.arange(c["kc"].shape[0]), c["table"]))[0][0]
    assert np.isnan(kvcache.load(c["vc"], page, 64, [spare * page])).all()
    was = c["table"].copy()
    for fill in (-1, spare, 1 << 30):
        for s, (m, n) in enumerate(zip(new, lens)):
            c["table"][s, -(-sinks // page):(n - m - window + 1) // page] = fill
        assert np.array_equal(_f64(_sinks(kq, c, window, sinks, max_new=max(new), max_kv=max_kv)), want)
        c["table"] = was.copy()


def test_sinks_need_no_more_workspace_than_attention(kq):
    # the bytes that kq_kv_attention_workspace names are enough whatever window and sinks are
    import torch

    rng = np.random.default_rng(12)
    for i in range(40):
        n, kv, group, d = int(rng.integers(1, 20)), int(rng.choice([1, 2, 8])), int(rng.choice([1, 4, 7])), int(rng.choice([32, 128, 256]))
        new = rng.integers(1, int(rng.choice([2, 30, 300])), n)
        c = _case(i, new, new + 5, kv * group, kv, d, 16)
        max_kv, window, sinks = (int(2 ** rng.uniform(0, 20)) for _ in range(3))
        need = kq.kq_kv_attention_workspace(int(new.sum()), n, kv * group, kv, d, int(new.max()), max_kv)
        ws = torch.empty(max(1, need), dtype=torch.uint8, device="cuda")
        got = _sinks(kq, c, window, sinks, "f32", max_new=int(new.max()), max_kv=max_kv, workspace=ws)
        if i % 8 == 0:
            _hold(c, got, "in that workspace", "f32", window=window, sinks=sinks)


# ---------------------------------------------------------------------------
# a shared prefix
# ---------------------------------------------------------------------------

def _shared(seed, new, own, n_prefix, hq, kv, d, page, q_dtype="f16", apart=(), q_scale=1.0, extra_tokens=0):
    """A batch whose requests share n_prefix pages and hold own[s] keys behind them (those in `apart`: own[s] keys of
    their own and no prefix)."""
    lens = [m if s in apart else n_prefix * page + m for s, m in enumerate(own)]
    c = _case(seed, new, lens, hq, kv, d, page, q_dtype, q_scale, extra_tokens)
    first = next(s for s in range(len(own)) if s not in apart)
    prefix = c["table"][first, :n_prefix].copy()
    for s in range(len(own)):
        if s not in apart:
            c["table"][s, :n_prefix] = -5  # (not read)
    c["prefix"] = prefix
    return c


def _prefix(kq, c, out="f16", **kw):
    o, a = _args(c, out)
    kq.kq_kv_attention_prefix("q4_0", *a, _i32(c["prefix"]), dev(c["kc"]), dev(c["vc"]), c["page"], o, **kw)
    return o


def _check_prefix(kq, c, what, out="f16", scale=None, **kw):
    _hold(c, _prefix(kq, c, out, scale=scale, **kw), what, out, scale, prefix=c["prefix"])


@pytest.mark.parametrize("q_dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq, kv, d, page", HEADS)
def test_prefix_single_tokens(kq, hq, kv, d, page, q_dtype):
    own = [1, 2, 15, 16, 17, 64, 0, 65, 130, 9]
    c = _shared(d, [1] * len(own), own, 5 if page < 128 else 1, hq, kv, d, page, q_dtype, apart=(6, 9))
    bounds = dict(max_new=1, max_kv=int(c["lens"].max()))
    _check_prefix(kq, c, "host bounds", q_dtype, **bounds)
    _check_prefix(kq, c, "no bounds", "f32")


@pytest.mark.parametrize("q_dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq, kv, d, page", HEADS)
def test_prefix_prompts(kq, hq, kv, d, page, q_dtype):
    new = [1, 37, 0, 64, 5, 3, 9, 100]
    own = [1, 37, 10, 130, 200, 0, 4, 100]
    c = _shared(d + 1, new, own, 9 if page < 128 else 2, hq, kv, d, page, q_dtype, apart=(2, 4, 5, 6), extra_tokens=3)
    bounds = dict(max_new=100, max_kv=int(c["lens"].max()))
    _check_prefix(kq, c, "host bounds", q_dtype, **bounds)
    _check_prefix(kq, c, "no bounds", "bf16")


@pytest.mark.parametrize("d, hq, kv, page", [(64, 4, 2, 16), (128, 8, 2, 128), (96, 3, 3, 64), (256, 4, 2, 32)])
@pytest.mark.parametrize("new, own, keys", [([1] * 3, [5, 1, 1], 4000), ([1] * 70, [3] * 70, 1000), ([2, 90, 1], [2100, 90, 1500], 256),
                                            ([1, 1], [3000, 1700], 128), ([300], [300], 640), ([6] * 9, [6] * 9, 144),
                                            ([200, 3], [2500, 1800], 256)])
def test_prefix_split_keys(kq, new, own, keys, d, hq, kv, page):
    # prefixes cut into parts, own keys shared by workgroups, and both
    c = _shared(sum(own) + d, new, own, max(1, keys // page), hq, kv, d, page)
    _check_prefix(kq, c, "split", "f32", max_new=max(new), max_kv=int(c["lens"].max()))


def _long(seed, new, own, n_prefix, hq, kv, d, page, q_dtype, apart):
    """_shared with rows of any codes, written page by page."""
    import torch

    rng = np.random.default_rng(seed)
    held = -(-own // page)
    pages = n_prefix + int(held.sum()) + 2
    caches = []
    for _ in range(2):
        codes = rng.integers(0, 256, (pages, kv, page * d // 2), dtype=np.uint8)
        scales = rng.uniform(0.1, 0.3, (pages, kv, page * d // 32)).astype(np.float16)
        caches.append(np.concatenate((codes, scales.view(np.uint8)), -1))
    ids = rng.permutation(pages)
    table, at = np.full((len(new), n_prefix + int(held.max())), -5), n_prefix
    for s, m in enumerate(held):
        b = 0 if s in apart else n_prefix
        table[s, b:b + m] = ids[at:at + m]
        at += m
        if own[s] % page:  # behind the last key: NaN
            for c in caches:
                tail = c[ids[at - 1], :, page * d // 2:].reshape(kv, page, -1)
                tail[:, own[s] % page:] = 255
                c[ids[at - 1], :, page * d // 2:] = tail.reshape(kv, -1)
    lens = own + np.where(np.isin(np.arange(len(new)), apart), 0, n_prefix * page)
    q = torch.from_numpy(rng.standard_normal((sum(new) + 2, hq, d)).astype(np.float32)).to(device="cuda", dtype=_tdt(q_dtype))
    return dict(q=q, cu=np.concatenate(([0], np.cumsum(new))), lens=lens, table=table, kc=caches[0], vc=caches[1], page=page, d=d,
                prefix=ids[:n_prefix].copy())


def _check_prefix_on_gpu(kq, c, what, out, scale=None, **kw):
    """_check_prefix with the reference as float64 products of a request at a time on the GPU, for prefixes so long that
    prompt tiles take them."""
    import torch

    page, d, pages = c["page"], c["d"], c["kc"].shape[0]
    q, prefix = c["q"].double(), c["prefix"]
    tokens, hq, _ = q.shape
    kv = c["kc"].shape[1]
    sc = d ** -0.5 if scale is None else float(np.float32(scale))
    ref, absv = torch.full_like(q, np.nan), torch.zeros_like(q)
    mag, count = (torch.zeros((tokens, hq), dtype=torch.float64, device="cuda") for _ in range(2))

    def rows(ids):
        there = np.repeat((ids >= 0) & (ids < pages), page)
        slots = np.repeat(np.where((ids >= 0) & (ids < pages), ids, 0), page) * page + np.tile(np.arange(page), len(ids))
        k, v = (torch.from_numpy(kvcache.load(x, page, d, slots)).cuda() for x in (c["kc"], c["vc"]))
        there = torch.from_numpy(there).cuda()
        return [torch.where(there[:, None, None], x, 0.0).transpose(0, 1).contiguous() for x in (k, v)] + [there]

    shared = rows(prefix)
    for s, length in enumerate(c["lens"]):
        a, b = int(c["cu"][s]), int(c["cu"][s + 1])
        at = len(prefix) if length - (b - a) >= len(prefix) * page else 0
        k, v, there = rows(c["table"][s, at:])
        if at:
            k, v, there = (torch.cat((x, y), -1 if x.dim() == 1 else 1) for x, y in zip(shared, (k, v, there)))
        k, v, there = k[:, :length], v[:, :length], there[:length]
        x = q[a:b].unflatten(1, (kv, hq // kv)).permute(1, 2, 0, 3).flatten(1, 2)  # [kv, group * n, d]
        p = torch.arange(length - (b - a), length, device="cuda").repeat(hq // kv)
        see = (torch.arange(k.shape[1], device="cuda") <= p[:, None]) & there
        w = torch.where(see, x @ k.transpose(1, 2).contiguous() * sc, -torch.inf)
        top = w.amax(-1, keepdim=True)
        w = torch.exp(w - torch.where(top == -torch.inf, 0.0, top))
        w = w / w.sum(-1, keepdim=True).clamp(min=1e-300)
        back = lambda y: y.unflatten(1, (hq // kv, b - a)).permute(2, 0, 1, *range(3, y.dim() + 1)).flatten(1, 2)
        ref[a:b], absv[a:b] = back(w @ v), back(w @ v.abs())
        mag[a:b] = back(torch.where(see, x.abs() @ k.abs().transpose(1, 2).contiguous() * abs(sc), 0.0).amax(-1))
        count[a:b] = back(see.sum(-1).expand(kv, -1).double())
    got = _f64(_prefix(kq, c, out, scale=scale, **kw))
    ref, absv, mag, count = (x.cpu().numpy() for x in (ref, absv, mag, count))
    none = np.isnan(ref)
    assert (got[none] == 77).all()
    ref[none] = got[none]
    vmax = np.nanmax(np.abs(kvcache.load(c["vc"], page, d, np.arange(pages * page))))
    assert not got[(count == 0) & ~none.any(-1)].any()
    _close(got, ref, _bound(ref, absv, mag, count, vmax, d, out), what)


@pytest.mark.parametrize("d, hq, kv, page, keys, new, q_dtype", [
    (128, 32, 8, 64, 16384, [1] * 40, "f16"), (256, 16, 4, 128, 8192, [2] * 30, "bf16"), (64, 7, 1, 16, 4816, [700, 1, 3], "bf16"),
    (96, 6, 3, 32, 10016, [1, 250, 49], "f16"), (32, 8, 4, 64, 23040, [1] * 256, "f16"), (160, 8, 4, 64, 4800, [1] * 256, "bf16"),
    (192, 8, 4, 16, 4016, [1] * 256, "f16"), (224, 8, 4, 64, 4160, [3] * 90, "f16"), (128, 8, 8, 256, 16384, [1] * 90, "bf16")])
def test_prefix_of_many_rows(kq, d, hq, kv, page, keys, new, q_dtype):
    # as much work over the prefix as prompt tiles take: rows that fill tiles in part, in full and several
    rng = np.random.default_rng(d + len(new))
    own = np.maximum(rng.integers(1, 60, len(new)), new)
    own[-1] += 400
    apart = (1,) if len(new) > 2 else ()
    c = _long(d, new, own, keys // page, hq, kv, d, page, q_dtype, apart)
    bounds = dict(max_new=max(new), max_kv=int(c["lens"].max()))
    _check_prefix_on_gpu(kq, c, "float32", "f32", **bounds)
    _check_prefix_on_gpu(kq, c, "mean", q_dtype, scale=0.0, **bounds)
    c["prefix"][[0, 7, -1]] = [-1, 1 << 30, c["kc"].shape[0]]
    _check_prefix_on_gpu(kq, c, "pages that are none", q_dtype, **bounds)


def test_both_references_agree(kq):
    c = _shared(3, [1, 5, 2, 9], [4, 5, 80, 3], 5, 4, 2, 64, 16, apart=(3,), extra_tokens=1)
    _check_prefix(kq, c, "oracle", "f32", max_new=9, max_kv=160)
    _check_prefix_on_gpu(kq, c, "on the GPU", "f32", max_new=9, max_kv=160)


def test_prefix_uniform_weights_count_every_key_once(kq):
    c = _shared(50, [1, 1, 3, 70, 1], [30, 1, 66, 200, 5], 21, 8, 2, 128, 16)
    _check_prefix(kq, c, "mean", "f32", scale=0.0, max_new=70, max_kv=540)
    _check_prefix(kq, c, "mean, no bounds", "f32", scale=0.0)


@pytest.mark.parametrize("new, own", [([1, 1, 1], [9, 200, 1]), ([90, 1], [90, 30])])
def test_prefix_pages_that_are_none(kq, new, own):
    # keys of entries that name no page are left out; a prefix of such alone is like none
    c = _shared(7, new, own, 12, 4, 2, 64, 16)
    bounds = dict(max_new=max(new), max_kv=int(c["lens"].max()))
    c["prefix"][[0, 3, 11]] = [-1, 1 << 30, c["kc"].shape[0]]
    _check_prefix(kq, c, "some", "f16", **bounds)
    c["prefix"][:] = -1
    _check_prefix(kq, c, "all", "f16", **bounds)


@pytest.mark.parametrize("scale, q_scale", [(20.0, 200.0), (-20.0, 200.0), (3e38, 1.0)])
def test_prefix_large_logits(kq, scale, q_scale):
    # logits far apart: the row is the value of its largest key, in the prefix or behind it
    c = _shared(70, [1, 1, 40], [40, 3, 90], 8, 8, 2, 64, 16, q_scale=q_scale)
    got, ref = _f64(_prefix(kq, c, "f32", scale=scale, max_new=40, max_kv=250)), kvcache.attention(
        _f64(c["q"]), c["cu"], c["lens"], c["table"], c["kc"], c["vc"], 16, float(np.float32(scale)), prefix=c["prefix"])
    assert np.isfinite(got).all()
    # products are off by 2^-11 of the largest at most; rows whose two largest are nearer than that say nothing
    sure = 0
    for t in range(got.shape[0]):
        for h in range(got.shape[1]):
            sure += np.abs(got[t, h] - ref[t, h]).max() <= 2.0 ** -10 * np.abs(ref[t, h]).max()
    assert sure >= 0.97 * got.shape[0] * got.shape[1]


def test_prefix_of_a_part_of_the_batch(kq):
    # requests 2 and 3 of four share a prefix: a call of their own, on slices, writes only their rows
    import torch

    c = _shared(90, [1, 3, 2, 5, 1], [30, 90, 7, 60, 4], 6, 4, 2, 128, 16, apart=(0, 1, 4))
    o, (q, cu, lens, table) = _args(c, "f16")
    kq.kq_kv_attention_prefix("q4_0", q, cu[2:5], lens[2:4], table[2:4], _i32(c["prefix"]), dev(c["kc"]), dev(c["vc"]), 16, o,
                              max_new=5, max_kv=160)
    torch.cuda.synchronize()
    assert (o[:4] == 77).all() and (o[11:] == 77).all()
    whole = _prefix(kq, c, "f16", max_new=5, max_kv=160)
    ref = _f64(whole)[4:11]
    assert np.abs(_f64(o)[4:11] - ref).max() <= 2.0 ** -9 * np.abs(ref).max()


def test_prefix_pages_behind_32_bits(kq):
    # the same rows in pages whose byte offsets pass 2^32
    import torch

    c = _shared(33, [1, 20, 1], [3, 40, 200], 4, 64, 64, 128, 64)
    near = _prefix(kq, c, "f16", max_new=20, max_kv=460)
    few, page_bytes = c["kc"].shape[0], c["kc"].shape[1] * c["kc"].shape[2]
    pages = (1 << 32) // page_bytes + few + 3
    kc, vc = (torch.zeros((pages, *x.shape[1:]), dtype=torch.uint8, device="cuda") for x in (c["kc"], c["vc"]))
    kc[-few:], vc[-few:] = dev(c["kc"]), dev(c["vc"])
    up = lambda t: _i32(np.where(np.asarray(t) >= 0, np.asarray(t) + pages - few, -1))
    o, (q, cu, lens, _) = _args(c, "f16")
    kq.kq_kv_attention_prefix("q4_0", q, cu, lens, up(c["table"]), up(c["prefix"]), kc, vc, 64, o, max_new=20, max_kv=460)
    assert torch.equal(o, near)


def test_two_calls_at_once(kq):
    # prefix calls on two streams, a workspace each
    import torch

    cs = [_shared(40 + i, [1] * 9, list(range(1, 10)), 30, 8, 2, 64, 16) for i in range(2)]
    sizes = 9, 9, 8, 2, 64, 480, 1, 489
    want = [_prefix(kq, c, "f32", max_new=1, max_kv=489) for c in cs]
    args = [_args(c, "f32") for c in cs]
    more = [(_i32(c["prefix"]), dev(c["kc"]), dev(c["vc"])) for c in cs]
    ws = [torch.empty(kq.kq_kv_attention_prefix_workspace(*sizes), dtype=torch.uint8, device="cuda") for _ in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(20):
        for (o, a), m, w, st in zip(args, more, ws, streams):
            with torch.cuda.stream(st):
                kq.kq_kv_attention_prefix("q4_0", *a, *m, 16, o, max_new=1, max_kv=489, workspace=w)
    torch.cuda.synchronize()
    for (o, _), w in zip(args, want):
        assert torch.equal(o, w)


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

HQ, KV, D, PAGE, PAGES, ROWS, WIDTH = 8, 2, 64, 16, 80, 5, 12


def test_serving_steps_together(kq):
    """A prompt, four samples of it, steps on the shared pages, a window that moves on, a compaction."""
    import torch

    rng = np.random.default_rng(4)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
    kc, vc = kq.kv_cache("q4_0", PAGES, KV, PAGE, D)
    table = torch.full((ROWS, WIDTH), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(PAGES, dtype=torch.int32, device="cuda")
    free = torch.from_numpy(rng.permutation(PAGES).astype(np.int32)).cuda()
    head = i32(0)
    freq, m = kq.kq_rope_freqs(D, 1e4, "yarn", 4.0, 512)
    ctx = torch.zeros(ROWS, dtype=torch.int32, device="cuda")

    def step(new):
        """One step of the batch: tables, rotation in place, store; its queries, offsets and lengths."""
        nonlocal head, ctx
        tokens = sum(new)
        slots, cu, lens, head, st = kq.block_tables(ctx, i32(*new), free, head, PAGE, table, tokens)
        assert st.item() == 0
        qkv = torch.from_numpy(rng.standard_normal((tokens, HQ + 2 * KV, D)).astype(np.float16)).cuda()
        q, k, v = qkv[:, :HQ], qkv[:, HQ:HQ + KV], qkv[:, HQ + KV:]
        was = qkv.clone()
        kq.kq_rope(q, k, cu, lens, freq, mscale=m)
        pos = kvcache.positions(host(cu), host(lens), tokens)
        ref = kvcache.rope(_f64(was[:, :HQ + KV]), pos, host(freq), "half", m)
        assert np.abs(_f64(qkv[:, :HQ + KV]) - ref).max() <= 2.0 ** -10 * np.abs(ref).max()
        kq.kq_kv_store("q4_0", k, v, slots, kc, vc, PAGE)
        ctx = lens
        return q, cu, lens

    def case(q, cu, lens):
        return dict(q=q, cu=host(cu), lens=host(lens), table=host(table), kc=host(kc), vc=host(vc), page=PAGE, d=D)

    def attend(fn, *a, **kw):
        o = torch.full((a[0].shape[0], HQ, D), 77.0, dtype=torch.float16, device="cuda")
        fn("q4_0", *a, kc, vc, PAGE, o, **kw)
        return o

    # the prompt of request 0
    q, cu, lens = step([70, 0, 0, 0, 0])
    _hold(case(q, cu, lens), attend(kq.kq_kv_attention, q, cu, lens, table), "prompt", "f16")
    # requests 1 to 4 continue from it, the last from its 64th token; the ends are copied
    src, dst, head, st = kq.kv_fork(i32(0, 0, 0, 0), i32(1, 2, 3, 4), i32(70, 70, 70, 64), PAGE, table, refs, free, head)
    kq.kq_kv_copy_pages(src, dst, kc, vc)
    assert st.item() == 0 and host(refs).sum() == 4 * 4 and (host(dst) >= 0).tolist() == [True, True, True, False]
    ctx = i32(70, 70, 70, 70, 64)
    prefix = table[0, :4].clone()
    for new in ([1, 1, 1, 1, 1], [0, 3, 1, 1, 40], [1] * 5):
        q, cu, lens = step(new)
        c = case(q, cu, lens)
        c["prefix"] = host(prefix)
        plain = attend(kq.kq_kv_attention, q, cu, lens, table)
        shared = attend(kq.kq_kv_attention_prefix, q, cu, lens, table, prefix)
        _hold(c, plain, "every request by itself", "f16")
        _hold(c, shared, "over the prefix", "f16", prefix=c["prefix"])
    # request 2 ends; the others keep 4 tokens and a window of 20: pages between go back
    n = host(lens)
    first = [1, 1, 0, 1, 1]
    last = [int((x - 20) // PAGE) for x in n]
    last[2] = -(-int(n[2]) // PAGE)
    before = host(head).item()
    head, st = kq.kv_free(i32(*first), i32(*last), table, refs, free, head)
    assert st.item() == 0 and host(head).item() < before
    for s in range(ROWS):
        table[s, first[s]:last[s]] = -1
    lens = lens.clone()
    lens[2] = 0
    c = case(q, cu, lens)
    got = attend(kq.kq_kv_attention_sinks, q, cu, lens, table, window=20, sinks=4)
    _hold(c, got, "sinks and window", "f16", window=20, sinks=4)
    # held pages to the front: rows read the same, bit for bit
    count = PAGES - (PAGES - host(head).item())
    remap, src, dst, st = kq.kv_compact(free, head, table, refs)
    kq.kq_kv_copy_pages(src, dst, kc, vc)
    assert st.item() == 0 and host(table).max() < count and host(head).item() == count
    assert sorted(host(free)[count:].tolist()) == list(range(count, PAGES))
    kc[count:], vc[count:] = 255, 255  # (nothing there is read)
    again = attend(kq.kq_kv_attention_sinks, q, cu, lens, table, window=20, sinks=4)
    assert torch.equal(got, again)
    holders = np.bincount(host(table)[host(table) >= 0], minlength=PAGES)
    assert (np.maximum(holders - 1, 0) == host(refs)).all()


def _all_calls(kq):
    """Calls of every operator on one set of buffers, and the buffers they write."""
    import torch

    rng = np.random.default_rng(6)
    c = _shared(30, [1, 3, 1], [700, 1300, 40], 6, HQ, KV, D, PAGE)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
    fill = lambda *s: torch.full(s, -99, dtype=torch.int32, device="cuda")
    q, cu, lens, table, pre = c["q"], _i32(c["cu"]), _i32(c["lens"]), _i32(c["table"]), _i32(c["prefix"])
    kc, vc = dev(c["kc"]), dev(c["vc"])
    pages = kc.shape[0]
    freq = torch.from_numpy(_freq()).cuda()
    b = dict(qo=torch.zeros_like(q), sinks=torch.zeros_like(q), prefix=torch.zeros_like(q), src=fill(2), dst=fill(2),
             head=fill(1), status=fill(1), table2=torch.full((4, 6), -1, dtype=torch.int32, device="cuda"),
             refs=torch.zeros(pages, dtype=torch.int32, device="cuda"), free=torch.arange(pages, dtype=torch.int32, device="cuda"),
             head2=fill(1), status2=fill(1), to=fill(4, 6), ro=fill(pages), fo=fill(pages), remap=fill(pages),
             csrc=fill(pages // 2), cdst=fill(pages // 2), ho=fill(1), kc=torch.randint_like(kc, 256), vc=torch.randint_like(vc, 256))
    b["table2"][0, :3] = i32(5, 1, 9)
    table0, refs0, free0 = b["table2"].clone(), b["refs"].clone(), b["free"].clone()
    parents, children, take, head0, first, last = i32(0, 0), i32(1, 3), i32(40, 32), i32(20), i32(0, 0, 0, 0), i32(0, 3, 0, 1)
    heads = i32(20)
    ws = [torch.empty(kq.kq_kv_attention_workspace(5, 3, HQ, KV, D, 3, 1400), dtype=torch.uint8, device="cuda"),
          torch.empty(kq.kq_kv_attention_prefix_workspace(5, 3, HQ, KV, D, 6 * PAGE, 3, 1400), dtype=torch.uint8, device="cuda")]

    def run(**kw):
        b["table2"].copy_(table0)
        b["refs"].copy_(refs0)
        b["free"].copy_(free0)
        kq.kq_rope(q, None, cu, lens, freq, b["qo"], **kw)
        kq.kq_kv_fork(parents, children, take, PAGE, b["table2"], b["refs"], b["free"], head0, b["src"], b["dst"], b["head"],
                      b["status"], **kw)
        kq.kq_kv_copy_pages(b["src"], b["dst"], b["kc"], b["vc"], **kw)
        kq.kq_kv_free(first, last, b["table2"], b["refs"], b["free"], b["head"], b["head2"], b["status2"], **kw)
        kq.kq_kv_compact(b["free"], heads, b["table2"], b["refs"], b["to"], b["ro"], b["fo"], b["remap"], b["csrc"], b["cdst"],
                         b["ho"], **kw)
        kq.kq_kv_attention_sinks("q4_0", b["qo"], cu, lens, table, kc, vc, PAGE, b["sinks"], 600, 30, max_new=3, max_kv=1400,
                                 workspace=ws[0], **kw)
        kq.kq_kv_attention_prefix("q4_0", b["qo"], cu, lens, table, pre, kc, vc, PAGE, b["prefix"], max_new=3, max_kv=1400,
                                  workspace=ws[1], **kw)

    return run, b, q


def _freq():
    return (1e4 ** (-np.arange(0, D, 2) / D)).astype(np.float32)


def test_both_python_paths_and_streams_give_the_same(kq, monkeypatch):
    import torch

    assert kq._kqcall is not None
    run, b, _ = _all_calls(kq)
    run()
    torch.cuda.synchronize()
    want = {n: x.clone() for n, x in b.items()}
    assert want["sinks"].abs().sum() > 0 and want["prefix"].abs().sum() > 0
    other = torch.cuda.Stream()

    def on_current():
        other.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(other):
            run()

    for what in ("ctypes", "another stream is current", "ctypes, another stream is current"):
        for n, x in b.items():
            if n not in ("kc", "vc"):
                x.zero_()
        torch.cuda.synchronize()
        with monkeypatch.context() as mp:
            if "ctypes" in what:
                mp.setattr(kq, "_kqcall", None)
            run() if what == "ctypes" else on_current()
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(b[n], want[n]), (what, n)


def test_a_given_stream(kq):
    # a call on a stream that is not the current one: after that stream's own work
    import torch

    run, b, q = _all_calls(kq)
    run()
    torch.cuda.synchronize()
    want = b["qo"].clone()
    other, src = torch.cuda.Stream(), q.clone()
    q.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        torch.cuda._sleep(10_000_000)
        q.copy_(src)
    cu, lens = _i32([0, 1, 4, 5]), _i32([796, 1396, 136])
    freq = torch.from_numpy(_freq()).cuda()
    out = torch.zeros_like(q)
    torch.cuda.current_stream().synchronize()
    kq.kq_rope(q, None, cu, lens, freq, out, stream=other)
    other.synchronize()
    assert torch.equal(out, want)


def test_graph_replays_match_eager(kq):
    import torch

    run, b, q = _all_calls(kq)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for i in range(4):
        q.copy_(torch.randn_like(q))
        caches = b["kc"].clone(), b["vc"].clone()
        graph.replay()
        torch.cuda.synchronize()
        got = {n: x.clone() for n, x in b.items()}
        b["kc"].copy_(caches[0])
        b["vc"].copy_(caches[1])
        run()
        torch.cuda.synchronize()
        for n in b:
            assert torch.equal(b[n], got[n]), (i, n)
        torch.zeros(1000, device="cuda").sum().item()


def test_both_python_paths_refuse_the_same(kq, monkeypatch):
    import torch

    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    kc, vc = (torch.zeros((6, 2, kq.kq_kv_page_bytes("q4_0", 16, 64)), dtype=torch.uint8, device="cuda") for _ in range(2))
    q, k = (torch.zeros((3, h, 64), dtype=torch.float16, device="cuda") for h in (4, 2))
    a = dict(q=q, k=k, cu=i32(3), lens=i32(2), freq=torch.zeros(32, device="cuda"), qo=torch.zeros_like(q), ko=torch.zeros_like(k),
             layout="half", m=1.0, parents=i32(2), children=i32(2), take=i32(2), page=16, table=i32(4, 2), refs=i32(9), free=i32(4),
             head=i32(1), src=i32(2), dst=i32(2), ho=i32(1), first=i32(4), last=i32(4), to=i32(4, 2), ro=i32(9), fo=i32(4),
             remap=i32(9), csrc=i32(4), cdst=i32(4), kc=kc, vc=vc, t2=i32(2, 3), prefix=i32(1), out=torch.zeros_like(q), window=8,
             sinks=2, max_new=2, max_kv=48, ws=torch.empty(1 << 20, dtype=torch.uint8, device="cuda"), codec="q4_0")
    ops = {"rope": lambda x: kq.kq_rope(x["q"], x["k"], x["cu"], x["lens"], x["freq"], x["qo"], x["ko"], x["layout"], x["m"]),
           "fork": lambda x: kq.kq_kv_fork(x["parents"], x["children"], x["take"], x["page"], x["table"], x["refs"], x["free"],
                                           x["head"], x["src"], x["dst"], x["ho"]),
           "free": lambda x: kq.kq_kv_free(x["first"], x["last"], x["table"], x["refs"], x["free"], x["head"], x["ho"]),
           "compact": lambda x: kq.kq_kv_compact(x["free"], x["head"], x["table"], x["refs"], x["to"], x["ro"], x["fo"], x["remap"],
                                                 x["csrc"], x["cdst"], x["ho"]),
           "copy": lambda x: kq.kq_kv_copy_pages(x["src"], x["dst"], x["kc"], x["vc"]),
           "sinks": lambda x: kq.kq_kv_attention_sinks(x["codec"], x["q"], x["cu"], x["lens"], x["t2"], x["kc"], x["vc"], x["page"],
                                                       x["out"], x["window"], x["sinks"], max_new=x["max_new"],
                                                       max_kv=x["max_kv"], workspace=x["ws"]),
           "prefix": lambda x: kq.kq_kv_attention_prefix(x["codec"], x["q"], x["cu"], x["lens"], x["t2"], x["prefix"], x["kc"],
                                                         x["vc"], x["page"], x["out"], max_new=x["max_new"],
                                                         max_kv=x["max_kv"], workspace=x["ws"])}
    bad = [("rope", dict(q=q.float())), ("rope", dict(q=q[:2])), ("rope", dict(qo=q[:, :2])), ("rope", dict(ko=k.float())),
           ("rope", dict(q=None)), ("rope", dict(q=None, k=None, qo=None, ko=None)), ("rope", dict(freq=a["freq"].double())),
           ("rope", dict(freq=a["freq"][:31])), ("rope", dict(freq=a["freq"][::2])), ("rope", dict(cu=i32(2))),
           ("rope", dict(lens=a["lens"].long())), ("rope", dict(layout=7)), ("rope", dict(m=float("nan"))), ("rope", dict(qo=q[1:])),
           ("rope", dict(q=q.transpose(0, 1))), ("rope", dict(cu=a["cu"].cpu())), ("rope", dict(q=q.cpu())), ("rope", dict(ko=a["qo"])),
           ("fork", dict(children=i32(3))), ("fork", dict(take=a["take"].float())), ("fork", dict(table=i32(8))),
           ("fork", dict(page=24)), ("fork", dict(ho=a["head"])), ("fork", dict(dst=i32(1))), ("fork", dict(refs=a["refs"][::2])),
           ("fork", dict(src=a["dst"])), ("fork", dict(free=a["free"].cpu())),
           ("free", dict(last=i32(3))), ("free", dict(table=i32(3, 2))), ("free", dict(refs=a["refs"].long())),
           ("free", dict(ho=i32(2))), ("free", dict(free=a["refs"])), ("free", dict(table=i32(2, 4).T)),
           ("compact", dict(to=i32(4, 3))), ("compact", dict(remap=i32(8))), ("compact", dict(csrc=i32(3), cdst=i32(3))),
           ("compact", dict(cdst=i32(3))), ("compact", dict(fo=a["remap"][:4])), ("compact", dict(head=i32(2))),
           ("copy", dict(dst=i32(3))), ("copy", dict(kc=kc.int())), ("copy", dict(vc=vc[1:])), ("copy", dict(vc=kc)),
           ("copy", dict(kc=kc.cpu())), ("copy", dict(src=a["src"].long())), ("copy", dict(kc=kc.transpose(0, 1))),
           ("sinks", dict(sinks=-1)), ("sinks", dict(window=-1)), ("sinks", dict(codec="q8_0")), ("sinks", dict(t2=i32(3, 2))),
           ("sinks", dict(out=q)), ("sinks", dict(max_kv=0)), ("sinks", dict(kc=kc.cpu())),
           ("prefix", dict(prefix=a["prefix"].long())), ("prefix", dict(prefix=i32(0))), ("prefix", dict(prefix=i32(4)[::2])),
           ("prefix", dict(prefix=a["prefix"].cpu())), ("prefix", dict(ws=a["ws"][:64])), ("prefix", dict(ws=a["ws"].cpu())),
           ("prefix", dict(max_new=0)), ("prefix", dict(page=32)), ("prefix", dict(out=a["out"].int()))]
    want = {n: x.clone() for n, x in a.items() if torch.is_tensor(x)}
    for i, (name, kw) in enumerate(bad):
        errors = []
        for module in (kq._kqcall, None):
            with monkeypatch.context() as mp:
                mp.setattr(kq, "_kqcall", module)
                with pytest.raises((ValueError, TypeError, kq.KQError)) as e:
                    ops[name](dict(a, **kw))
                errors.append((e.type, str(e.value)))
        assert errors[0] == errors[1], (i, name, list(kw), errors)
    torch.cuda.synchronize()
    for n, x in want.items():
        assert torch.equal(a[n], x), n
