"""GPU tests of pages that were given back: what windows leave behind, forks and frees of requests whose entries still name
such pages."""

import numpy as np
import pytest

from _gpu import dev, host
from oracle import kvcache
from test_gpu_kv import _case, _f64, _i32
from test_gpu_kv_pages import _fork, _free
from test_gpu_kv_sinks_prefix import _args, _hold, _sinks

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kq():
    from gguf_quant_matmul_amd import kq as mod

    return mod


# ---------------------------------------------------------------------------
# keys before a window
# ---------------------------------------------------------------------------

def _windowed(kq, c, window, out, **kw):
    o, a = _args(c, out)
    kq.kq_kv_attention("q4_0", *a, dev(c["kc"]), dev(c["vc"]), c["page"], o, window=window, **kw)
    return o


@pytest.mark.parametrize("call", ["window", "no sinks"])
@pytest.mark.parametrize("page, window", [(16, 203), (16, 50), (32, 100), (16, 17)])
@pytest.mark.parametrize("new, lens, max_kv", [([1, 1], [3000, 900], 3000), ([1, 1], [3000, 900], 500), ([70, 1], [2000, 500], 2000),
                                               ([70, 40], [2000, 1500], 1 << 20), ([300], [1111], 1111)])
def test_pages_before_the_window_are_not_read(kq, new, lens, max_kv, page, window, call):
    # a window's first step of 64 keys holds keys, and whole pages, that no row sees any more: given back, their table
    # entries name no pages, or ones full of NaN
    c = _case(9, new, lens, 4, 2, 64, page)
    kw = dict(max_new=max(new), max_kv=max_kv)
    run = lambda out: _windowed(kq, c, window, out, **kw) if call == "window" else _sinks(kq, c, window, 0, out, **kw)
    want = _f64(run("f16"))
    _hold(c, run("f32"), "whole table", "f32", window=window)
    spare = np.nonzero(~np.isin(np.arange(c["kc"].shape[0]), c["table"]))[0][0]
    assert np.isnan(kvcache.load(c["vc"], page, 64, [spare * page])).all()
    was = c["table"].copy()
    for fill in (-1, spare, 1 << 30):
        for s, (m, n) in enumerate(zip(new, lens)):
            c["table"][s, :(n - m - window + 1) // page] = fill
        assert np.array_equal(_f64(run("f16")), want), fill
        c["table"] = was.copy()


# ---------------------------------------------------------------------------
# pages of the free list given back once more
# ---------------------------------------------------------------------------

def test_pages_that_left_with_the_window_and_again_with_the_request(kq):
    # columns 0 .. 3 given back as a window passes, then the whole row: the four stay listed once
    table, refs = np.array([[7, 2, 9, 4, 1, 3]]), np.zeros(12, int)
    refs[9] = 1  # (held by another request too)
    free, head = np.array([5, 8, 7, 2, 4, 1, 3, 0, 6]), 7
    _free(kq, [0], [4], table, refs, free, head, "window")
    refs, free, head, status = kvcache.free([0], [4], table, refs, free, head)
    assert (free[head:], status) == ([2, 4, 7, 0, 6], 0)
    _free(kq, [0], [6], table, refs, free, head, "request")
    refs, free, head, status = kvcache.free([0], [6], table, refs, free, head)
    assert (sorted(free[head:]), status, sum(refs)) == ([0, 1, 2, 3, 4, 6, 7, 9], 1, 0)


@pytest.mark.parametrize("n, width, pages", [(1, 1, 2), (5, 9, 40), (64, 130, 9001), (3, 700, 40000), (2, 3, 70001), (900, 20, 300000)])
def test_listed_pages_given_back(kq, n, width, pages):
    # entries that name held and listed pages, once and several times; counts and list as the oracle's
    rng = np.random.default_rng(pages)
    ids = rng.permutation(pages)
    held = pages // 2
    free = np.concatenate((rng.integers(0, pages, held), ids[held:]))
    refs = np.zeros(pages, int)
    refs[ids[:held:3]] = rng.integers(1, 4, len(ids[:held:3]))
    table = rng.integers(-2, pages + 2, (n, width))
    table[rng.random((n, width)) < 0.2] = ids[-1]
    for head in (held, held + 1, len(free), len(free) + 1, -1):
        _free(kq, rng.integers(0, 2, n), np.full(n, width), table, refs, free, head, f"head {head}")
    _free(kq, np.zeros(n, int), np.zeros(n, int), table, refs, free, held, "nothing given back")
    refs[ids[held:]] = (1 << 27) - 1  # (the largest count)
    refs[ids[:held]] = (1 << 27) - 1
    _free(kq, np.zeros(n, int), np.full(n, width), table, refs, free, held, "largest counts")
    # a list that names pages more than once
    free[held:held + pages // 8] = free[-1 - pages // 8:-1]
    _free(kq, np.zeros(n, int), np.full(n, width), table, np.zeros(pages, int), free, held, "listed twice")


# ---------------------------------------------------------------------------
# forks of requests whose window gave pages back
# ---------------------------------------------------------------------------

def test_forks_of_a_request_whose_middle_was_given_back(kq):
    # request 0 keeps its sinks' column and its window's; the columns between are given back, set to -1, and request 1
    # takes their pages; a fork of request 0 counts the held columns alone, and every page comes back in the end
    page, width, pages, new = 16, 8, 14, 100
    table = np.full((3, width), -1)
    table[0, :7] = [9, 4, 11, 2, 6, 0, 13]
    refs, free, head = np.zeros(pages, int), np.array([-1] * 7 + [1, 3, 5, 7, 8, 10, 12]), 7
    t, r, f, h = _i32(table), _i32(refs), _i32(free), _i32([head])
    i32 = lambda *x: _i32(list(x))

    def state(what, status, want):
        got = [host(x).tolist() for x in (t, r, f[int(host(h)[0]):])]
        for g, w in zip(got, want):
            assert g == w, what
        assert host(status).tolist() == [0], what

    h, st = kq.kv_free(i32(1, 0, 0), i32(4, 0, 0), t, r, f, h)
    t[0, 1:4] = -1
    state("window", st, ([[9, -1, -1, -1, 6, 0, 13, -1], [-1] * 8, [-1] * 8], [0] * pages, [2, 4, 11, 1, 3, 5, 7, 8, 10, 12]))
    _, _, _, h, st = kq.block_tables(i32(0, 0, 0), i32(0, 40, 0), f, h, page, t, 40)
    state("handed out anew", st, ([[9, -1, -1, -1, 6, 0, 13, -1], [2, 4, 11] + [-1] * 5, [-1] * 8], [0] * pages,
                                  [1, 3, 5, 7, 8, 10, 12]))
    src, dst, h, st = kq.kv_fork(i32(0), i32(2), i32(new), page, t, r, f, h)
    assert (host(src).tolist(), host(dst).tolist()) == ([13], [1])
    count = [0] * pages
    for p in (9, 6, 0):
        count[p] = 1
    state("fork", st, ([[9, -1, -1, -1, 6, 0, 13, -1], [2, 4, 11] + [-1] * 5, [9, -1, -1, -1, 6, 0, 1, -1]], count,
                       [3, 5, 7, 8, 10, 12]))
    h, st = kq.kv_free(i32(0, 0, 0), i32(0, 0, width), t, r, f, h)  # the fork ends, then all others
    state("fork ends", st, (host(t).tolist(), [0] * pages, [1, 3, 5, 7, 8, 10, 12]))
    t[2] = -1
    h, st = kq.kv_free(i32(0, 0, 0), i32(width, width, width), t, r, f, h)
    assert host(st).tolist() == [0] and host(h).tolist() == [0] and not host(r).any()
    assert sorted(host(f).tolist()) == list(range(pages))


def test_an_entry_that_was_not_blanked_gives_its_page_a_holder(kq):
    # what the header warns of: the fork cannot tell an entry whose page was given back
    table = [[5, 3, 8, 1], [-1] * 4]
    refs, free, head, status = kvcache.free([1, 0], [3, 0], table, [0] * 10, [0, 0, 7, 9], 2)
    assert (free[head:], status) == ([3, 8, 7, 9], 0)
    _fork(kq, [0], [1], [64], 16, table, refs, free, head, "stale")
    assert kvcache.fork([0], [1], [64], 16, table, refs, free, head)[1][3] == 1
    table[0][1:3] = [-1, -1]
    _fork(kq, [0], [1], [64], 16, table, refs, free, head, "blanked")
    assert kvcache.fork([0], [1], [64], 16, table, refs, free, head)[1][3] == 0
