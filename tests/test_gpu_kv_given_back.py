"""GPU tests of pages that were given back: what windows leave behind, forks and frees of requests whose entries still name
such pages."""

import numpy as np
import pytest

from oracle import kvcache
from test_gpu_kv import _case, _f64
from test_gpu_kv_pages import _free
from test_gpu_kv_sinks_prefix import _args, _hold, _sinks, dev

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
