"""GPU tests of pages that were given back: what windows leave behind, forks and frees of requests whose entries still name
such pages."""

import numpy as np
import pytest

from oracle import kvcache
from test_gpu_kv import _case, _f64
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
