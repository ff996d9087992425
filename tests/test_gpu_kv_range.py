"""GPU attention over the 4-bit cache where the number types run out of range.

Bounds are derived in each test; the parity tests' own are in ``test_gpu_kv``.
"""

import numpy as np
import pytest

from _gpu import dev
from oracle import kvcache
from test_gpu_kv import _attn, _close, _f64, _tdt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kq():
    from gguf_quant_matmul_amd import kq as mod

    return mod


def _batch(new, lens, hq, kv, d, page, keys, values, q, q_dtype):
    """A batch whose request s holds keys(s), values(s) [lens[s], kv, d] and whose queries are q [tokens, hq, d]."""
    held = [-(-n // page) for n in lens]
    table = np.full((len(lens), max(held)), -1)
    caches = [np.zeros((sum(held) + 1, kv, kvcache.page_bytes(page, d)), np.uint8) for _ in range(2)]
    at = 1
    for s, n in enumerate(lens):
        table[s, :held[s]] = np.arange(at, at + held[s])[::-1]
        at += held[s]
        slots = table[s][np.arange(n) // page] * page + np.arange(n) % page
        for c, x in zip(caches, (keys(s), values(s))):
            kvcache.store(c, page, slots, *kvcache.encode(x.astype(np.float32)))
    return dict(q=dev(q.astype(np.float32)).to(_tdt(q_dtype)), cu=np.concatenate(([0], np.cumsum(new))),
                lens=np.asarray(lens), table=table, kc=caches[0], vc=caches[1], page=page, d=d)


# (new tokens, lengths, max_kv): one workgroup a tile, keys shared by workgroups, prompt tiles, shared prompt tiles
BATCHES = [([1, 1, 1], [1, 70, 330], 330), ([1, 2, 1], [3000, 900, 5], 3000), ([130], [200], 200),
           ([45, 1, 33], [2500, 1700, 33], 2500)]


@pytest.mark.parametrize("q_dtype, q_size, scale", [("f16", 200.0, 20.0), ("f16", 200.0, -20.0), ("f16", 1.0, 3e38),
                                                    ("bf16", 1e30, 1.0), ("bf16", -1e-30, 3e38), ("bf16", 300.0, 3e38)])
@pytest.mark.parametrize("new, lens, max_kv", BATCHES)
def test_large_logits_pick_the_largest(kq, new, lens, max_kv, q_dtype, q_size, scale):
    # Key j is 500 c_j in every place, c_j whole numbers up to 16.  Products are
    # off by (2^-11 + d 2^-23) of the largest, less than a hundredth of the step
    # between two c, and a step is 10^8 and more of a logit: a row is the mean
    # of the values of the largest keys it sees, which are equal bit for bit.
    # Its error is that of the values as float16 and of the float32 sums.
    hq, kv, d, page = 8, 2, 128, 64
    rng = np.random.default_rng(int(max_kv) + len(new))
    sign = 1.0 if q_size * scale > 0 else -1.0
    level = [rng.integers(-16, 17, n) for n in lens]
    for x in level:
        x[:3] = 9
        x[x * sign > 9] = -9 * sign  # (the largest several times)
    c = _batch(new, lens, hq, kv, d, page, lambda s: np.broadcast_to(level[s][:, None, None] * 500.0, (lens[s], kv, d)),
               lambda s: rng.standard_normal((lens[s], kv, d)), np.full((sum(new), hq, d), q_size), q_dtype)
    q = _f64(c["q"])
    ref = kvcache.attention(q, c["cu"], c["lens"], c["table"], c["kc"], c["vc"], page, float(np.float32(scale)))
    got = _f64(_attn(kq, c, "f32", scale, max_new=max(new), max_kv=max_kv))
    vmax = np.abs(kvcache.load(c["vc"], page, d, np.arange(c["vc"].shape[0] * page))).max()
    _close(got, ref, np.full(ref.shape, (2.0 ** -11 + 2.0 ** -16) * vmax), f"{q_dtype} {q_size} scale {scale}")
