"""GPU attention over the 4-bit cache where the number types run out of range.

Bounds are derived in each test; the parity tests' own are in ``test_gpu_kv``.
"""

import numpy as np
import pytest

from _gpu import dev
from oracle import kvcache
from test_gpu_kv import HALF_STEP, _attn, _close, _f64, _tdt

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


@pytest.mark.parametrize("gap", [10.0, 16.0, 17.5, 20.0])
@pytest.mark.parametrize("hq, kv, d, q_dtype", [(4, 2, 128, "f16"), (6, 1, 64, "bf16")])
@pytest.mark.parametrize("new, lens, max_kv, at", [([1], [4096], 512, 0), ([1, 1], [4096, 3000], 4096, 0),
                                                   ([130], [4000], 200000, 0), ([130], [4000], 4000, 1500),
                                                   ([40, 1, 35], [4000, 3000, 2100], 4000, 70)])
def test_many_small_weights_beside_a_large_one(kq, new, lens, max_kv, at, hq, kv, d, q_dtype, gap):
    # Key `at` has logit `gap` and value 0, all others logit 0: the output is
    # what the small weights add up to.  A probability is off by 2^-11 of
    # itself or, as a subnormal float16, by 2^-25 where the largest is 2^7, so
    # by 2^-32 of the largest, in the sum over values and in the sum of
    # weights; logits, values, float32 sums and the store as in the parity
    # tests.
    page = 64
    rng = np.random.default_rng(7)

    def keys(s):
        k = np.zeros((lens[s], kv, d))
        k[at] = 7.0  # (code 15 of scale 1)
        return k

    def values(s):
        v = rng.standard_normal((lens[s], kv, d)) + 2.0
        v[at] = 0
        return v

    scale = gap / (7 * d)
    c = _batch(new, lens, hq, kv, d, page, keys, values, np.ones((sum(new), hq, d)), q_dtype)
    ref, absv, mag, count = kvcache.attention(_f64(c["q"]), c["cu"], c["lens"], c["table"], c["kc"], c["vc"], page,
                                              float(np.float32(scale)), detail=True)
    got = _f64(_attn(kq, c, "f32", scale, max_new=max(new), max_kv=max_kv))
    vmax = np.abs(kvcache.load(c["vc"], page, d, np.arange(c["vc"].shape[0] * page))).max()
    # keys, queries and their products are exact here: a logit is off by the rounding of scale * log2(e) and of the
    # exponent's sum, 2^-22 of itself
    p = absv * (np.expm1(2 * 2.0 ** -22 * mag[..., None]) + 2 * 2.0 ** -11 + 2.0 ** -11 + 2.0 ** -16) * 1.01
    bound = p + 2 * count[..., None] * 2.0 ** -32 * vmax
    _close(got, ref, bound + HALF_STEP["f32"] * (np.abs(ref) + bound), f"gap {gap}")


def test_more_steps_to_share_than_32_bits_count(kq):
    # One request of 2^30 - 4096 keys, one page over and over, 132 tiles of 16
    # rows: 2.2e9 steps.  Keys are 0 and the values the same in every key, so
    # that a row is these values, whoever does its steps.  A wave adds up
    # n = 2.2e9 * 64 / 4096 = 2^25.05 keys of one weight.  The matrix cores
    # align an instruction's products to its largest term, the sum so far, and
    # keep three bits below its last place: the product for key i is off by at
    # most i 2^-26 of itself, their sum by n 2^-27 = 0.26 of itself.  Joining
    # 4096 such sums adds 2^-12 at most.
    import torch

    hq, d, page, tokens = 64, 32, 4096, 33
    width = (1 << 30) // page - 1
    kc, vc = (np.zeros((1, 1, kvcache.page_bytes(page, d)), np.uint8) for _ in range(2))
    v = np.arange(d) % 15 - 7.0  # (scale 1)
    kvcache.store(vc, page, np.arange(page), *kvcache.encode(np.broadcast_to(v, (page, 1, d)).astype(np.float32)))
    q = torch.ones((tokens, hq, d), dtype=torch.float16, device="cuda")
    c = dict(q=q, cu=[0, tokens], lens=[width * page], table=np.zeros((1, width)), kc=kc, vc=vc, page=page)
    got = _f64(_attn(kq, c, "f32", max_new=1, max_kv=width * page))
    assert (np.abs(got - v) <= 0.2605 * np.abs(v)).all()
