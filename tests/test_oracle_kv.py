"""Pins of the 4-bit cache oracle (oracle/kvcache.py)."""

import math
from fractions import Fraction

import numpy as np
import pytest

from oracle import codecs, encode, kvcache


def test_encoding_is_the_q4_0_wire_encoding_in_range():
    rng = np.random.default_rng(5)
    x = (rng.standard_normal((40, 96)) * rng.choice([1e-3, 1, 500], (40, 1))).astype(np.float32)
    codes, scales = kvcache.encode(x)
    wire = codecs.dequantize("q4_0", encode.quantize("q4_0", x), 96)
    assert np.array_equal(kvcache.values(codes, scales).astype(np.float32), wire)


def test_encoding_takes_the_nearest_value_exactly():
    rng = np.random.default_rng(6)
    x = rng.standard_normal((3, 32)).astype(np.float16).astype(np.float32)
    x[1] = np.arange(32) / 4 - 4  # many ties: half steps of scale 4 / 7's float16
    x[2, 0], x[2, 1:] = 7, np.clip((np.arange(31) - 15) / 2, -7, 7)  # scale 1: every odd half is a tie
    codes, scales = kvcache.encode(x)
    for i in range(3):
        d = Fraction(float(scales[i, 0]))
        for v, c in zip(x[i], codes[i]):
            dist = [abs(Fraction(float(v)) - d * (k - 8)) for k in range(16)]
            assert c == dist.index(min(dist))
    assert scales[2, 0] == 1 and codes[2, 1:6].tolist() == [1, 1, 1, 2, 2]  # -6.5 and -5.5 tie


def test_encoding_is_total():
    x = np.zeros((6, 32), np.float32)
    x[0, :4] = [np.nan, 1, -2, 0.5]
    x[1, :4] = [np.inf, -np.inf, 65504, 1]
    x[2, 0] = 3e38
    x[3, 0] = 1e-9
    x[5] = np.nan
    codes, scales = kvcache.encode(x)
    v = kvcache.values(codes, scales)
    assert np.isfinite(v).all() and np.abs(v).max() == 65504
    assert v[0, 0] == 0 and v[1, 0] == 57316 and v[1, 1] == -65504 and scales[1, 0] == 8188
    assert not v[3].any() and not v[4].any() and not v[5].any() and (codes[3] == 8).all()


def test_layout_of_a_page():
    page, d = 16, 32
    cache = np.zeros((2, 1, kvcache.page_bytes(page, d)), np.uint8)
    codes = np.arange(32, dtype=np.uint8).reshape(1, 1, 32) % 16
    kvcache.store(cache, page, [16 + 3, ], codes, np.array([[[2.0]]], np.float16))
    assert cache.shape[2] == 16 * 18
    assert not cache[0].any()
    assert cache[1, 0, 48:64].tolist() == [0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE] * 2
    assert cache[1, 0, 256 + 6:256 + 8].tolist() == [0x00, 0x40]
    assert kvcache.load(cache, page, d, [19])[0, 0].tolist() == [2.0 * (c - 8) for c in list(range(16)) * 2]
    before = cache.copy()
    kvcache.store(cache, page, [-1], codes, np.array([[[1.0]]], np.float16))
    kvcache.store(cache, page, [32], codes, np.array([[[1.0]]], np.float16))
    assert np.array_equal(cache, before)


def test_block_tables_by_hand():
    table = [[7, 9, -1, -1], [-1, -1, -1, -1], [3, -1, -1, -1]]
    got = kvcache.block_tables([17, 0, 16], [20, 0, 1], 16, [50, 51, 52, 53], 1, table, 24)
    t, slots, cu, lens, head, status = got
    assert t == [[7, 9, 51, -1], [-1] * 4, [3, 52, -1, -1]]
    assert slots == [9 * 16 + i for i in range(1, 16)] + [51 * 16 + i for i in range(5)] + [52 * 16] + [-1] * 3
    assert cu == [0, 20, 20, 21] and lens == [37, 0, 17] and head == 3 and status == 0


def test_block_tables_refuse():
    table = [[-1, -1] for _ in range(6)]
    # too wide; out of pages; needs none and goes on; past the rows; negative; fits
    t, slots, cu, lens, head, status = kvcache.block_tables([0, 0, 5, 0, -1, 30], [33, 17, 1, 9, 2, 1], 16, [1], 0,
                                                            table, 55)
    assert t == table and status == 1 | 2 | 4 | 8 and head == 0
    assert lens == [0, 0, 6, 0, 0, 0] and cu == [0, 33, 50, 51, 55, 55, 55]
    assert slots == [-1] * 55  # the third request's page id is -1


@pytest.mark.parametrize("window", [0, 5])
def test_attention_against_scalar_loops(window):
    rng = np.random.default_rng(8)
    page, d, hq, kv = 16, 32, 4, 2
    caches = []
    for _ in range(2):
        c = np.zeros((5, kv, kvcache.page_bytes(page, d)), np.uint8)
        kvcache.store(c, page, np.arange(80), *kvcache.encode(rng.standard_normal((80, kv, d)).astype(np.float32)))
        caches.append(c)
    table = np.array([[4, 1], [2, 9], [0, 3]])
    cu, lens = [0, 3, 5, 6], [20, 18, 0]
    q = rng.standard_normal((7, hq, d))
    out = kvcache.attention(q, cu, lens, table, *caches, page, 0.3, window)
    assert np.isnan(out[6]).all() and not out[5].any()
    for s, t in ((0, 0), (0, 2), (1, 4)):
        n, p = cu[s + 1] - cu[s], lens[s] - (cu[s + 1] - cu[s]) + t - cu[s]
        for h in range(hq):
            num, den = np.zeros(d), 0.0
            for j in range(p + 1):
                pid = table[s][j // page]
                if pid >= 5 or (window and j <= p - window):
                    continue
                k, v = (kvcache.load(c, page, d, [pid * page + j % page])[0, h // 2] for c in caches)
                w = math.exp(0.3 * sum(x * y for x, y in zip(q[t, h], k)))
                num, den = num + w * v, den + w
            assert np.allclose(out[t, h], num / den, rtol=1e-12, atol=1e-13), (s, n, t, h)


def test_attention_closed_forms():
    rng = np.random.default_rng(9)
    page, d = 16, 64
    kc, vc = (np.zeros((1, 1, kvcache.page_bytes(page, d)), np.uint8) for _ in range(2))
    rows = rng.standard_normal((2, 9, 1, d)).astype(np.float32)
    for c, r in zip((kc, vc), rows):
        kvcache.store(c, page, np.arange(9), *kvcache.encode(r))
    v = kvcache.load(vc, page, d, np.arange(9))[:, 0]
    q = rng.standard_normal((9, 1, d))
    out = kvcache.attention(q, [0, 9], [9], [[0]], kc, vc, page, 0.0)
    for t in range(9):
        assert np.allclose(out[t, 0], v[:t + 1].mean(0), rtol=1e-13, atol=1e-14)
    # more new tokens than keys: the first ones stand before the first key
    out = kvcache.attention(q, [0, 9], [4], [[0]], kc, vc, page, 1.0)
    assert not out[:5].any() and np.allclose(out[5, 0], v[0])
