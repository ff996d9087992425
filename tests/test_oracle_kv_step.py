"""Pins of the oracle's pages, rotary positions, sinks and shared prefixes (no GPU needed)."""

import numpy as np
import pytest

from oracle import kvcache


def test_fork_by_hand():
    # pages of 16; request 0 holds 40 tokens in pages 5, 3, 8
    table = [[5, 3, 8, -1], [-1] * 4, [-1] * 4, [-1] * 4]
    t, refs, src, dst, head, status = kvcache.fork([0, 0, 0], [1, 2, 3], [40, 32, 17], 16, table, [0] * 10, [9, 7, 6, 1], 1)
    assert t == [[5, 3, 8, -1], [5, 3, 7, -1], [5, 3, -1, -1], [5, 6, -1, -1]]
    assert refs == [0, 0, 0, 2, 0, 3, 0, 0, 0, 0]
    assert (src, dst, head, status) == ([8, -1, 3], [7, -1, 6], 3, 0)
    # one free page for two that ask; a row that is none, itself, too long, negative
    got = kvcache.fork([0, 0, 0, 9, 0, 0], [1, 2, 3, 1, 0, 1], [1, 2, 16, 1, 1, -1], 16, table, [0] * 10, [9], 0)
    assert got[2:] == ([5, -1, -1, -1, -1, -1], [9, -1, -1, -1, -1, -1], 1, 1 | 4 | 8)
    assert got[0] == [[5, 3, 8, -1], [9, -1, -1, -1], [-1] * 4, [5, -1, -1, -1]]
    assert kvcache.fork([0], [1], [65], 16, table, [0] * 10, [9], 0)[5] == 2


def test_free_by_hand():
    table = [[5, 3, 8], [5, 3, 7], [2, -1, 99]]
    refs, free, head, status = kvcache.free([0, 2, 0], [3, 3, 3], table, [0, 0, 0, 1, 0, 1, 0, 0, 0, 0], [4, 1, 6, 9, 0], 3)
    assert refs == [0] * 10 and status == 0
    assert free == [2, 7, 8, 9, 0] and head == 0
    # given back twice; no room
    refs, free, head, status = kvcache.free([0, 0], [1, 1], [[2], [2]], [0] * 4, [7, 7], 0)
    assert (refs, free, head, status) == ([0] * 4, [7, 7], 0, 3)


def test_free_of_listed_pages_by_hand():
    # page 2 stands in the list: given back once more it stays there once, and that is told
    refs, free, head, status = kvcache.free([0], [2], [[2, 3]], [0] * 5, [0, 4, 2], 1)
    assert (refs, free, head, status) == ([0] * 5, [3, 4, 2], 0, 1)
    # in front of the head it does not count
    refs, free, head, status = kvcache.free([0], [2], [[2, 3]], [0] * 5, [2, 4, 1], 2)
    assert (refs, free, head, status) == ([0] * 5, [2, 3, 1], 0, 0)


def test_compact_by_hand():
    # held: 0, 2, 5, 6 of 7 pages; 5 and 6 go to 1 and 3
    got = kvcache.compact([0, 4, 1, 3], 1, [6, 5, -1, 2, 4, 0], [1, 0, 2, 0, 0, 3, 4], 4)
    assert got == ([3, 1, -1, 2, -1, 0], [1, 3, 2, 4, 0, 0, 0], [0, 4, 5, 6], [0, -1, 2, -1, -1, 1, 3], [5, 6, -1, -1],
                   [1, 3, -1, -1], 1, 0)
    # listed twice, and no page: counted once, told
    got = kvcache.compact([1, 1, 9], 0, [2], [0, 0, 7], 1)
    assert got == ([1], [0, 7, 0], [1, 1, 2], [0, -1, 1], [2], [1], 2, 1)


def test_pages_keep_what_every_request_reads():
    # forks, frees and a compaction at random: the row that each request reads at each of its places never changes
    rng = np.random.default_rng(1)
    page, pages, rows, width = 16, 60, 12, 6
    data = rng.integers(0, 1 << 30, (pages, page))
    table, lens = [[-1] * width for _ in range(rows)], [0] * rows
    refs, free, head = [0] * pages, list(rng.permutation(pages)), 0
    seen = [[] for _ in range(rows)]

    def check():
        holders = np.zeros(pages, int)
        for s in range(rows):
            assert [data[table[s][i // page]][i % page] for i in range(lens[s])] == seen[s]
            for j in range(-(-lens[s] // page)):
                holders[table[s][j]] += 1
        assert [max(0, h - 1) for h in holders] == refs
        assert sorted(free[head:]) == [p for p in range(pages) if holders[p] == 0]

    for step in range(200):
        s = int(rng.integers(rows))
        if lens[s] and rng.random() < 0.4:  # ends
            f, last = [0] * rows, [0] * rows
            last[s] = -(-lens[s] // page)
            refs, free, head, st = kvcache.free(f, last, table, refs, free, head)
            assert st == 0
            lens[s], seen[s], table[s] = 0, [], [-1] * width
        elif lens[s]:
            to = [r for r in range(rows) if lens[r] == 0]
            if to:
                n = int(rng.integers(1, lens[s] + 1))
                table, refs, src, dst, head, st = kvcache.fork([s], [to[0]], [n], page, table, refs, free, head)
                if st == 0:
                    if dst[0] >= 0:
                        data[dst[0]] = data[src[0]]
                    lens[to[0]], seen[to[0]] = n, seen[s][:n]
        elif head < pages - 4:  # a new request
            n = int(rng.integers(1, 50))
            for j in range(-(-n // page)):
                table[s][j] = int(free[head])
                head += 1
            lens[s] = n
            seen[s] = [data[table[s][i // page]][i % page] for i in range(n)]
        if step % 20 == 19:
            flat, refs, free, remap, src, dst, head, st = kvcache.compact(free, head, sum(table, []), refs, pages // 2)
            assert st == 0
            table = [flat[i * width:(i + 1) * width] for i in range(rows)]
            for a, b in zip(src, dst):
                if a >= 0:
                    data[b] = data[a]
            assert sorted(free[head:]) == list(range(pages - len(free[head:]), pages))
        check()


@pytest.mark.parametrize("layout", ["half", "pairs"])
def test_rope_is_a_complex_product(layout):
    rng = np.random.default_rng(2)
    x, f, half = rng.standard_normal((4, 2, 12)), rng.random(4).astype(np.float32), 4
    pos = [7, None, 100000, 0]
    y = kvcache.rope(x, pos, f, layout, 1.5)
    assert np.isnan(y[1]).all()
    z = lambda v: v[:, 0:8:2] + 1j * v[:, 1:8:2] if layout == "pairs" else v[:, :half] + 1j * v[:, half:8]
    for t in (0, 2, 3):
        want = z(x[t]) * 1.5 * np.exp(1j * pos[t] * f.astype(np.float64))
        assert np.allclose(z(y[t]), want, rtol=0, atol=1e-12) and np.array_equal(y[t][:, 8:], x[t][:, 8:])


def test_positions_follow_the_offsets():
    assert kvcache.positions([0, 2, 2, 5], [10, 3, 2], 7) == [8, 9, None, 0, 1, None, None]


def _one(rows, page, kv, d, rng):
    """A cache of `rows` random rows in pages 1.., and the table row of them."""
    pages = -(-rows // page)
    c = [np.zeros((pages + 1, kv, kvcache.page_bytes(page, d)), np.uint8) for _ in range(2)]
    ids = np.arange(1, pages + 1)[::-1]
    slots = ids[np.arange(rows) // page] * page + np.arange(rows) % page
    for x in c:
        kvcache.store(x, page, slots, *kvcache.encode(rng.standard_normal((rows, kv, d)).astype(np.float32)))
    return c, ids


def test_sinks_and_prefix_by_masks():
    rng = np.random.default_rng(3)
    n, page, d = 70, 16, 32
    (kc, vc), ids = _one(n, page, 1, d, rng)
    q = rng.standard_normal((2, 1, d))
    slots = ids[np.arange(n) // page] * page + np.arange(n) % page
    k, v = (kvcache.load(c, page, d, slots)[:, 0] for c in (kc, vc))
    out = kvcache.attention(q, [0, 2], [n], [ids], kc, vc, page, 0.3, window=10, sinks=3)
    for t, p in enumerate((n - 2, n - 1)):
        see = [j for j in range(p + 1) if j > p - 10 or j < 3]
        w = np.exp(0.3 * k[see] @ q[t, 0])
        assert np.allclose(out[t, 0], w @ v[see] / w.sum())
    # the prefix's pages in the place of the table's, for rows behind it only
    full = kvcache.attention(q, [0, 2], [n], [ids], kc, vc, page, 0.3)
    other = np.concatenate(([0, 0], ids[2:]))
    assert np.array_equal(kvcache.attention(q, [0, 2], [n], [other], kc, vc, page, 0.3, prefix=ids[:2]), full)
    with_zeros = kvcache.attention(q, [0, 2], [33], [other], kc, vc, page, 0.3, prefix=ids[:2])
    assert np.array_equal(with_zeros, kvcache.attention(q, [0, 2], [33], [other], kc, vc, page, 0.3))
