"""GPU parity of the page operators: everything they write equals the oracle exactly."""

import numpy as np
import pytest

from _gpu import host
from oracle import kvcache
from test_gpu_kv import _i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kq():
    from gguf_quant_matmul_amd import kq as mod

    return mod


def _fill(*shape):
    import torch

    return torch.full(shape, -99, dtype=torch.int32, device="cuda")


def _same(got, want, what):
    for name, (g, w) in zip(want, zip(got, want.values())):
        assert host(g).reshape(-1).tolist() == np.asarray(w).reshape(-1).tolist(), f"{what}: {name}"


# ---------------------------------------------------------------------------
# fork
# ---------------------------------------------------------------------------

def _fork(kq, parents, children, lens, page, table, refs, free, head, what):
    want = kvcache.fork(parents, children, lens, page, table, refs, free, head)
    t, r, n = _i32(table), _i32(refs), len(parents)
    src, dst, ho, st = _fill(n), _fill(n), _fill(1), _fill(1)
    kq.kq_kv_fork(_i32(parents), _i32(children), _i32(lens), page, t, r, _i32(free), _i32([head]), src, dst, ho, st)
    _same((t, r, src, dst, ho, st), dict(zip(("table", "refs", "src", "dst", "head", "status"), want)), what)


@pytest.mark.parametrize("n, parents, page, most", [(1, 1, 16, 1), (8, 1, 16, 330), (3, 2, 64, 5000), (65, 7, 32, 900),
                                                    (700, 30, 16, 200), (4500, 3, 16, 40), (2, 2, 4096, 300000)])
def test_forks_equal_the_oracle(kq, n, parents, page, most):
    rng = np.random.default_rng(n)
    held = rng.integers(1, most + 1, parents)
    width = int(-(-held.max() // page)) + 2
    cols = -(-held // page)
    ids = rng.permutation(int(cols.sum()) + n + 5)
    table, at = np.full((parents + n, width), -1), 0
    for s in range(parents):
        table[s, :cols[s]] = ids[at:at + cols[s]]
        at += cols[s]
    order = rng.permutation(parents + n)  # rows of the batch in any order
    table = table[order]
    row = np.argsort(order)
    p = rng.integers(0, parents, n)
    lens = np.minimum(rng.integers(0, most + 1, n), held[p])
    lens[rng.random(n) < 0.2] = 0
    for extra in (2, -1):  # enough free pages, one too few
        need = int((lens % page > 0).sum())
        free = np.concatenate((np.full(3, -7), ids[at:at + max(0, need + extra)]))
        _fork(kq, row[p], row[parents:], lens, page, table, rng.integers(0, 3, len(ids)), free, 3, f"extra {extra}")


def test_forks_of_odd_inputs(kq):
    table = [[5, 3, 8, -1], [-4, 77, 2, 1], [-1] * 4, [-1] * 4]
    refs = [0] * 10
    _fork(kq, [0, 0, 9, -1, 2, 0, 0], [1, 4, 1, 2, 2, 3, 2], [40, 1, 1, 1, 1, -1, 65], 16, table, refs, [9, 6], 0, "refused")
    _fork(kq, [1, 1], [2, 3], [64, 33], 16, table, refs, [9, 6], 0, "entries that are no pages")
    for head in (2, 3, -1):
        _fork(kq, [0, 0], [2, 3], [32, 33], 16, table, refs, [9, 6], head, f"head {head}")
    _fork(kq, [], [], [], 16, table, refs, [9, 6], 1, "no fork")
    _fork(kq, [0], [2], [5], 16, table, refs, [2 ** 31 - 1], 0, "a fresh id that is no page")
    _fork(kq, [0], [2], [2 ** 31 - 1], 4096, table, refs, [1], 0, "longer than any row")


# ---------------------------------------------------------------------------
# free
# ---------------------------------------------------------------------------

def _free(kq, first, last, table, refs, free, head, what):
    want = kvcache.free(first, last, table, refs, free, head)
    r, f, ho, st = _i32(refs), _i32(free), _fill(1), _fill(1)
    t = _i32(table)
    kq.kq_kv_free(_i32(first), _i32(last), t, r, f, _i32([head]), ho, st)
    _same((r, f, ho, st), dict(zip(("refs", "free", "head", "status"), want)), what)
    assert host(t).tolist() == np.asarray(table).reshape(t.shape).tolist()


@pytest.mark.parametrize("n, width, pages", [(1, 1, 1), (1, 700, 700), (5, 9, 40), (64, 130, 9001), (500, 33, 16384),
                                             (3000, 4, 12001)])
def test_frees_equal_the_oracle(kq, n, width, pages):
    rng = np.random.default_rng(n + width)
    ids = rng.permutation(pages)
    taken = min(pages, n * width) - (1 if pages > 1 else 0)
    table = np.full((n, width), -1)
    table.reshape(-1)[rng.permutation(n * width)[:taken]] = ids[:taken]
    # some pages in a second row as well
    refs = np.zeros(pages, int)
    spots = np.argwhere(table < 0)
    for p, (s, j) in zip(ids[:taken:3], spots):
        table[s, j] = p
        refs[p] += 1
    first = rng.integers(0, width + 1, n)
    last = np.minimum(width, first + rng.integers(0, width + 1, n))
    free = np.concatenate((rng.permutation(pages)[:taken], ids[taken:]))
    _free(kq, first, last, table, refs, free, taken, "some")
    _free(kq, np.zeros(n, int), np.full(n, width), table, refs, free, taken, "all")


def test_frees_of_odd_inputs(kq):
    table = [[2, -1, 99, 0], [2, 3, -7, 4]]
    _free(kq, [-5, 1], [2 ** 31 - 1, 2], table, [0] * 6, [1, 1, 1, 1, 1, 5], 5, "bounds past the row")
    _free(kq, [0, 0], [1, 1], table, [0] * 6, [1, 1, 5], 2, "given back twice")
    _free(kq, [0, 0], [1, 1], table, [0, 0, 1, 0, 0, 0], [1, 1, 5], 2, "given back by both its holders")
    _free(kq, [0, 0], [4, 4], table, [0] * 6, [1, 1, 5], 1, "less room than pages")
    _free(kq, [0, 0], [4, 4], table, [0] * 6, [1, 1, 5], 0, "no room")
    _free(kq, [0, 0], [4, 4], table, [0] * 6, [1, 1, 5], -1, "head before the list")
    _free(kq, [0, 0], [4, 4], table, [0] * 6, [1, 1, 5], 5, "head behind the list")
    _free(kq, [3, 3], [1, 3], table, [0] * 6, [1, 1, 5], 2, "nothing")
    _free(kq, [0, 0], [0, 0], np.zeros((2, 0), int), [0] * 6, [1, 5], 1, "no columns")
    _free(kq, [], [], np.zeros((0, 4), int), [0] * 6, [1, 5], 1, "no rows")
    _free(kq, [0], [4], table[:1], [0] * 6, [], 0, "no list")


def test_a_long_free_list(kq):
    # more pages than the collecting workgroup reads at once, from its first and last
    pages = 300001
    table = np.array([[0, pages - 1, 150000, 8191, 8192]])
    refs = np.zeros(pages, int)
    refs[150000] = 1
    _free(kq, [0], [5], table, refs, np.arange(9), 8, "long")


# ---------------------------------------------------------------------------
# compact
# ---------------------------------------------------------------------------

def _compact(kq, free, head, table, refs, n_copy, what, in_place=True):
    import torch

    want = dict(zip(("table", "refs", "free", "remap", "src", "dst", "head", "status"),
                    kvcache.compact(free, head, table, refs, n_copy)))
    for same in ((False, True) if in_place else (False,)):
        fp, fh, t, r = _i32(free), _i32([head]), _i32(table), _i32(refs)
        to, ro, fo, ho = (t, r, fp, fh) if same else (_fill(len(table)), _fill(len(refs)), _fill(len(free)), _fill(1))
        remap, src, dst, st = _fill(len(refs)), _fill(n_copy), _fill(n_copy), _fill(1)
        kq.kq_kv_compact(fp, fh, t, r, to, ro, fo, remap, src, dst, ho, st)
        torch.cuda.synchronize()
        _same((to, ro, fo, remap, src, dst, ho, st), want, f"{what}, in place {same}")


@pytest.mark.parametrize("pages", [1, 2, 31, 32, 33, 256, 257, 1000, 40000, 262145])
def test_compactions_equal_the_oracle(kq, pages):
    rng = np.random.default_rng(pages)
    for share in (0.0, 0.1, 0.5, 0.9, 1.0):
        held = np.nonzero(rng.random(pages) < share)[0]
        free = np.concatenate((rng.integers(0, pages, 3), rng.permutation(np.setdiff1d(np.arange(pages), held))))
        entries = np.concatenate((rng.permutation(held), [-1, pages, 2 ** 31 - 1, -2 ** 31]))
        if len(free) > 3:
            entries = np.append(entries, free[-1])  # (an entry whose page is free)
        most = min(len(free), pages // 2)
        _compact(kq, free, 3, entries, rng.integers(0, 9, pages), most + 2, f"share {share}")


def test_compactions_of_odd_inputs(kq):
    refs = np.arange(50) % 5
    table = [3, 9, 49, 48, 20, 0]
    _compact(kq, [3, 3, 10, 50, -1, 11, 10], 1, table, refs, 7, "twice, and no pages")
    _compact(kq, [3, 10], 3, table, refs, 2, "head behind the list")
    _compact(kq, [3, 10], -1, table, refs, 2, "head before the list")
    _compact(kq, [3, 10], 2, table, refs, 2, "nothing free")
    _compact(kq, [], 0, table, refs, 0, "no list")
    _compact(kq, np.arange(50), 0, [], refs, 25, "all free, no table")


def test_the_largest_compaction(kq):
    pages = 1 << 20
    rng = np.random.default_rng(0)
    held = rng.random(pages) < 0.7
    free = np.nonzero(~held)[0][::-1]
    _compact(kq, free, 0, np.nonzero(held)[0][::7], rng.integers(0, 3, pages), pages // 2, "2^20 pages", in_place=False)


# ---------------------------------------------------------------------------
# copy
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("pages, heads, page, d", [(9, 1, 16, 32), (40, 2, 16, 64), (300, 5, 32, 96), (12, 8, 64, 128),
                                                   (7, 1, 4096, 256), (5, 3, 512, 224)])
def test_copies(kq, pages, heads, page, d):
    import torch

    rng = np.random.default_rng(pages)
    shape = (pages, heads, kvcache.page_bytes(page, d))
    caches = [rng.integers(0, 256, shape, dtype=np.uint8) for _ in range(2)]
    kc, vc = (torch.from_numpy(c).cuda() for c in caches)
    ids = rng.permutation(pages)
    n = pages // 2
    src, dst = list(ids[:n]), list(ids[n:2 * n])
    for i, (a, b) in enumerate(zip(src, dst)):
        for c in caches:
            c[b] = c[a]
    # pairs that are none
    src += [-1, int(ids[0]), pages, 2 ** 31 - 1, int(ids[0])]
    dst += [int(ids[0]), -1, int(ids[0]), int(ids[0]), pages]
    if n > 1:
        src, dst = src[1:] + src[:1], dst[1:] + dst[:1]
    kq.kq_kv_copy_pages(_i32(src), _i32(dst), kc, vc)
    assert np.array_equal(host(kc), caches[0]) and np.array_equal(host(vc), caches[1])


def test_copies_behind_32_bits(kq):
    # pages whose byte offsets pass 2^32
    import torch

    heads, page, d = 64, 256, 128
    pb = kvcache.page_bytes(page, d)
    pages = (1 << 32) // (heads * pb) + 20
    kc = torch.zeros((pages, heads, pb), dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    kc[3], vc[pages - 2] = 7, 9
    kq.kq_kv_copy_pages(_i32([3, pages - 2]), _i32([pages - 1, 5]), kc, vc)
    assert (kc[pages - 1] == 7).all() and (vc[5] == 9).all() and not vc[pages - 1].any() and not kc[5].any()
    assert kc[:3].sum() == 0 and kc[4:pages - 1].max() == 0
