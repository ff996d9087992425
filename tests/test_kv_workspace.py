"""A workspace of kq_kv_attention_prefix serves every smaller call (no GPU needed)."""

import random

import pytest

kq = pytest.importorskip("gguf_quant_matmul_amd.kq", reason="libkq.so not built")
need = kq.kq_kv_attention_prefix_workspace


def test_a_batch_that_shrinks_needs_no_more():
    # 32 / 8 heads of 128 behind 16384 keys: 64 tokens are cut into more parts than 65 or 96
    sizes = [need(t, t, 32, 8, 128, 16384, 1, 17000) for t in range(1, 300)]
    assert sizes == sorted(sizes)
    # what the sums themselves take at least
    assert all(n >= t * 32 * 130 * 4 for t, n in enumerate(sizes, 1))


@pytest.mark.parametrize("seed", range(40))
def test_no_smaller_size_needs_more(seed):
    rng = random.Random(seed)
    kv, group, d = rng.choice([1, 2, 3, 8, 16, 40, 65]), rng.choice([1, 4, 7, 16]), 32 * rng.randint(1, 8)
    most = [int(2 ** rng.uniform(0, x)) for x in (13, 11, 15, 10, 18)]
    size = lambda tokens, n, prefix, new, keys: need(tokens, n, kv * group, kv, d, prefix, new, keys)
    top = size(*most)
    for _ in range(200):
        assert size(*(rng.randint(1, x) if rng.random() < 0.5 else x for x in most)) <= top
