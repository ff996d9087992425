"""GPU test of one workspace for batches behind a shared prefix that shrink, and of what a call writes of it."""

import pytest

from test_gpu_kv_sinks_prefix import _check_prefix_on_gpu, _long

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kq():
    from gguf_quant_matmul_amd import kq as mod

    return mod


@pytest.mark.parametrize("hq, kv, d, page, keys, counts, most_new", [(32, 8, 128, 64, 16384, (96, 65, 64, 17, 1), 1),
                                                                     (8, 2, 64, 16, 1008, (40, 9, 2), 30),
                                                                     (4, 4, 256, 32, 256, (5, 3), 200)])
def test_a_workspace_serves_every_smaller_batch(kq, hq, kv, d, page, keys, counts, most_new):
    import numpy as np
    import torch

    rng = np.random.default_rng(d)
    max_kv = keys + 1500
    need = kq.kq_kv_attention_prefix_workspace(counts[0] * most_new, counts[0], hq, kv, d, keys, most_new, max_kv)
    ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    for n in counts:
        new = rng.integers(1, most_new + 1, n)
        own = np.maximum(rng.integers(1, 60, n), new)
        own[-1] += 1200
        c = _long(n, list(new), own, keys // page, hq, kv, d, page, "f16", ())
        c["q"] = c["q"][:int(new.sum())]
        _check_prefix_on_gpu(kq, c, f"{n} requests", "f32", max_new=most_new, max_kv=max_kv, workspace=ws[:need])
        assert (ws[need:] == 0xA5).all()
