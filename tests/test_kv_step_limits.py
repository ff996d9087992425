"""Rotary frequencies at the limits of their divisors (no GPU needed)."""

import numpy as np
import pytest
import torch

kq = pytest.importorskip("gguf_quant_matmul_amd.kq", reason="libkq.so not built")


@pytest.mark.parametrize("small", [1e-45, 1e-39, 9e-31, 0.0, -1.0, float("nan"), float("inf"), 2e30])
def test_divisors_out_of_range_are_refused(small):
    div = torch.ones(32)
    div[5] = small
    with pytest.raises(kq.KQError, match=r"factors\[5\]"):
        kq.kq_rope_freqs(64, factors=div, device="cpu")


@pytest.mark.parametrize("edge", [1e-30, 1e30])
@pytest.mark.parametrize("scaling", [{}, dict(scaling="linear", factor=3.0), dict(scaling="yarn", factor=8.0, original=4096)])
def test_the_smallest_and_largest_divisors_give_finite_frequencies(edge, scaling):
    f, _ = kq.kq_rope_freqs(64, base=10000.0, factors=torch.full((32,), edge), device="cpu", **scaling)
    plain, _ = kq.kq_rope_freqs(64, base=10000.0, device="cpu", **scaling)
    assert torch.isfinite(f).all()
    want = plain.numpy().astype(np.float64) / np.float64(np.float32(edge))
    # two roundings of a frequency, and its smallest steps below float32's normal range
    assert (np.abs(f.numpy() - want) <= 2.0 ** -23 * want + 2.0 ** -149).all()
