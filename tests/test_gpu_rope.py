"""GPU parity of kq_rope.

A result is m (x_i cos a - x_j sin a).  The angle is exact in float64 and
leaves less than 2^-26 there; its float32 rest is off by 2^-25 at most, the
Taylor sums by 2^-24 more, and m times each is rounded once: cosine and sine
are within 2^-23 + 2^-24 of theirs, times m.  The two products' float32
roundings add 2^-23 of (|x_i| + |x_j|) m.  Together 2^-22 (|x_i| + |x_j|) m, then half a
step of the output type.
"""

import numpy as np
import pytest

from _gpu import host
from oracle import kvcache
from test_gpu_kv import HALF_STEP, _close, _f64, _i32, _tdt

pytestmark = pytest.mark.gpu

TINY = {"f32": 2.0 ** -126, "f16": 2.0 ** -25, "bf16": 2.0 ** -126}


@pytest.fixture(scope="module")
def kq():
    from gguf_quant_matmul_amd import kq as mod

    return mod


def _rows(rng, shape, dtype):
    import torch

    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(device="cuda", dtype=_tdt(dtype))


def _freqs(rng, rot):
    return (10000.0 ** (-np.arange(0, rot, 2) / rot) * (1 + 0.01 * rng.random(rot // 2))).astype(np.float32)


def _check(got, x, pos, f, layout, m, dtype, what, untouched=7.0):
    got, x = _f64(got), _f64(x)
    ref = kvcache.rope(x, pos, f, layout, m)
    none = np.isnan(ref)
    assert (got[none] == untouched).all(), f"{what}: rows without a position were written"
    rot = 2 * len(f)
    other = np.zeros(x.shape)  # |x| of each value's partner, and of itself
    if layout == "pairs":
        other[..., 0:rot:2], other[..., 1:rot:2] = abs(x[..., 1:rot:2]), abs(x[..., 0:rot:2])
    else:
        other[..., :rot // 2], other[..., rot // 2:rot] = abs(x[..., rot // 2:rot]), abs(x[..., :rot // 2])
    err = 2.0 ** -22 * m * (abs(x) + other)
    err[..., rot:] = 0
    bound = err + HALF_STEP[dtype] * (np.abs(ref) + err) + TINY[dtype]
    bound[..., rot:] = 0
    ref[none] = got[none]
    bound[none] = 1
    bound[..., rot:] += 1e-300
    _close(got, ref, bound, what)


SHAPES = [(4, 2, 64, 64), (8, 1, 128, 32), (3, 3, 96, 24), (2, 5, 256, 256), (7, 7, 32, 8), (1, 1, 64, 16), (32, 8, 128, 128),
          (16, 2, 160, 40)]


@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("hq, hkv, d, rot", SHAPES)
def test_rows_equal_the_oracle(kq, hq, hkv, d, rot, dtype, layout):
    import torch

    rng = np.random.default_rng(hq + d + rot)
    new, lens, pad = [1, 37, 0, 5, 3], [1, 2 ** 30, 10, 200, 2], 4  # (the last request has fewer keys than tokens)
    cu = np.concatenate(([0], np.cumsum(new)))
    tokens = int(cu[-1]) + pad
    f, m = _freqs(rng, rot), 1.25
    pos = kvcache.positions(cu, lens, tokens)
    args = _i32(cu), _i32(lens), torch.from_numpy(f).cuda()
    q, k = (_rows(rng, (tokens, h, d), dtype) for h in (hq, hkv))
    qo, ko = (torch.full_like(x, 7.0) for x in (q, k))
    kq.kq_rope(q, k, *args, qo, ko, layout=layout, mscale=m)
    _check(qo, q, pos, f, layout, m, dtype, "q")
    _check(ko, k, pos, f, layout, m, dtype, "k")
    # in place, as slices of a fused projection
    qkv = _rows(rng, (tokens, hq + 2 * hkv, d), dtype)
    was = qkv.clone()
    kq.kq_rope(qkv[:, :hq], qkv[:, hq:hq + hkv], *args, layout=layout, mscale=m)
    live = np.array([p is not None for p in pos])
    for a, b in ((0, hq), (hq, hq + hkv)):
        apart = torch.full_like(qkv[:, a:b], 7.0).contiguous()
        kq.kq_rope(was[:, a:b], None, *args, apart, layout=layout, mscale=m)
        assert torch.equal(qkv[:, a:b][torch.from_numpy(live).cuda()], apart[torch.from_numpy(live).cuda()])
    assert torch.equal(qkv[:, hq + hkv:], was[:, hq + hkv:])
    assert torch.equal(qkv[torch.from_numpy(~live).cuda()], was[torch.from_numpy(~live).cuda()])
    # keys alone, queries in place and keys apart
    ko2, q2 = torch.full_like(k, 7.0), q.clone()
    kq.kq_rope(None, k, *args, None, ko2, layout=layout, mscale=m)
    assert torch.equal(ko2, ko)
    kq.kq_rope(q2, k, *args, None, ko2.fill_(7.0), layout=layout, mscale=m)
    assert torch.equal(ko2, ko) and torch.equal(q2[torch.from_numpy(live).cuda()], qo[torch.from_numpy(live).cuda()])


@pytest.mark.parametrize("n, most", [(1, 3000), (63, 9), (64, 1), (65, 1), (300, 5), (4097, 2), (5000, 1)])
def test_requests_are_found(kq, n, most):
    # one head, one pair: each row's position is told by its rotation
    import torch

    rng = np.random.default_rng(n)
    new = rng.integers(0, most + 1, n)
    new[-1] = most
    cu = np.concatenate(([0], np.cumsum(new))) + 2  # (two rows before the first request)
    tokens = int(cu[-1]) + 3
    lens = new + rng.integers(0, 1000, n)
    lens[rng.random(n) < 0.1] = 0  # refused
    f = np.array([1e-3, 0, 0, 0], np.float32)
    q = torch.zeros((tokens, 1, 32), device="cuda")
    q[:, 0, 0] = 1
    out = torch.full_like(q, 7.0)
    kq.kq_rope(q, None, _i32(cu), _i32(lens), torch.from_numpy(f).cuda(), out, layout="pairs")
    got, pos = host(out).astype(np.float64), kvcache.positions(cu, lens, tokens)
    for t, p in enumerate(pos):
        if p is None:
            assert (got[t] == 7).all()
        else:
            assert abs(got[t, 0, 0] - np.cos(p * float(f[0]))) < 3e-7 and abs(got[t, 0, 1] - np.sin(p * float(f[0]))) < 3e-7


def test_offsets_that_are_not_a_batchs(kq):
    import torch

    rng = np.random.default_rng(9)
    q, f = _rows(rng, (10, 2, 64), "f32"), _freqs(rng, 64)
    for cu, lens in (([-3, 2, 9, 100], [5, 7, 30]), ([0, 0, 0, 0], [5, 6, 7]), ([4, 4, 20, 20], [1, 40, 3]),
                     ([0, 3, 6, 10], [-5, 2 ** 31 - 1, 4])):
        out = torch.full_like(q, 7.0)
        kq.kq_rope(q, None, _i32(cu), _i32(lens), torch.from_numpy(f).cuda(), out)
        _check(out, q, kvcache.positions(cu, lens, 10), f, "half", 1.0, "f32", str(cu))


def test_far_positions_and_quarter_turns(kq):
    # angles p f with f = 1 to 2^30, and multiples of pi / 2 as near as float32 frequencies come to them
    import torch

    lens = [1, 2, 3, 1000003, 2 ** 24 + 1, 2 ** 30 - 7, 2 ** 31 - 1]
    f = np.array([1.0, 0.5, np.pi / 2, np.pi / 4, np.pi, 2.0 ** -20, 3.0, 1e-8] * 2, np.float32)
    q = torch.ones((len(lens), 1, 32), device="cuda")
    q[:, :, 16:] = 0.25
    out = torch.full_like(q, 7.0)
    cu = np.arange(len(lens) + 1)
    kq.kq_rope(q, None, _i32(cu), _i32(lens), torch.from_numpy(f).cuda(), out)
    _check(out, q, kvcache.positions(cu, lens, len(lens)), f, "half", 1.0, "f32", "far")


def test_infinities_stay_in_their_pairs(kq):
    import torch

    q = torch.ones((1, 2, 64), dtype=torch.float16, device="cuda")
    q[0, 0, 3], q[0, 0, 9] = float("inf"), float("nan")
    out = torch.empty_like(q)
    kq.kq_rope(q, None, _i32([0, 1]), _i32([50]), torch.full((32,), 0.1, device="cuda"), out)
    bad = ~np.isfinite(host(out.float()))
    assert set(zip(*np.nonzero(bad))) == {(0, 0, 3), (0, 0, 35), (0, 0, 9), (0, 0, 41)}
