"""The Python side of the 4-bit cache operators: which tensors and modules it takes (no GPU needed)."""

import os
import subprocess
import sys

import pytest
import torch

kq = pytest.importorskip("gguf_quant_matmul_amd.kq", reason="libkq.so not built")


def _call(name, dev, **kw):
    """One valid call of an operator on tensors of a device."""
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)
    kc, vc = (torch.zeros((4, 2, kq.kq_kv_page_bytes("q4_0", 16, 64)), dtype=torch.uint8, device=dev) for _ in range(2))
    k, v, q = (torch.zeros((3, h, 64), dtype=torch.float16, device=dev) for h in (2, 2, 4))
    if name == "tables":
        return kq.kq_block_tables(i32(2), i32(2), i32(4), i32(1), 16, i32(2, 2), i32(3), i32(3), i32(2), i32(1), **kw)
    if name == "store":
        return kq.kq_kv_store("q4_0", k, v, i32(3), kc, vc, 16, **kw)
    if name == "load":
        return kq.kq_kv_load("q4_0", kc, vc, i32(3), 16, k, v, **kw)
    return kq.kq_kv_attention("q4_0", q, i32(3), i32(2), i32(2, 2), kc, vc, 16, torch.zeros_like(q), max_new=2,
                              max_kv=32, **kw)


@pytest.mark.parametrize("kw", [{}, {"stream": 0}])
@pytest.mark.parametrize("name", ["tables", "store", "load", "attention"])
def test_host_tensors_are_refused(name, kw):
    with pytest.raises(ValueError, match="on the GPU"):
        _call(name, "cpu", **kw)


def test_host_tensors_are_refused_before_a_workspace_is_made():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    kc, vc = (torch.zeros((4, 2, kq.kq_kv_page_bytes("q4_0", 16, 64)), dtype=torch.uint8) for _ in range(2))
    q = torch.zeros((1, 4, 64), dtype=torch.float16)
    with pytest.raises(ValueError, match="on the GPU"):
        kq.kq_kv_attention("q4_0", q, i32(2), i32(1), i32(1, 2), kc, vc, 16, q.clone(), max_new=1, max_kv=100000,
                           stream=0)


CHILD = """
import sys, types, warnings
what = sys.argv[1]
if what == "missing":
    sys.modules["gguf_quant_matmul_amd._kqcall"] = None  # its import raises ImportError
else:  # built against other headers than the torch that runs
    import gguf_quant_matmul_amd
    fake = types.ModuleType("gguf_quant_matmul_amd._kqcall")
    fake.TORCH = "1.0.0"
    sys.modules[fake.__name__] = gguf_quant_matmul_amd._kqcall = fake
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    from gguf_quant_matmul_amd import kq
import torch
assert any("_kqcall" in str(w.message) for w in seen), seen
assert kq.kq_row_bytes("q4_k", 256) == 144 and kq.kq_kv_page_bytes("q4_0", 16, 64) == 16 * 36
sys.path.insert(0, "tests")
import test_kv_binding as t
for name in ("tables", "store", "load", "attention"):
    try:
        t._call(name, "cpu")
    except ValueError as e:
        assert "on the GPU" in str(e)
    else:
        raise SystemExit(name)
print("ok")
"""


@pytest.mark.parametrize("what", ["missing", "other torch"])
def test_the_library_works_without_its_host_module(what):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-c", CHILD, what], cwd=root, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and res.stdout.strip().endswith("ok"), res.stderr


def test_the_host_module_is_built_for_this_torch():
    assert kq._kqcall is not None and kq._kqcall.TORCH == torch.__version__
