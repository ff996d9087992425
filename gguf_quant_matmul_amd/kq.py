"""Thin ctypes binding of libkq (include/kq.h): same names, argument marshalling.

Every function here forwards device pointers, sizes and the current HIP stream
to the C ABI; all work runs in libkq's HIP kernels.  The cache operators also
check their tensors, and go through the host module _kqcall where it is there.  PyTorch supplies device
memory and streams.  There is no fallback: if libkq.so is missing the import
fails, and a failing call raises ``KQError`` with the library's message.
"""

from __future__ import annotations

import ctypes
import os
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libkq.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; run `python -m gguf_quant_matmul_amd.build`")

# torch's HIP runtime must be the only one in the process.  libkq.so asks for
# libamdhip64.so.7 and takes whichever copy of that soname is already loaded;
# torch's own libraries name their bundled copy by another file name, so
# opening libkq.so first would bring in a second HIP runtime that, once torch
# holds the GPU, finds no device.
import torch  # noqa: E402,F401

_lib = ctypes.CDLL(LIB_PATH)


def _host_module():
    """_kqcall (csrc/kq_call.cpp): the cache operators' calls straight from tensors.  None where it is not built, or for
    another torch, whose tensors it would misread; the calls then go through ctypes as all others do."""
    try:
        from . import _kqcall as mod
    except ImportError as e:
        why = str(e)
    else:
        built = getattr(mod, "TORCH", None)
        if built == torch.__version__:
            return mod
        why = f"built for torch {built}, this is {torch.__version__}"
    warnings.warn(f"_kqcall cannot be used ({why}): calls of the cache operators take 4 to 7 us longer; run "
                  "`python -m gguf_quant_matmul_amd.build`", RuntimeWarning, stacklevel=2)
    return None


_kqcall = _host_module()

c_int, c_i64, c_vp, c_cp = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p, ctypes.c_char_p
_P = ctypes.POINTER

_SIGS = {
    "kq_codec_from_name": (c_int, [c_cp, _P(c_int)]),
    "kq_codec_info": (c_int, [c_int, _P(c_int), _P(c_int)]),
    "kq_row_bytes": (c_int, [c_int, c_i64, _P(c_i64)]),
    "kq_last_error": (c_cp, []),
    "kq_version": (c_cp, []),
    "kq_dequantize": (c_int, [c_int, c_vp, c_i64, c_i64, c_vp, c_int, c_vp]),
    "kq_qmv": (c_int, [c_int, c_vp, c_i64, c_i64, c_vp, c_i64, c_vp, c_int, c_vp]),
    "kq_qmm": (c_int, [c_int, c_vp, c_i64, c_i64, c_vp, c_i64, c_vp, c_int, c_vp]),
    "kq_quantized_matmul": (c_int, [c_int, c_vp, c_i64, c_i64, c_vp, c_i64, c_vp, c_int, c_vp]),
    "kq_quantized_matmul_residual": (c_int, [c_int, c_vp, c_i64, c_i64, c_vp, c_i64, c_vp, c_vp, c_i64, c_vp, c_int,
                                             c_vp]),
    "kq_quantized_matmul_qmv_bias": (c_int, [c_int, c_vp, c_i64, c_i64, c_vp, c_i64, c_vp, c_vp, c_int, c_vp]),
    "kq_quantized_matmul_glu": (c_int, [c_int, c_vp, c_vp, c_i64, c_i64, c_vp, c_i64, c_int, c_vp, c_int, c_vp]),
    "kq_expert_tile_map_capacity": (c_i64, [c_i64, c_i64]),
    "kq_expert_tile_map": (c_int, [c_vp, c_i64, c_i64, c_vp, c_vp, c_i64, c_vp, c_vp]),
    "kq_gather_qmm_seg": (c_int, [c_int, c_vp, c_i64, c_i64, c_i64, c_vp, c_i64, c_vp, c_vp, c_i64, c_vp, c_int, c_vp]),
    "kq_gather_qmv": (c_int, [c_int, c_vp, c_i64, c_i64, c_i64, c_vp, c_vp, c_i64, c_vp, c_int, c_vp]),
    "kq_moe_glu_gather": (c_int, [c_int, c_vp, c_vp, c_i64, c_i64, c_i64, c_vp, c_i64, c_vp, c_i64, c_int,
                                  ctypes.c_float, c_vp, c_int, c_vp]),
    "kq_gather_mix": (c_int, [c_vp, c_i64, c_i64, c_vp, c_vp, c_i64, c_i64, c_vp, c_int, c_vp]),
    "kq_quantize": (c_int, [c_int, c_vp, c_i64, c_i64, c_vp, c_vp]),
    "kq_stream_read": (c_int, [c_vp, c_i64, c_vp, c_i64, c_vp]),
    "kq_qmv_bf16": (c_int, [c_int, c_vp, c_i64, c_i64, c_vp, c_i64, c_vp, c_int, c_vp]),
    "kq_qmm_bf16": (c_int, [c_int, c_vp, c_i64, c_i64, c_vp, c_i64, c_vp, c_int, c_vp]),
    "kq_gather_qmm_seg_bf16": (c_int, [c_int, c_vp, c_i64, c_i64, c_i64, c_vp, c_i64, c_vp, c_vp, c_i64, c_vp, c_int,
                                       c_vp]),
    "kq_kv_page_bytes": (c_int, [c_int, c_i64, c_i64, _P(c_i64)]),
    "kq_block_tables": (c_int, [c_vp, c_vp, c_i64, c_i64, c_vp, c_i64, c_vp, c_vp, c_i64, c_vp, c_i64, c_vp, c_vp, c_vp,
                                c_vp, c_vp]),
    "kq_kv_store": (c_int, [c_int, c_vp, c_vp, c_int, c_i64, c_i64, c_i64, c_i64, c_i64, c_vp, c_vp, c_vp, c_i64, c_i64,
                            c_vp]),
    "kq_kv_load": (c_int, [c_int, c_vp, c_vp, c_i64, c_i64, c_i64, c_i64, c_vp, c_i64, c_vp, c_vp, c_int, c_vp]),
    "kq_kv_attention_workspace": (c_int, [c_i64, c_i64, c_i64, c_i64, c_i64, c_i64, c_i64, _P(c_i64)]),
    "kq_kv_attention": (c_int, [c_int, c_vp, c_int, c_i64, c_i64, c_i64, c_i64, c_i64, c_vp, c_vp, c_i64, c_vp, c_i64,
                                c_vp, c_vp, c_i64, c_i64, ctypes.c_float, c_i64, c_i64, c_i64, c_vp, c_int, c_vp, c_i64,
                                c_vp]),
    "kq_kv_attention_sinks": (c_int, [c_int, c_vp, c_int, c_i64, c_i64, c_i64, c_i64, c_i64, c_vp, c_vp, c_i64, c_vp,
                                      c_i64, c_vp, c_vp, c_i64, c_i64, ctypes.c_float, c_i64, c_i64, c_i64, c_i64, c_vp,
                                      c_int, c_vp, c_i64, c_vp]),
    "kq_kv_attention_prefix_workspace": (c_int, [c_i64, c_i64, c_i64, c_i64, c_i64, c_i64, c_i64, c_i64, _P(c_i64)]),
    "kq_kv_attention_prefix": (c_int, [c_int, c_vp, c_int, c_i64, c_i64, c_i64, c_i64, c_i64, c_vp, c_vp, c_i64, c_vp,
                                       c_i64, c_vp, c_i64, c_vp, c_vp, c_i64, c_i64, ctypes.c_float, c_i64, c_i64, c_vp,
                                       c_int, c_vp, c_i64, c_vp]),
    "kq_kv_fork": (c_int, [c_vp, c_vp, c_vp, c_i64, c_i64, c_vp, c_i64, c_i64, c_vp, c_i64, c_vp, c_i64, c_vp, c_vp, c_vp,
                           c_vp, c_vp, c_vp]),
    "kq_kv_free": (c_int, [c_vp, c_vp, c_i64, c_vp, c_i64, c_vp, c_i64, c_vp, c_i64, c_vp, c_vp, c_vp, c_vp]),
    "kq_kv_compact": (c_int, [c_vp, c_i64, c_vp, c_vp, c_i64, c_vp, c_i64, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_i64, c_vp,
                              c_vp, c_vp]),
    "kq_kv_copy_pages": (c_int, [c_vp, c_vp, c_i64, c_vp, c_vp, c_i64, c_i64, c_vp]),
    "kq_rope": (c_int, [c_vp, c_i64, c_i64, c_vp, c_i64, c_i64, c_int, c_i64, c_i64, c_i64, c_int, c_vp, c_vp, c_i64, c_vp,
                        ctypes.c_float, c_vp, c_i64, c_vp, c_i64, c_vp]),
    "kq_rope_freqs": (c_int, [c_i64, ctypes.c_double, c_int, ctypes.c_double, c_i64, ctypes.c_double, ctypes.c_double, c_vp,
                              _P(ctypes.c_float), _P(ctypes.c_float)]),
}

#: every symbol the header declares
EXPORTS = tuple(_SIGS)

for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args

# ids and enums of include/kq.h
KQ_Q4_0, KQ_Q4_1, KQ_Q5_0, KQ_Q5_1, KQ_Q8_0 = 2, 3, 6, 7, 8
KQ_Q2_K, KQ_Q3_K, KQ_Q4_K, KQ_Q5_K, KQ_Q6_K = 10, 11, 12, 13, 14
KQ_F32, KQ_F16, KQ_BF16 = 0, 1, 2
KQ_GLU_SILU, KQ_GLU_GELU_TANH, KQ_GLU_SILU_LIMIT = 0, 1, 2
_GLU_ACTS = {"silu": KQ_GLU_SILU, "gelu": KQ_GLU_GELU_TANH, "gelu_tanh": KQ_GLU_GELU_TANH,
             "silu_limit": KQ_GLU_SILU_LIMIT}
KQ_ROPE_HALF, KQ_ROPE_PAIRS = 0, 1
KQ_ROPE_NONE, KQ_ROPE_LINEAR, KQ_ROPE_NTK, KQ_ROPE_YARN = 0, 1, 2, 3
_ROPE_LAYOUTS = {"half": KQ_ROPE_HALF, "pairs": KQ_ROPE_PAIRS}
_ROPE_SCALINGS = {"none": KQ_ROPE_NONE, "linear": KQ_ROPE_LINEAR, "ntk": KQ_ROPE_NTK, "yarn": KQ_ROPE_YARN}
KQ_OK, KQ_ERR_ARG, KQ_ERR_CODEC, KQ_ERR_SHAPE, KQ_ERR_ALIGN, KQ_ERR_CAPACITY, KQ_ERR_HIP = 0, -1, -2, -3, -4, -5, -6
STATUS_NAMES = {0: "KQ_OK", -1: "KQ_ERR_ARG", -2: "KQ_ERR_CODEC", -3: "KQ_ERR_SHAPE", -4: "KQ_ERR_ALIGN",
                -5: "KQ_ERR_CAPACITY", -6: "KQ_ERR_HIP"}


class KQError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


def _check(status: int) -> None:
    if status != KQ_OK:
        raise KQError(status, _lib.kq_last_error().decode())


def _codec(c) -> int:
    if isinstance(c, str):
        return kq_codec_from_name(c)
    return int(c)


def _ptr(t) -> int | None:
    """Device pointer of a tensor (None for None)."""
    if t is None:
        return None
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is not None:
        return int(stream) if isinstance(stream, int) else stream.cuda_stream
    return torch.cuda.current_stream().cuda_stream


def _dtype_id(t) -> int:
    import torch

    if t.dtype == torch.float32:
        return KQ_F32
    if t.dtype == torch.float16:
        return KQ_F16
    if t.dtype == torch.bfloat16:
        return KQ_BF16
    raise TypeError(f"output dtype must be float32, float16 or bfloat16, got {t.dtype}")


def _bf16(x) -> bool:
    """True for bfloat16 activations (the *_bf16 entry points), False for float16."""
    import torch

    if x.dtype == torch.bfloat16:
        return True
    if x.dtype == torch.float16:
        return False
    raise TypeError(f"activations must be float16 or bfloat16, got {x.dtype}")


# ---------------------------------------------------------------------------
# registry
# ---------------------------------------------------------------------------

def kq_codec_from_name(name: str) -> int:
    out = c_int()
    _check(_lib.kq_codec_from_name(name.encode(), ctypes.byref(out)))
    return out.value


def kq_codec_info(codec) -> tuple[int, int]:
    bv, bb = c_int(), c_int()
    _check(_lib.kq_codec_info(_codec(codec), ctypes.byref(bv), ctypes.byref(bb)))
    return bv.value, bb.value


def kq_row_bytes(codec, k: int) -> int:
    out = c_i64()
    _check(_lib.kq_row_bytes(_codec(codec), k, ctypes.byref(out)))
    return out.value


def kq_last_error() -> str:
    return _lib.kq_last_error().decode()


def kq_version() -> str:
    return _lib.kq_version().decode()


def kq_expert_tile_map_capacity(rows: int, n_experts: int) -> int:
    return int(_lib.kq_expert_tile_map_capacity(rows, n_experts))


# ---------------------------------------------------------------------------
# ops: tensors in, outputs written in place (the caller allocates)
# ---------------------------------------------------------------------------

def kq_dequantize(codec, w, k: int, out, stream=None) -> None:
    """w: uint8 [rows, row_bytes] -> out: float32/float16 [rows, k]."""
    rows = w.shape[0] if w.dim() > 1 else 1
    _check(_lib.kq_dequantize(_codec(codec), _ptr(w), rows, k, _ptr(out), _dtype_id(out), _stream(stream)))


def kq_qmv(codec, w, n: int, k: int, x, y, stream=None) -> None:
    """y[m, n] = x[m, :] . dequant(w)[n, :]; x float16 or bfloat16 [m, k] with 1 <= m <= 16."""
    fn = _lib.kq_qmv_bf16 if _bf16(x) else _lib.kq_qmv
    _check(fn(_codec(codec), _ptr(w), n, k, _ptr(x), x.shape[0], _ptr(y), _dtype_id(y), _stream(stream)))


def kq_qmm(codec, w, n: int, k: int, x, y, stream=None) -> None:
    fn = _lib.kq_qmm_bf16 if _bf16(x) else _lib.kq_qmm
    _check(fn(_codec(codec), _ptr(w), n, k, _ptr(x), x.shape[0], _ptr(y), _dtype_id(y), _stream(stream)))


def kq_quantized_matmul(codec, w, n: int, k: int, x, y, stream=None) -> None:
    if _bf16(x):  # bfloat16: the GEMV to 16 rows, the GEMM above
        fn = _lib.kq_qmv_bf16 if x.shape[0] <= 16 else _lib.kq_qmm_bf16
        _check(fn(_codec(codec), _ptr(w), n, k, _ptr(x), x.shape[0], _ptr(y), _dtype_id(y), _stream(stream)))
        return
    _check(_lib.kq_quantized_matmul(_codec(codec), _ptr(w), n, k, _ptr(x), x.shape[0], _ptr(y), _dtype_id(y),
                                    _stream(stream)))


def kq_quantized_matmul_residual(codec, w, n: int, k: int, x, residual, y, gate=None, stream=None) -> None:
    """y = residual + gate * (x @ dequant(w)^T).  residual, y [M, n]; gate None, [n] or [G, n] (G rows, one per
    M / G consecutive rows), all three in y's dtype.  residual may be y itself."""
    gate_rows = 0 if gate is None else gate.numel() // max(n, 1)
    _check(_lib.kq_quantized_matmul_residual(_codec(codec), _ptr(w), n, k, _ptr(x), x.shape[0], _ptr(residual),
                                             _ptr(gate), gate_rows, _ptr(y), _dtype_id(y), _stream(stream)))


def kq_quantized_matmul_qmv_bias(codec, w, n: int, k: int, x, bias, y, stream=None) -> None:
    """y = x @ dequant(w)^T + bias for one row of x; bias [n] in y's dtype."""
    _check(_lib.kq_quantized_matmul_qmv_bias(_codec(codec), _ptr(w), n, k, _ptr(x), x.shape[0], _ptr(bias), _ptr(y),
                                             _dtype_id(y), _stream(stream)))


def kq_quantized_matmul_glu(codec, w_gate, w_up, n: int, k: int, x, y, act="silu", stream=None) -> None:
    """y = act(x @ dequant(w_gate)^T) * (x @ dequant(w_up)^T); act 'silu' or 'gelu_tanh' (or a KQ_GLU_* id)."""
    a = _GLU_ACTS[act] if isinstance(act, str) else int(act)
    _check(_lib.kq_quantized_matmul_glu(_codec(codec), _ptr(w_gate), _ptr(w_up), n, k, _ptr(x), x.shape[0], a,
                                        _ptr(y), _dtype_id(y), _stream(stream)))


def kq_expert_tile_map(sorted_ids, n_experts: int, map_, counts, status=None, stream=None) -> None:
    """sorted_ids uint32 (int32 storage) [rows]; map_ [cap, 3]; counts [1]; status [1] or None."""
    _check(_lib.kq_expert_tile_map(_ptr(sorted_ids), sorted_ids.numel(), n_experts, _ptr(map_), _ptr(counts),
                                   map_.shape[0], _ptr(status), _stream(stream)))


def kq_gather_qmm_seg(codec, w, n_experts: int, n: int, k: int, x, map_, counts, y, stream=None) -> None:
    """w uint8 [E, n, row_bytes]; x float16 or bfloat16 [rows, k] expert-sorted; y [rows, n]."""
    fn = _lib.kq_gather_qmm_seg_bf16 if _bf16(x) else _lib.kq_gather_qmm_seg
    _check(fn(_codec(codec), _ptr(w), n_experts, n, k, _ptr(x), x.shape[0], _ptr(map_), _ptr(counts), map_.shape[0],
              _ptr(y), _dtype_id(y), _stream(stream)))


def kq_gather_qmv(codec, w, n_experts: int, n: int, k: int, x, ids, y, stream=None) -> None:
    """w uint8 [E, n, row_bytes]; x float16 [rows, k]; ids int32/uint32 [rows]; y [rows, n]."""
    _check(_lib.kq_gather_qmv(_codec(codec), _ptr(w), n_experts, n, k, _ptr(x), _ptr(ids), x.shape[0], _ptr(y),
                              _dtype_id(y), _stream(stream)))


def kq_moe_glu_gather(codec, gate_w, up_w, n_experts: int, n: int, k: int, x, ids, y, act="silu",
                      limit: float = 0.0, stream=None) -> None:
    """gate_w, up_w uint8 [E, n, row_bytes]; x float16 [T, k]; ids int32/uint32 [T, R]; y [T * R, n] (or
    [T, R, n]).  act: 'silu', 'gelu' (tanh form) or 'silu_limit', or a KQ_GLU_* id."""
    a = _GLU_ACTS[act] if isinstance(act, str) else int(act)
    top_k = ids.shape[1] if ids.dim() > 1 else 1
    _check(_lib.kq_moe_glu_gather(_codec(codec), _ptr(gate_w), _ptr(up_w), n_experts, n, k, _ptr(x), x.shape[0],
                                  _ptr(ids), top_k, a, float(limit), _ptr(y), _dtype_id(y), _stream(stream)))


def kq_gather_mix(y, inv_order, scores, out, stream=None) -> None:
    """y [rows, n] (float16/float32, routing-sorted rows); inv_order int32/uint32 [T * k]; scores float32 [T, k];
    out [T, n] of y's dtype."""
    if out.dtype != y.dtype:
        raise TypeError("out must have y's dtype")
    tokens, top_k = scores.shape
    _check(_lib.kq_gather_mix(_ptr(y), y.shape[0], y.shape[1], _ptr(inv_order), _ptr(scores), tokens, top_k,
                              _ptr(out), _dtype_id(out), _stream(stream)))


def kq_quantize(codec, w, out, stream=None) -> None:
    """w float32 [rows, k] -> out uint8 [rows, row_bytes]."""
    rows, k = (w.shape[0], w.shape[1]) if w.dim() > 1 else (1, w.shape[0])
    _check(_lib.kq_quantize(_codec(codec), _ptr(w), rows, k, _ptr(out), _stream(stream)))


def kq_stream_read(src, out, nbytes: int | None = None, stream=None) -> None:
    """Plain read of src's bytes (a multiple of 16) by out.numel() // 4 workgroups; out int32/uint32 [4 * groups]
    (one word per wave)."""
    nb = src.numel() * src.element_size() if nbytes is None else nbytes
    _check(_lib.kq_stream_read(_ptr(src), nb, _ptr(out), out.numel() // 4, _stream(stream)))


# ---------------------------------------------------------------------------
# key/value cache in 4 bits
# ---------------------------------------------------------------------------

# These calls are often shorter than their Python side: tensors of the current
# device on its current stream go through _kqcall, which makes the same checks
# and returns None for everything it leaves to the code here.
_INTS = (torch.int32, torch.uint32)
_DTYPES = {torch.float32: KQ_F32, torch.float16: KQ_F16, torch.bfloat16: KQ_BF16}


def _index_error(op: str, name: str, t, n: int | None, device: int) -> None:
    """Raise for an index array that is not contiguous 32-bit integers (n of them, where n is given) on the device."""
    if t.dtype not in _INTS:
        raise TypeError(f"{op}: {name} must be int32, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{op}: {name} must be contiguous")
    if n is not None and t.numel() != n:
        raise ValueError(f"{op}: {name} has {t.numel()} entries, expected {n}")
    raise ValueError(f"{op}: {name} is on device {t.get_device()}, not {device}")


def _index(op: str, name: str, t, n: int | None, device: int) -> int:
    """Device pointer of an index array, checked."""
    if (t.dtype not in _INTS or not t.is_contiguous() or (n is not None and t.numel() != n)
            or t.get_device() != device):
        _index_error(op, name, t, n, device)
    return t.data_ptr()


def _on_gpu(op: str, device: int) -> None:
    """Raise for tensors of the host (device -1): a kernel that reads their addresses faults."""
    if device < 0:
        raise ValueError(f"{op}: tensors must be on the GPU")


def _call_on(device: int, stream, fn, *args) -> None:
    """fn(*args, stream) with `device` current: on the given stream, else on that device's current one."""
    _on_gpu(fn.__name__, device)
    if device == torch.cuda.current_device():
        status = fn(*args, _stream(stream))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _stream(stream))
    if status != KQ_OK:
        _check(status)


_PAGE_BYTES: dict = {}  # (codec, page, d) -> (codec id, bytes): pure functions of their arguments


def _page_bytes(codec, page: int, d: int) -> tuple[int, int]:
    key = (codec, page, d)
    got = _PAGE_BYTES.get(key)
    if got is None:
        out, cid = c_i64(), _codec(codec)
        _check(_lib.kq_kv_page_bytes(cid, page, d, ctypes.byref(out)))
        got = _PAGE_BYTES[key] = (cid, out.value)
    return got


def _cache(op: str, codec, k_cache, v_cache, page: int, d: int, heads: int | None, device: int):
    """(codec id, pages, kv heads) of two caches uint8 [pages, kv_heads, page_bytes]."""
    cid, pb = _page_bytes(codec, page, d)
    shape = k_cache.shape
    if (k_cache.dtype is not torch.uint8 or v_cache.dtype is not torch.uint8 or len(shape) != 3
            or v_cache.shape != shape or not k_cache.is_contiguous() or not v_cache.is_contiguous()):
        raise ValueError(f"{op}: k_cache and v_cache must be contiguous uint8 [pages, kv_heads, {pb}]")
    pages, cache_heads, have = shape
    if have != pb:
        raise ValueError(f"{op}: pages hold {have} bytes a head, {pb} expected for page={page}, d={d}")
    if heads is not None and cache_heads != heads:
        raise ValueError(f"{op}: rows of {heads} heads, a cache of {cache_heads}")
    if k_cache.get_device() != device or v_cache.get_device() != device:
        raise ValueError(f"{op}: caches on devices {k_cache.get_device()} and {v_cache.get_device()}, rows on {device}")
    return cid, pages, cache_heads


def _row_stride(op: str, name: str, x, shape) -> int:
    """Elements between rows of x [tokens, heads, d], whose rows are dense."""
    tokens, heads, d = shape
    st = x.stride()
    if x.numel() and (st[2] != 1 or (heads > 1 and st[1] != d)):
        raise ValueError(f"{op}: the rows of {name} must be dense")
    return st[0] if tokens > 1 else heads * d


def kq_kv_page_bytes(codec, page: int, d: int) -> int:
    """Bytes of one (page, kv head) of a 4-bit key or value cache."""
    return _page_bytes(codec, page, d)[1]


def kq_block_tables(ctx_lens, new_lens, free_pages, free_head, page: int, table, slots, cu_new, seq_lens,
                    free_head_out, status=None, stream=None) -> None:
    """Pages and slots of a step's new tokens.  ctx_lens, new_lens, seq_lens int32 [n]; free_pages int32 [n_free] from
    free_head int32 [1]; table int32 [n, width]; slots int32 [tokens]; cu_new int32 [n + 1]; free_head_out, status [1]."""
    if _kqcall is not None and stream is None and ctx_lens.is_cuda:
        dev = torch._C._cuda_getDevice()
        st = _kqcall.block_tables(ctx_lens, new_lens, free_pages, free_head, page, table, slots, cu_new, seq_lens,
                                  free_head_out, status, torch._C._cuda_getCurrentRawStream(dev), dev)
        if st is not None:
            return _check(st)
    op, n, dev = "kq_block_tables", ctx_lens.numel(), ctx_lens.get_device()
    if table.dim() != 2 or table.shape[0] != n:
        raise ValueError(f"{op}: table must be [{n}, width]")
    _call_on(dev, stream, _lib.kq_block_tables, _index(op, "ctx_lens", ctx_lens, n, dev),
             _index(op, "new_lens", new_lens, n, dev), n, page, _index(op, "free_pages", free_pages, None, dev),
             free_pages.numel(), _index(op, "free_head", free_head, 1, dev), _index(op, "table", table, None, dev),
             table.shape[1], _index(op, "slots", slots, None, dev), slots.numel(),
             _index(op, "cu_new", cu_new, n + 1, dev), _index(op, "seq_lens", seq_lens, n, dev),
             _index(op, "free_head_out", free_head_out, 1, dev),
             None if status is None else _index(op, "status", status, 1, dev))


def kq_kv_store(codec, k, v, slots, k_cache, v_cache, page: int, stream=None) -> None:
    """k, v float32/float16/bfloat16 [tokens, kv_heads, d] (dense rows, any row stride) into slots int32 [tokens] of
    k_cache, v_cache uint8 [pages, kv_heads, page_bytes]."""
    if _kqcall is not None and stream is None and k.is_cuda and (codec == "q4_0" or codec == KQ_Q4_0):
        dev = torch._C._cuda_getDevice()
        st = _kqcall.kv_store(k, v, slots, k_cache, v_cache, page, torch._C._cuda_getCurrentRawStream(dev), dev)
        if st is not None:
            return _check(st)
    op, shape, dt, dev = "kq_kv_store", k.shape, _DTYPES.get(k.dtype), k.get_device()
    if len(shape) != 3 or v.shape != shape or v.dtype is not k.dtype or dt is None or v.get_device() != dev:
        raise ValueError(f"{op}: k and v must be [tokens, kv_heads, d] of one float dtype and device")
    tokens, heads, d = shape
    ks, vs = _row_stride(op, "k", k, shape), _row_stride(op, "v", v, shape)
    cid, pages, _ = _cache(op, codec, k_cache, v_cache, page, d, heads, dev)
    _call_on(dev, stream, _lib.kq_kv_store, cid, k.data_ptr(), v.data_ptr(), dt, tokens, heads, d, ks, vs,
             _index(op, "slots", slots, tokens, dev),
             k_cache.data_ptr(), v_cache.data_ptr(), pages, page)


def kq_kv_load(codec, k_cache, v_cache, slots, page: int, k, v, stream=None) -> None:
    """The rows at slots int32 [tokens] of the caches to k, v [tokens, kv_heads, d] (float32, float16 or bfloat16)."""
    if _kqcall is not None and stream is None and k.is_cuda and (codec == "q4_0" or codec == KQ_Q4_0):
        dev = torch._C._cuda_getDevice()
        st = _kqcall.kv_load(k_cache, v_cache, slots, page, k, v, torch._C._cuda_getCurrentRawStream(dev), dev)
        if st is not None:
            return _check(st)
    op, shape, dt, dev = "kq_kv_load", k.shape, _DTYPES.get(k.dtype), k.get_device()
    if (len(shape) != 3 or v.shape != shape or v.dtype is not k.dtype or dt is None or v.get_device() != dev
            or not k.is_contiguous() or not v.is_contiguous()):
        raise ValueError(f"{op}: k and v must be contiguous [tokens, kv_heads, d] of one float dtype and device")
    tokens, heads, d = shape
    cid, pages, _ = _cache(op, codec, k_cache, v_cache, page, d, heads, dev)
    _call_on(dev, stream, _lib.kq_kv_load, cid, k_cache.data_ptr(), v_cache.data_ptr(), pages, page, heads, d,
             _index(op, "slots", slots, tokens, dev), tokens, k.data_ptr(), v.data_ptr(), dt)


def kq_kv_attention_workspace(tokens: int, n_seqs: int, q_heads: int, kv_heads: int, d: int, max_new: int,
                              max_kv: int) -> int:
    """Bytes of workspace that kq_kv_attention needs for these sizes (0: none)."""
    out = c_i64()
    _check(_lib.kq_kv_attention_workspace(tokens, n_seqs, q_heads, kv_heads, d, max_new, max_kv, ctypes.byref(out)))
    return out.value


def kq_kv_attention(codec, q, cu_new, seq_lens, table, k_cache, v_cache, page: int, out, scale: float | None = None,
                    window: int = 0, max_new: int | None = None, max_kv: int | None = None, workspace=None,
                    stream=None) -> None:
    """out[t, h] = softmax(scale * q . K^T) V over the 4-bit rows each token sees (causal, window > 0: the last `window`
    keys).  q float16/bfloat16 [tokens, q_heads, d] (dense rows, any row stride); cu_new int32 [n + 1], seq_lens int32
    [n], table int32 [n, width]; out [tokens, q_heads, d]; scale defaults to d^-0.5.  max_new and max_kv bound a
    request's new tokens and length (default: tokens, width * page).  workspace: uint8 of kq_kv_attention_workspace
    bytes; allocated on the current stream if left out."""
    if _kqcall is not None and stream is None and q.is_cuda and (codec == "q4_0" or codec == KQ_Q4_0) \
            and max_new is not None and max_kv is not None:
        dev = torch._C._cuda_getDevice()
        st = _kqcall.kv_attention(q, cu_new, seq_lens, table, k_cache, v_cache, page, out,
                                  q.size(-1) ** -0.5 if scale is None else scale, window, max_new, max_kv, workspace,
                                  torch._C._cuda_getCurrentRawStream(dev), dev)
        if st is not None:
            return _check(st)
    _attention("kq_kv_attention", _lib.kq_kv_attention, codec, q, cu_new, seq_lens, table, None, k_cache, v_cache, page, out,
               scale, (window,), max_new, max_kv, workspace, stream)


def kq_kv_attention_sinks(codec, q, cu_new, seq_lens, table, k_cache, v_cache, page: int, out, window: int, sinks: int,
                          scale: float | None = None, max_new: int | None = None, max_kv: int | None = None, workspace=None,
                          stream=None) -> None:
    """kq_kv_attention where each token sees the last `window` keys and its request's first `sinks` ones.  Workspace of
    kq_kv_attention_workspace."""
    if _kqcall is not None and stream is None and q.is_cuda and (codec == "q4_0" or codec == KQ_Q4_0) \
            and max_new is not None and max_kv is not None:
        dev = torch._C._cuda_getDevice()
        st = _kqcall.kv_attention_sinks(q, cu_new, seq_lens, table, k_cache, v_cache, page, out,
                                        q.size(-1) ** -0.5 if scale is None else scale, window, sinks, max_new, max_kv,
                                        workspace, torch._C._cuda_getCurrentRawStream(dev), dev)
        if st is not None:
            return _check(st)
    _attention("kq_kv_attention_sinks", _lib.kq_kv_attention_sinks, codec, q, cu_new, seq_lens, table, None, k_cache, v_cache,
               page, out, scale, (window, sinks), max_new, max_kv, workspace, stream)


def kq_kv_attention_prefix_workspace(tokens: int, n_seqs: int, q_heads: int, kv_heads: int, d: int, prefix_len: int,
                                     max_new: int, max_kv: int) -> int:
    """Bytes of workspace that kq_kv_attention_prefix needs for these sizes and smaller ones; prefix_len in keys."""
    out = c_i64()
    _check(_lib.kq_kv_attention_prefix_workspace(tokens, n_seqs, q_heads, kv_heads, d, prefix_len, max_new, max_kv,
                                                 ctypes.byref(out)))
    return out.value


def kq_kv_attention_prefix(codec, q, cu_new, seq_lens, table, prefix, k_cache, v_cache, page: int, out,
                           scale: float | None = None, max_new: int | None = None, max_kv: int | None = None, workspace=None,
                           stream=None) -> None:
    """kq_kv_attention for requests whose first keys are the pages prefix int32 [n_prefix], read once for all of them.
    seq_lens and table count the prefix in; a request whose new tokens do not all stand behind it reads its own row of the
    table alone.  workspace: uint8 of kq_kv_attention_prefix_workspace bytes; allocated if left out."""
    if _kqcall is not None and stream is None and q.is_cuda and (codec == "q4_0" or codec == KQ_Q4_0) \
            and max_new is not None and max_kv is not None:
        dev = torch._C._cuda_getDevice()
        st = _kqcall.kv_attention_prefix(q, cu_new, seq_lens, table, prefix, k_cache, v_cache, page, out,
                                         q.size(-1) ** -0.5 if scale is None else scale, max_new, max_kv, workspace,
                                         torch._C._cuda_getCurrentRawStream(dev), dev)
        if st is not None:
            return _check(st)
    _attention("kq_kv_attention_prefix", _lib.kq_kv_attention_prefix, codec, q, cu_new, seq_lens, table, prefix, k_cache,
               v_cache, page, out, scale, (), max_new, max_kv, workspace, stream)


def _attention(op, fn, codec, q, cu_new, seq_lens, table, prefix, k_cache, v_cache, page, out, scale, windows, max_new,
               max_kv, workspace, stream) -> None:
    """An attention call through ctypes, its tensors checked."""
    n, shape, dev = seq_lens.numel(), q.shape, q.get_device()
    qdt, odt = _DTYPES.get(q.dtype), _DTYPES.get(out.dtype)
    if len(shape) != 3 or qdt is None or odt is None:
        raise ValueError(f"{op}: q must be float16 or bfloat16 [tokens, q_heads, d], out a float tensor of its shape")
    tokens, heads, d = shape
    if out.shape != shape or not out.is_contiguous() or out.get_device() != dev:
        raise ValueError(f"{op}: out must be a contiguous [{tokens}, {heads}, {d}] on q's device")
    tshape = table.shape
    if len(tshape) != 2 or tshape[0] != n:
        raise ValueError(f"{op}: table must be [{n}, width]")
    cid, pages, kv_heads = _cache(op, codec, k_cache, v_cache, page, d, None, dev)
    width = tshape[1]
    if max_new is None:
        max_new = max(tokens, 1)
    if max_kv is None:
        max_kv = max(width * page, 1)
    if workspace is None:
        if prefix is None:
            need = kq_kv_attention_workspace(tokens, n, heads, kv_heads, d, max_new, max_kv)
        else:
            need = kq_kv_attention_prefix_workspace(tokens, n, heads, kv_heads, d, prefix.numel() * page, max_new, max_kv)
        ws = None
        if need:
            _on_gpu(op, dev)
            if stream is not None and _stream(stream) != torch.cuda.current_stream(q.device).cuda_stream:
                raise ValueError(f"{op}: a call on another stream than the current one needs its own workspace")
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
            ws = workspace.data_ptr()
    else:
        if not workspace.is_contiguous() or workspace.get_device() != dev:
            raise ValueError(f"{op}: workspace must be contiguous, on q's device")
        need, ws = workspace.numel() * workspace.element_size(), workspace.data_ptr()
    more = () if prefix is None else (_index(op, "prefix", prefix, None, dev), prefix.numel())
    _call_on(dev, stream, fn, cid, q.data_ptr(), qdt, tokens, heads, kv_heads, d,
             _row_stride(op, "q", q, shape), _index(op, "cu_new", cu_new, n + 1, dev),
             _index(op, "seq_lens", seq_lens, n, dev), n, _index(op, "table", table, None, dev), width,
             *more, k_cache.data_ptr(), v_cache.data_ptr(), pages, page, d ** -0.5 if scale is None else scale, *windows,
             max_new, max_kv, out.data_ptr(), odt, ws, need)


# ---------------------------------------------------------------------------
# pages of the cache shared, given back and moved; rotary positions
# ---------------------------------------------------------------------------

def kq_kv_fork(parents, children, lens, page: int, table, refs, free_pages, free_head, copy_src, copy_dst, free_head_out,
               status=None, stream=None) -> None:
    """Rows children int32 [n] of table int32 [n_seqs, width] start with the first lens int32 [n] tokens of rows parents
    int32 [n].  refs int32 [pages]; copy_src, copy_dst int32 [n] are for kq_kv_copy_pages; free list as in kq_block_tables.
    Columns of a parent that were given back are set to -1 before."""
    if _kqcall is not None and stream is None and parents.is_cuda:
        dev = torch._C._cuda_getDevice()
        st = _kqcall.kv_fork(parents, children, lens, page, table, refs, free_pages, free_head, copy_src, copy_dst,
                             free_head_out, status, torch._C._cuda_getCurrentRawStream(dev), dev)
        if st is not None:
            return _check(st)
    op, n, dev = "kq_kv_fork", parents.numel(), parents.get_device()
    if table.dim() != 2:
        raise ValueError(f"{op}: table must be [n_seqs, width]")
    _call_on(dev, stream, _lib.kq_kv_fork, _index(op, "parents", parents, n, dev), _index(op, "children", children, n, dev),
             _index(op, "lens", lens, n, dev), n, page, _index(op, "table", table, None, dev), table.shape[0], table.shape[1],
             _index(op, "refs", refs, None, dev), refs.numel(), _index(op, "free_pages", free_pages, None, dev),
             free_pages.numel(), _index(op, "free_head", free_head, 1, dev), _index(op, "copy_src", copy_src, n, dev),
             _index(op, "copy_dst", copy_dst, n, dev), _index(op, "free_head_out", free_head_out, 1, dev),
             None if status is None else _index(op, "status", status, 1, dev))


def kq_kv_free(first, last, table, refs, free_pages, free_head, free_head_out, status=None, stream=None) -> None:
    """The entries first[s] <= j < last[s] (int32 [n_seqs]) of table int32 [n_seqs, width] are given back: refs int32
    [pages] counts them off, pages without a holder go back to the free list."""
    if _kqcall is not None and stream is None and first.is_cuda:
        dev = torch._C._cuda_getDevice()
        st = _kqcall.kv_free(first, last, table, refs, free_pages, free_head, free_head_out, status,
                             torch._C._cuda_getCurrentRawStream(dev), dev)
        if st is not None:
            return _check(st)
    op, n, dev = "kq_kv_free", first.numel(), first.get_device()
    if table.dim() != 2 or table.shape[0] != n:
        raise ValueError(f"{op}: table must be [{n}, width]")
    _call_on(dev, stream, _lib.kq_kv_free, _index(op, "first", first, n, dev), _index(op, "last", last, n, dev), n,
             _index(op, "table", table, None, dev), table.shape[1], _index(op, "refs", refs, None, dev), refs.numel(),
             _index(op, "free_pages", free_pages, None, dev), free_pages.numel(), _index(op, "free_head", free_head, 1, dev),
             _index(op, "free_head_out", free_head_out, 1, dev),
             None if status is None else _index(op, "status", status, 1, dev))


def kq_kv_compact(free_pages, free_head, table, refs, table_out, refs_out, free_out, remap, copy_src, copy_dst, free_head_out,
                  status=None, stream=None) -> None:
    """The held pages move to the front of the cache: copy_src, copy_dst int32 [n_copy] are for kq_kv_copy_pages, remap
    int32 [pages] has the new ids; table, refs and free list by them in the outputs, which may be the inputs."""
    if _kqcall is not None and stream is None and free_pages.is_cuda:
        dev = torch._C._cuda_getDevice()
        st = _kqcall.kv_compact(free_pages, free_head, table, refs, table_out, refs_out, free_out, remap, copy_src, copy_dst,
                                free_head_out, status, torch._C._cuda_getCurrentRawStream(dev), dev)
        if st is not None:
            return _check(st)
    op, dev, n_free, entries, pages, n = ("kq_kv_compact", free_pages.get_device(), free_pages.numel(), table.numel(),
                                          refs.numel(), copy_src.numel())
    _call_on(dev, stream, _lib.kq_kv_compact, _index(op, "free_pages", free_pages, None, dev), n_free,
             _index(op, "free_head", free_head, 1, dev), _index(op, "table", table, None, dev), entries,
             _index(op, "refs", refs, None, dev), pages, _index(op, "table_out", table_out, entries, dev),
             _index(op, "refs_out", refs_out, pages, dev), _index(op, "free_out", free_out, n_free, dev),
             _index(op, "remap", remap, pages, dev), _index(op, "copy_src", copy_src, None, dev),
             _index(op, "copy_dst", copy_dst, n, dev), n, _index(op, "free_head_out", free_head_out, 1, dev),
             None if status is None else _index(op, "status", status, 1, dev))


def kq_kv_copy_pages(src, dst, k_cache, v_cache, stream=None) -> None:
    """Page src[i] to page dst[i] (int32 [n]) of k_cache and v_cache uint8 [pages, kv_heads, page_bytes]; pairs with an id
    that is no page are skipped."""
    if _kqcall is not None and stream is None and src.is_cuda:
        dev = torch._C._cuda_getDevice()
        st = _kqcall.kv_copy_pages(src, dst, k_cache, v_cache, torch._C._cuda_getCurrentRawStream(dev), dev)
        if st is not None:
            return _check(st)
    op, n, dev = "kq_kv_copy_pages", src.numel(), src.get_device()
    if (k_cache.dtype is not torch.uint8 or v_cache.dtype is not torch.uint8 or k_cache.dim() != 3
            or v_cache.shape != k_cache.shape or not k_cache.is_contiguous() or not v_cache.is_contiguous()):
        raise ValueError(f"{op}: k_cache and v_cache must be contiguous uint8 [pages, kv_heads, page_bytes]")
    if k_cache.get_device() != dev or v_cache.get_device() != dev:
        raise ValueError(f"{op}: caches on devices {k_cache.get_device()} and {v_cache.get_device()}, lists on {dev}")
    _call_on(dev, stream, _lib.kq_kv_copy_pages, _index(op, "src", src, n, dev), _index(op, "dst", dst, n, dev), n,
             k_cache.data_ptr(), v_cache.data_ptr(), k_cache.shape[0], k_cache.shape[1] * k_cache.shape[2])


def _rope_rows(op: str, name: str, x, out, dev: int):
    """(pointer, heads, row stride, pointer, row stride) of rows and where they go; out None: in place."""
    if out is None:
        out = x
    if x.dim() != 3 or x.dtype not in _DTYPES or out.shape != x.shape or out.dtype is not x.dtype:
        raise ValueError(f"{op}: {name} and {name}_out must be [tokens, heads, d] of one float dtype")
    if x.get_device() != dev or out.get_device() != dev:
        raise ValueError(f"{op}: {name} and {name}_out must be on the device of cu_new")
    return (x.data_ptr(), x.shape[1], _row_stride(op, name, x, x.shape), out.data_ptr(),
            _row_stride(op, name + "_out", out, x.shape))


def kq_rope(q, k, cu_new, seq_lens, inv_freq, q_out=None, k_out=None, layout="half", mscale: float = 1.0,
            stream=None) -> None:
    """q [tokens, q_heads, d] and k [tokens, kv_heads, d] (float32, float16 or bfloat16, dense rows, any row stride; one of
    them may be None) turned to their positions, in place or to q_out and k_out.  cu_new int32 [n + 1], seq_lens int32 [n];
    inv_freq float32 [rot / 2]: the first rot values of a head turn; layout 'half' or 'pairs' (or a KQ_ROPE_* id)."""
    lay = _ROPE_LAYOUTS[layout] if isinstance(layout, str) else int(layout)
    if _kqcall is not None and stream is None and cu_new.is_cuda:
        dev = torch._C._cuda_getDevice()
        st = _kqcall.rope(q, k, cu_new, seq_lens, inv_freq, q_out, k_out, lay, mscale,
                          torch._C._cuda_getCurrentRawStream(dev), dev)
        if st is not None:
            return _check(st)
    op, n, dev = "kq_rope", seq_lens.numel(), cu_new.get_device()
    if (q is None and k is None) or (q is None and q_out is not None) or (k is None and k_out is not None):
        raise ValueError(f"{op}: q or k is wanted, and no output without its input")
    one = k if q is None else q
    none = (None, 0, 0, None, 0)
    qa = none if q is None else _rope_rows(op, "q", q, q_out, dev)
    ka = none if k is None else _rope_rows(op, "k", k, k_out, dev)
    if q is not None and k is not None and (q.shape[0] != k.shape[0] or q.shape[2] != k.shape[2] or q.dtype is not k.dtype):
        raise ValueError(f"{op}: q and k must have the same tokens, head size and dtype")
    if inv_freq.dtype is not torch.float32 or not inv_freq.is_contiguous() or inv_freq.get_device() != dev:
        raise ValueError(f"{op}: inv_freq must be contiguous float32 on the device of cu_new")
    _call_on(dev, stream, _lib.kq_rope, *qa[:3], *ka[:3], _DTYPES[one.dtype], one.shape[0], one.shape[2], 2 * inv_freq.numel(),
             lay, _index(op, "cu_new", cu_new, n + 1, dev), _index(op, "seq_lens", seq_lens, n, dev), n, inv_freq.data_ptr(),
             mscale, *qa[3:], *ka[3:])


def kq_rope_freqs(rot: int, base: float = 10000.0, scaling="none", factor: float = 1.0, original: int = 0,
                  fast: float = 32.0, slow: float = 1.0, factors=None, device="cuda"):
    """(inv_freq float32 [rot / 2] on `device`, mscale) for kq_rope.  scaling 'none', 'linear', 'ntk' or 'yarn' by `factor`
    over `original` positions; factors: a float tensor [rot / 2] of divisors (a GGUF file's rope_freqs)."""
    sc = _ROPE_SCALINGS[scaling] if isinstance(scaling, str) else int(scaling)
    div = None
    if factors is not None:
        div = factors.detach().to(device="cpu", dtype=torch.float32).contiguous()
        if div.numel() != rot // 2:
            raise ValueError(f"kq_rope_freqs: factors has {div.numel()} entries, expected {rot // 2}")
    out, m = (ctypes.c_float * max(1, rot // 2))(), ctypes.c_float()
    _check(_lib.kq_rope_freqs(rot, base, sc, factor, original, fast, slow, _ptr(div), out, ctypes.byref(m)))
    return torch.tensor(list(out), dtype=torch.float32, device=device), m.value


# ---------------------------------------------------------------------------
# allocating conveniences (torch allocates; the library computes)
# ---------------------------------------------------------------------------

def dequantize(codec, w, k: int, dtype=None):
    import torch

    out = torch.empty((w.shape[0], k), dtype=dtype or torch.float16, device=w.device)
    kq_dequantize(codec, w, k, out)
    return out


def quantized_matmul(codec, w, n: int, k: int, x, out_dtype=None):
    import torch

    y = torch.empty((x.shape[0], n), dtype=out_dtype or x.dtype, device=x.device)
    kq_quantized_matmul(codec, w, n, k, x, y)
    return y


def quantize(codec, w):
    import torch

    out = torch.empty((w.shape[0], kq_row_bytes(codec, w.shape[1])), dtype=torch.uint8, device=w.device)
    kq_quantize(codec, w, out)
    return out


def expert_tile_map(sorted_ids, n_experts: int):
    import torch

    cap = kq_expert_tile_map_capacity(sorted_ids.numel(), n_experts)
    map_ = torch.empty((max(cap, 1), 3), dtype=torch.int32, device=sorted_ids.device)
    counts = torch.empty((1,), dtype=torch.int32, device=sorted_ids.device)
    kq_expert_tile_map(sorted_ids, n_experts, map_[:cap] if cap else map_, counts)
    return map_, counts


def kv_cache(codec, pages: int, kv_heads: int, page: int, d: int, device="cuda"):
    """A zeroed key and value cache, uint8 [pages, kv_heads, page_bytes] each."""
    shape = (pages, kv_heads, kq_kv_page_bytes(codec, page, d))
    return tuple(torch.zeros(shape, dtype=torch.uint8, device=device) for _ in range(2))


def block_tables(ctx_lens, new_lens, free_pages, free_head, page: int, table, tokens: int):
    """(slots [tokens], cu_new [n + 1], seq_lens [n], free_head_out [1], status [1]) of a step; table is updated."""
    n, dev = ctx_lens.numel(), ctx_lens.device
    slots, cu, lens, head, status = (torch.empty((m,), dtype=torch.int32, device=dev) for m in (tokens, n + 1, n, 1, 1))
    kq_block_tables(ctx_lens, new_lens, free_pages, free_head, page, table, slots, cu, lens, head, status)
    return slots, cu, lens, head, status


def kv_attention(codec, q, cu_new, seq_lens, table, k_cache, v_cache, page: int, scale=None, window: int = 0,
                 max_new=None, max_kv=None, out_dtype=None):
    out = torch.zeros(q.shape, dtype=out_dtype or q.dtype, device=q.device)
    kq_kv_attention(codec, q, cu_new, seq_lens, table, k_cache, v_cache, page, out, scale, window, max_new, max_kv)
    return out


def kv_attention_sinks(codec, q, cu_new, seq_lens, table, k_cache, v_cache, page: int, window: int, sinks: int, scale=None,
                       max_new=None, max_kv=None, out_dtype=None):
    out = torch.zeros(q.shape, dtype=out_dtype or q.dtype, device=q.device)
    kq_kv_attention_sinks(codec, q, cu_new, seq_lens, table, k_cache, v_cache, page, out, window, sinks, scale, max_new, max_kv)
    return out


def kv_attention_prefix(codec, q, cu_new, seq_lens, table, prefix, k_cache, v_cache, page: int, scale=None, max_new=None,
                        max_kv=None, out_dtype=None):
    out = torch.zeros(q.shape, dtype=out_dtype or q.dtype, device=q.device)
    kq_kv_attention_prefix(codec, q, cu_new, seq_lens, table, prefix, k_cache, v_cache, page, out, scale, max_new, max_kv)
    return out


def kv_fork(parents, children, lens, page: int, table, refs, free_pages, free_head):
    """(copy_src [n], copy_dst [n], free_head_out [1], status [1]) of forks; table and refs are updated."""
    n, dev = parents.numel(), parents.device
    src, dst, head, status = (torch.empty((m,), dtype=torch.int32, device=dev) for m in (n, n, 1, 1))
    kq_kv_fork(parents, children, lens, page, table, refs, free_pages, free_head, src, dst, head, status)
    return src, dst, head, status


def kv_free(first, last, table, refs, free_pages, free_head):
    """(free_head_out [1], status [1]); refs and free_pages are updated."""
    head, status = (torch.empty((1,), dtype=torch.int32, device=first.device) for _ in range(2))
    kq_kv_free(first, last, table, refs, free_pages, free_head, head, status)
    return head, status


def kv_compact(free_pages, free_head, table, refs):
    """(remap [pages], copy_src, copy_dst, status [1]); table, refs, free_pages and free_head are updated."""
    pages, dev = refs.numel(), refs.device
    most = min(free_pages.numel(), pages // 2)
    remap, src, dst, status = (torch.empty((m,), dtype=torch.int32, device=dev) for m in (pages, most, most, 1))
    kq_kv_compact(free_pages, free_head, table, refs, table, refs, free_pages, remap, src, dst, free_head, status)
    return remap, src, dst, status
