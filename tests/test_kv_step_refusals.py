"""Refusals of kq_rope, the page operators and the attention with sinks or a shared prefix: every one returns before a
launch (no GPU needed)."""

import ctypes

import numpy as np
import pytest
import torch

kq = pytest.importorskip("gguf_quant_matmul_amd.kq", reason="libkq.so not built")
L = kq._lib
A = 0x100000  # a 16-byte aligned address that is never read
NAMES = ["q", "k", "v", "cu", "lens", "freq", "qo", "ko", "parents", "children", "table", "refs", "free", "head", "src", "dst",
         "head_out", "status", "first", "last", "table_out", "refs_out", "free_out", "remap", "kc", "vc", "prefix", "out", "ws"]
ADDR = {name: A * (i + 1) for i, name in enumerate(NAMES)}


def rope(**kw):
    a = dict(ADDR, hq=4, qs=256, hkv=2, ks=128, dt=1, tokens=3, d=64, rot=64, layout=0, n=2, m=1.0, qos=256, kos=128)
    a.update(kw)
    return L.kq_rope(a["q"], a["hq"], a["qs"], a["k"], a["hkv"], a["ks"], a["dt"], a["tokens"], a["d"], a["rot"], a["layout"],
                     a["cu"], a["lens"], a["n"], a["freq"], a["m"], a["qo"], a["qos"], a["ko"], a["kos"], None)


def freqs(**kw):
    a = dict(rot=64, base=1e4, scaling=0, factor=1.0, original=0, fast=32.0, slow=1.0, factors=None,
             out=(ctypes.c_float * 64)(), m=ctypes.byref(ctypes.c_float()))
    a.update(kw)
    return L.kq_rope_freqs(a["rot"], a["base"], a["scaling"], a["factor"], a["original"], a["fast"], a["slow"], a["factors"],
                           a["out"], a["m"])


def fork(**kw):
    a = dict(ADDR, n=3, page=16, rows=8, width=4, pages=20, n_free=8)
    a.update(kw)
    return L.kq_kv_fork(a["parents"], a["children"], a["lens"], a["n"], a["page"], a["table"], a["rows"], a["width"], a["refs"],
                        a["pages"], a["free"], a["n_free"], a["head"], a["src"], a["dst"], a["head_out"], a["status"], None)


def free(**kw):
    a = dict(ADDR, rows=8, width=4, pages=20, n_free=8)
    a.update(kw)
    return L.kq_kv_free(a["first"], a["last"], a["rows"], a["table"], a["width"], a["refs"], a["pages"], a["free"], a["n_free"],
                        a["head"], a["head_out"], a["status"], None)


def compact(**kw):
    a = dict(ADDR, n_free=8, entries=32, pages=20, n_copy=8)
    a.update(kw)
    return L.kq_kv_compact(a["free"], a["n_free"], a["head"], a["table"], a["entries"], a["refs"], a["pages"], a["table_out"],
                           a["refs_out"], a["free_out"], a["remap"], a["src"], a["dst"], a["n_copy"], a["head_out"],
                           a["status"], None)


def copy(**kw):
    a = dict(ADDR, n=3, pages=20, bytes=576)
    a.update(kw)
    return L.kq_kv_copy_pages(a["src"], a["dst"], a["n"], a["kc"], a["vc"], a["pages"], a["bytes"], None)


ATTN = dict(ADDR, codec=2, qdt=1, tokens=3, hq=8, hkv=2, d=64, stride=512, n=2, width=4, pages=4, page=16, scale=0.1, window=8,
            sinks=4, n_prefix=2, max_new=2, max_kv=64, odt=1, ws_bytes=1 << 30)


def sinks(**kw):
    a = dict(ATTN, **kw)
    return L.kq_kv_attention_sinks(a["codec"], a["q"], a["qdt"], a["tokens"], a["hq"], a["hkv"], a["d"], a["stride"], a["cu"],
                                   a["lens"], a["n"], a["table"], a["width"], a["kc"], a["vc"], a["pages"], a["page"],
                                   a["scale"], a["window"], a["sinks"], a["max_new"], a["max_kv"], a["out"], a["odt"], a["ws"],
                                   a["ws_bytes"], None)


def prefix(**kw):
    a = dict(ATTN, **kw)
    return L.kq_kv_attention_prefix(a["codec"], a["q"], a["qdt"], a["tokens"], a["hq"], a["hkv"], a["d"], a["stride"], a["cu"],
                                    a["lens"], a["n"], a["table"], a["width"], a["prefix"], a["n_prefix"], a["kc"], a["vc"],
                                    a["pages"], a["page"], a["scale"], a["max_new"], a["max_kv"], a["out"], a["odt"], a["ws"],
                                    a["ws_bytes"], None)


ARG, CODEC, SHAPE, ALIGN, CAP = kq.KQ_ERR_ARG, kq.KQ_ERR_CODEC, kq.KQ_ERR_SHAPE, kq.KQ_ERR_ALIGN, kq.KQ_ERR_CAPACITY
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("call, kw, status, msg", [
    (rope, dict(dt=3), ARG, "dtype"),
    (rope, dict(d=48, rot=48), SHAPE, "d=48"),
    (rope, dict(d=288, rot=64), SHAPE, "d=288"),
    (rope, dict(rot=72), SHAPE, "rot=72"),
    (rope, dict(rot=12), SHAPE, "rot=12"),
    (rope, dict(rot=0), SHAPE, "rot=0"),
    (rope, dict(layout=2), ARG, "layout=2"),
    (rope, dict(hq=-1), ARG, "q_heads"),
    (rope, dict(hkv=5000), ARG, "kv_heads"),
    (rope, dict(n=65537), ARG, "n_seqs"),
    (rope, dict(tokens=-1), ARG, "tokens"),
    (rope, dict(tokens=1 << 27), ARG, "tokens"),
    (rope, dict(m=NAN), ARG, "mscale"),
    (rope, dict(m=INF), ARG, "mscale"),
    (rope, dict(qs=255), SHAPE, "q's row stride"),
    (rope, dict(kos=120), SHAPE, "k_out's row stride"),
    (rope, dict(ks=132), ALIGN, "k's row stride"),
    (rope, dict(q=None), ARG, "null"),
    (rope, dict(ko=None), ARG, "null"),
    (rope, dict(freq=None), ARG, "null"),
    (rope, dict(cu=None), ARG, "null"),
    (rope, dict(q=ADDR["q"] + 8), ALIGN, "16-byte"),
    (rope, dict(ko=ADDR["ko"] + 4), ALIGN, "16-byte"),
    (rope, dict(lens=ADDR["lens"] + 2), ALIGN, "4-byte"),
    (rope, dict(qo=ADDR["q"] + 16), ARG, "q_out overlaps q"),
    (rope, dict(qo=ADDR["q"], qos=264), ARG, "q_out overlaps q"),
    (rope, dict(qo=ADDR["k"]), ARG, "q_out overlaps k"),
    (rope, dict(ko=ADDR["qo"]), ARG, "q_out and k_out overlap"),
    (rope, dict(qs=512, k=ADDR["q"] + 256, ks=512, qo=ADDR["q"], qos=512, ko=ADDR["q"] + 256, kos=512), ARG, "q_out overlaps k"),
    (rope, dict(qo=ADDR["cu"]), ARG, "q_out overlaps cu_new"),
    (rope, dict(ko=ADDR["freq"] - 16), ARG, "k_out overlaps inv_freq"),
    (freqs, dict(rot=7), SHAPE, "rot=7"),
    (freqs, dict(rot=0), SHAPE, "rot=0"),
    (freqs, dict(base=1.0), ARG, "base"),
    (freqs, dict(base=NAN), ARG, "base"),
    (freqs, dict(scaling=4), ARG, "scaling=4"),
    (freqs, dict(scaling=1, factor=0.5), ARG, "factor"),
    (freqs, dict(scaling=2, factor=NAN), ARG, "factor"),
    (freqs, dict(scaling=2, factor=2.0, rot=2), SHAPE, "rot=2"),
    (freqs, dict(scaling=3, factor=2.0), ARG, "original"),
    (freqs, dict(scaling=3, factor=2.0, original=100, fast=1.0, slow=1.0), ARG, "fast"),
    (freqs, dict(factors=(ctypes.c_float * 32)()), ARG, "factors[0]"),
    (freqs, dict(out=None), ARG, "null"),
    (fork, dict(page=24), SHAPE, "page=24"),
    (fork, dict(n=-1), ARG, "n=-1"),
    (fork, dict(n=65537), ARG, "n=65537"),
    (fork, dict(rows=65537), ARG, "n_seqs"),
    (fork, dict(width=-1), ARG, "width"),
    (fork, dict(width=1 << 30, rows=1 << 11), ARG, "width"),
    (fork, dict(pages=0), ARG, "pages"),
    (fork, dict(n_free=-1), ARG, "n_free"),
    (fork, dict(head=None), ARG, "null"),
    (fork, dict(refs=None), ARG, "null"),
    (fork, dict(table=None), ARG, "null"),
    (fork, dict(free=None), ARG, "null"),
    (fork, dict(src=ADDR["src"] + 2), ALIGN, "copy_src"),
    (fork, dict(lens=ADDR["lens"] + 1), ALIGN, "lens"),
    (fork, dict(head_out=ADDR["head"]), ARG, "free_head_out overlaps free_head"),
    (fork, dict(dst=ADDR["src"] + 8), ARG, "overlaps copy_src"),
    (fork, dict(refs=ADDR["table"] + 4 * 31), ARG, "refs overlaps table"),
    (fork, dict(table=ADDR["lens"]), ARG, "table overlaps lens"),
    (free, dict(rows=-1), ARG, "n_seqs"),
    (free, dict(pages=1 << 31), ARG, "pages"),
    (free, dict(refs=None), ARG, "null"),
    (free, dict(last=None), ARG, "null"),
    (free, dict(free=None), ARG, "null"),
    (free, dict(table=ADDR["table"] + 2), ALIGN, "table"),
    (free, dict(head_out=ADDR["head"]), ARG, "overlaps free_head"),
    (free, dict(free=ADDR["refs"] + 4 * 19), ARG, "free_pages overlaps refs"),
    (free, dict(status=ADDR["head_out"]), ARG, "status overlaps free_head_out"),
    (compact, dict(pages=(1 << 20) + 1, n_copy=1 << 20), ARG, "pages"),
    (compact, dict(pages=0), ARG, "pages"),
    (compact, dict(n_copy=7), CAP, "n_copy=7"),
    (compact, dict(n_free=30, n_copy=9), CAP, "n_copy=9"),
    (compact, dict(remap=None), ARG, "null"),
    (compact, dict(free_out=None), ARG, "null"),
    (compact, dict(dst=None), ARG, "null"),
    (compact, dict(remap=ADDR["remap"] + 1), ALIGN, "remap"),
    (compact, dict(remap=ADDR["refs"]), ARG, "remap overlaps refs"),
    (compact, dict(table_out=ADDR["table"] + 4), ARG, "table_out overlaps table"),
    (compact, dict(table_out=ADDR["refs"]), ARG, "table_out overlaps refs"),
    (compact, dict(refs_out=ADDR["refs"] + 4), ARG, "refs_out overlaps refs"),
    (compact, dict(free_out=ADDR["free"] + 4), ARG, "free_out overlaps free_pages"),
    (compact, dict(head_out=ADDR["refs"]), ARG, "free_head_out overlaps refs"),
    (copy, dict(n=-1), ARG, "n=-1"),
    (copy, dict(pages=0), ARG, "pages"),
    (copy, dict(bytes=24), SHAPE, "bytes=24"),
    (copy, dict(bytes=0), SHAPE, "bytes=0"),
    (copy, dict(kc=None), ARG, "null cache"),
    (copy, dict(vc=ADDR["vc"] + 8), ALIGN, "caches"),
    (copy, dict(vc=ADDR["kc"] + 576), ARG, "overlap"),
    (copy, dict(src=None), ARG, "null"),
    (copy, dict(dst=ADDR["dst"] + 2), ALIGN, "src and dst"),
    (copy, dict(src=ADDR["kc"] + 64), ARG, "overlaps a cache"),
    (sinks, dict(sinks=-1), ARG, "sinks=-1"),
    (sinks, dict(window=-1), ARG, "window"),
    (sinks, dict(codec=3), CODEC, "q4_0"),
    (sinks, dict(out=ADDR["kc"]), ARG, "out overlaps k_cache"),
    (sinks, dict(max_kv=1 << 20, window=1 << 19, ws_bytes=0), CAP, "workspace"),
    (prefix, dict(prefix=None), ARG, "null prefix"),
    (prefix, dict(n_prefix=0), ARG, "n_prefix"),
    (prefix, dict(n_prefix=-1), ARG, "n_prefix"),
    (prefix, dict(n_prefix=1 << 26), ARG, "prefix of"),
    (prefix, dict(n_prefix=1 << 62), ARG, "n_prefix"),
    (prefix, dict(prefix=ADDR["prefix"] + 2), ALIGN, "4-byte"),
    (prefix, dict(out=ADDR["prefix"] - 64), ARG, "out overlaps prefix"),
    (prefix, dict(ws_bytes=64), CAP, "workspace of 64"),
    (prefix, dict(ws=None), CAP, "workspace of 0"),
    (prefix, dict(ws=ADDR["ws"] + 8), ALIGN, "workspace="),
    (prefix, dict(ws=ADDR["out"]), ARG, "workspace overlaps out"),
    (prefix, dict(prefix=ADDR["ws"] + 128), ARG, "workspace overlaps prefix"),
    (prefix, dict(hq=7), SHAPE, "q_heads=7"),
])
def test_refused_before_launch(call, kw, status, msg):
    ret = call(**kw)
    err = kq.kq_last_error()
    assert ret == status, (ret, err)
    assert msg in err and err.startswith("[kq_"), err


def test_empty_calls_do_nothing():
    assert rope(tokens=0, q=None, k=None) == 0
    assert rope(n=0, cu=None, lens=None) == 0
    assert rope(hq=0, hkv=0, q=None, k=None, qo=None, ko=None) == 0
    assert copy(n=0, src=None, dst=None) == 0
    assert sinks(tokens=0, q=None, out=None) == 0
    assert prefix(n=0, cu=None, lens=None, table=None) == 0


def test_prefix_workspace():
    need = kq.kq_kv_attention_prefix_workspace
    assert need(0, 0, 8, 8, 64, 16, 1, 17) == 0
    # sums and a pair of statistics for every row and split, at least one
    assert need(5, 5, 32, 8, 128, 64, 1, 65) >= 5 * 32 * 130 * 4
    for args in ((1, 1, 8, 8, 64, 0, 1, 17), (1, 1, 8, 8, 64, 1 << 30, 1, 17), (1, 1, 6, 4, 64, 16, 1, 1)):
        with pytest.raises(kq.KQError):
            need(*args)


def test_binding_checks_shapes():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    q, k, f = torch.zeros(3, 4, 64), torch.zeros(3, 2, 64), torch.zeros(32)
    with pytest.raises(ValueError, match="q or k is wanted"):
        kq.kq_rope(None, None, i32(3), i32(2), f)
    with pytest.raises(ValueError, match="no output without"):
        kq.kq_rope(q, None, i32(3), i32(2), f, None, k)
    with pytest.raises(ValueError, match="one float dtype"):
        kq.kq_rope(q, k, i32(3), i32(2), f, q.half())
    with pytest.raises(ValueError, match="same tokens"):
        kq.kq_rope(q, k[:2], i32(3), i32(2), f)
    with pytest.raises(ValueError, match="inv_freq"):
        kq.kq_rope(q, k, i32(3), i32(2), f.double())
    with pytest.raises(ValueError, match="dense"):
        kq.kq_rope(q.transpose(0, 1), None, i32(3), i32(2), f)
    with pytest.raises(KeyError):
        kq.kq_rope(q, k, i32(3), i32(2), f, layout="whole")
    with pytest.raises(ValueError, match="factors has 3"):
        kq.kq_rope_freqs(64, factors=torch.ones(3), device="cpu")
    with pytest.raises(ValueError, match="children has 2"):
        kq.kq_kv_fork(i32(3), i32(2), i32(3), 16, i32(4, 2), i32(9), i32(4), i32(1), i32(3), i32(3), i32(1))
    with pytest.raises(ValueError, match=r"table must be \[3, width\]"):
        kq.kq_kv_free(i32(3), i32(3), i32(4, 2), i32(9), i32(4), i32(1), i32(1))
    with pytest.raises(ValueError, match="refs_out has 8"):
        kq.kq_kv_compact(i32(4), i32(1), i32(4, 2), i32(9), i32(4, 2), i32(8), i32(4), i32(9), i32(4), i32(4), i32(1))
    with pytest.raises(ValueError, match="caches must be|must be contiguous"):
        kq.kq_kv_copy_pages(i32(3), i32(3), torch.zeros(4, 2, 288), torch.zeros(4, 2, 288))


def _calls(dev):
    """A valid call of every operator on tensors of a device."""
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)
    kc, vc = (torch.zeros((4, 2, kq.kq_kv_page_bytes("q4_0", 16, 64)), dtype=torch.uint8, device=dev) for _ in range(2))
    q, k = (torch.zeros((3, h, 64), dtype=torch.float16, device=dev) for h in (4, 2))
    f = torch.zeros(32, device=dev)
    att = q, i32(3), i32(2), i32(2, 3)
    return {"rope": lambda **kw: kq.kq_rope(q, k, i32(3), i32(2), f, **kw),
            "fork": lambda **kw: kq.kq_kv_fork(i32(2), i32(2), i32(2), 16, i32(4, 2), i32(9), i32(4), i32(1), i32(2), i32(2),
                                               i32(1), **kw),
            "free": lambda **kw: kq.kq_kv_free(i32(4), i32(4), i32(4, 2), i32(9), i32(4), i32(1), i32(1), **kw),
            "compact": lambda **kw: kq.kq_kv_compact(i32(4), i32(1), i32(4, 2), i32(9), i32(4, 2), i32(9), i32(4), i32(9),
                                                     i32(4), i32(4), i32(1), **kw),
            "copy": lambda **kw: kq.kq_kv_copy_pages(i32(2), i32(2), kc, vc, **kw),
            "sinks": lambda **kw: kq.kq_kv_attention_sinks("q4_0", *att, kc, vc, 16, torch.zeros_like(q), 8, 2, max_new=2,
                                                           max_kv=48, **kw),
            "prefix": lambda **kw: kq.kq_kv_attention_prefix("q4_0", *att, i32(1), kc, vc, 16, torch.zeros_like(q), max_new=2,
                                                             max_kv=48, **kw)}


@pytest.mark.parametrize("kw", [{}, {"stream": 0}])
@pytest.mark.parametrize("name", ["rope", "fork", "free", "compact", "copy", "sinks", "prefix"])
def test_host_tensors_are_refused(name, kw):
    with pytest.raises(ValueError, match="on the GPU"):
        _calls("cpu")[name](**kw)


# ---------------------------------------------------------------------------
# frequencies (computed on the host)
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("rot, base", [(64, 1e4), (128, 5e5), (8, 1e6)])
def test_rope_freqs(rot, base):
    i = np.arange(0, rot, 2, dtype=np.float64)
    plain = base ** (-i / rot)
    get = lambda **kw: (lambda f, m: (f.numpy(), m))(*kq.kq_rope_freqs(rot, base, device="cpu", **kw))
    near = lambda got, want: np.abs(got - want).max() <= 0 or (np.abs(got - want) <= 2.0 ** -24 * 1.001 * np.abs(want)).all()
    f, m = get()
    assert near(f, plain) and m == 1
    assert near(get(scaling="linear", factor=4.0)[0], plain / 4)
    f, m = get(scaling="ntk", factor=8.0)
    assert near(f, (base * 8 ** (rot / (rot - 2))) ** (-i / rot)) and m == 1
    # the lowest frequency is an eighth of what it was, the highest the same
    assert np.isclose(f[-1], plain[-1] / 8, rtol=1e-6) and f[0] == 1
    div = np.linspace(1, 32, rot // 2).astype(np.float32)
    assert near(get(factors=torch.from_numpy(div))[0], plain / div)
    f, m = get(scaling="yarn", factor=16.0, original=4096)
    assert m == np.float32(0.1 * np.log(16) + 1)
    turns = 4096 * plain / (2 * np.pi)
    # kept above 32 turns, divided below one, between the two in between (the ramp starts and ends at whole pairs)
    lo = max(0, np.floor(rot * np.log(4096 / (32 * 2 * np.pi)) / (2 * np.log(base))))
    hi = min(rot - 1, np.ceil(rot * np.log(4096 / (2 * np.pi)) / (2 * np.log(base))))
    ramp = np.clip((np.arange(rot // 2) - lo) / max(hi - lo, 0.001), 0, 1)
    assert near(f, plain / 16 * ramp + plain * (1 - ramp))
    assert (f[turns > 2 * 32 * base ** (2 / rot)] == plain.astype(np.float32)[turns > 2 * 32 * base ** (2 / rot)]).all()
    assert near(f[ramp == 1], plain[ramp == 1] / 16)
