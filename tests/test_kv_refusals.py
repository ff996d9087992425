"""Refusals of the 4-bit cache entry points: every one returns before a launch (no GPU needed)."""

import pytest
import torch

kq = pytest.importorskip("gguf_quant_matmul_amd.kq", reason="libkq.so not built")
L = kq._lib
A = 0x100000  # a 16-byte aligned address that is never read
ADDR = {name: A * (i + 1) for i, name in enumerate(
    ["ctx", "new", "free", "head", "table", "slots", "cu", "lens", "head_out", "status", "k", "v", "kc", "vc", "q",
     "out", "ws"])}


def tables(**kw):
    a = dict(ADDR, n=4, page=16, n_free=8, width=4, tokens=10)
    a.update(kw)
    return L.kq_block_tables(a["ctx"], a["new"], a["n"], a["page"], a["free"], a["n_free"], a["head"], a["table"],
                             a["width"], a["slots"], a["tokens"], a["cu"], a["lens"], a["head_out"], a["status"], None)


def store(**kw):
    a = dict(ADDR, codec=2, dt=1, tokens=3, heads=2, d=64, ks=128, vs=128, pages=4, page=16)
    a.update(kw)
    return L.kq_kv_store(a["codec"], a["k"], a["v"], a["dt"], a["tokens"], a["heads"], a["d"], a["ks"], a["vs"],
                         a["slots"], a["kc"], a["vc"], a["pages"], a["page"], None)


def load(**kw):
    a = dict(ADDR, codec=2, dt=1, tokens=3, heads=2, d=64, pages=4, page=16)
    a.update(kw)
    return L.kq_kv_load(a["codec"], a["kc"], a["vc"], a["pages"], a["page"], a["heads"], a["d"], a["slots"],
                        a["tokens"], a["k"], a["v"], a["dt"], None)


def attn(**kw):
    a = dict(ADDR, codec=2, qdt=1, tokens=3, hq=8, hkv=2, d=64, stride=512, n=2, width=4, pages=4, page=16, scale=0.1,
             window=0, max_new=2, max_kv=64, odt=1, ws_bytes=0)
    a.update(kw)
    return L.kq_kv_attention(a["codec"], a["q"], a["qdt"], a["tokens"], a["hq"], a["hkv"], a["d"], a["stride"],
                             a["cu"], a["lens"], a["n"], a["table"], a["width"], a["kc"], a["vc"], a["pages"],
                             a["page"], a["scale"], a["window"], a["max_new"], a["max_kv"], a["out"], a["odt"],
                             a["ws"], a["ws_bytes"], None)


ARG, CODEC, SHAPE, ALIGN, CAP = kq.KQ_ERR_ARG, kq.KQ_ERR_CODEC, kq.KQ_ERR_SHAPE, kq.KQ_ERR_ALIGN, kq.KQ_ERR_CAPACITY


@pytest.mark.parametrize("call, kw, status, msg", [
    (tables, dict(page=24), SHAPE, "page=24"),
    (tables, dict(page=8), SHAPE, "page=8"),
    (tables, dict(page=8192), SHAPE, "page=8192"),
    (tables, dict(n=-1), ARG, "n_seqs"),
    (tables, dict(n=(1 << 20) + 1), ARG, "n_seqs"),
    (tables, dict(n_free=-1), ARG, "n_free"),
    (tables, dict(width=-1), ARG, "width"),
    (tables, dict(tokens=-1), ARG, "tokens"),
    (tables, dict(head=None), ARG, "null"),
    (tables, dict(cu=None), ARG, "null"),
    (tables, dict(lens=None), ARG, "null"),
    (tables, dict(slots=None), ARG, "null"),
    (tables, dict(free=None), ARG, "null"),
    (tables, dict(slots=ADDR["slots"] + 2), ALIGN, "aligned"),
    (tables, dict(ctx=ADDR["ctx"] + 1), ALIGN, "aligned"),
    (tables, dict(head_out=ADDR["head"]), ARG, "overlaps an input"),
    (tables, dict(lens=ADDR["ctx"] + 12), ARG, "overlaps an input"),
    (tables, dict(cu=ADDR["slots"] + 36), ARG, "two outputs"),
    (tables, dict(status=ADDR["head_out"]), ARG, "two outputs"),
    (store, dict(codec=8), CODEC, "q4_0"),
    (store, dict(d=48), SHAPE, "d=48"),
    (store, dict(d=288, ks=1000, vs=1000), SHAPE, "d=288"),
    (store, dict(d=0), SHAPE, "d=0"),
    (store, dict(heads=0), ARG, "kv_heads"),
    (store, dict(dt=5), ARG, "dtype 5"),
    (store, dict(tokens=-2), ARG, "tokens"),
    (store, dict(tokens=1 << 30), ARG, "tokens"),
    (store, dict(ks=120), SHAPE, "strides"),
    (store, dict(vs=132), ALIGN, "multiples of 8"),
    (store, dict(pages=0), ARG, "pages"),
    (store, dict(pages=1 << 28), ARG, "pages"),
    (store, dict(kc=None), ARG, "null cache"),
    (store, dict(vc=ADDR["vc"] + 8), ALIGN, "caches"),
    (store, dict(vc=ADDR["kc"] + 16), ARG, "overlap"),
    (store, dict(k=None), ARG, "null"),
    (store, dict(v=ADDR["v"] + 8), ALIGN, "16-byte"),
    (store, dict(slots=ADDR["slots"] + 1), ALIGN, "slots"),
    (load, dict(codec=12), CODEC, "q4_0"),
    (load, dict(page=100), SHAPE, "page=100"),
    (load, dict(dt=-1), ARG, "dtype"),
    (load, dict(v=ADDR["k"] + 16), ARG, "overlap"),
    (load, dict(k=ADDR["k"] + 4), ALIGN, "16-byte"),
    (load, dict(slots=None), ARG, "null"),
    (tables, dict(n=65537), ARG, "n_seqs"),
    (store, dict(kc=ADDR["k"] + 64), ARG, "overlap a cache"),
    (store, dict(slots=ADDR["vc"] + 4), ARG, "overlap a cache"),
    (load, dict(k=ADDR["vc"] + 16), ARG, "overlaps a cache"),
    (attn, dict(out=ADDR["kc"] + 16), ARG, "out overlaps k_cache"),
    (attn, dict(table=ADDR["out"] + 16), ARG, "out overlaps table"),
    (attn, dict(max_kv=1 << 20, q=ADDR["ws"] + 4096, ws_bytes=1 << 40), ARG, "workspace overlaps q"),
    (attn, dict(codec=3), CODEC, "q4_0"),
    (attn, dict(qdt=0), ARG, "query dtype"),
    (attn, dict(odt=4), ARG, "output dtype"),
    (attn, dict(hq=7), SHAPE, "q_heads=7"),
    (attn, dict(hkv=0), ARG, "kv_heads"),
    (attn, dict(d=80), SHAPE, "d=80"),
    (attn, dict(stride=504), SHAPE, "stride"),
    (attn, dict(stride=516), ALIGN, "stride"),
    (attn, dict(tokens=1 << 22), ARG, "tokens"),
    (attn, dict(n=1 << 21), ARG, "n_seqs"),
    (attn, dict(width=1 << 26), ARG, "width"),
    (attn, dict(scale=float("nan")), ARG, "scale"),
    (attn, dict(scale=float("inf")), ARG, "scale"),
    (attn, dict(window=-1), ARG, "window"),
    (attn, dict(max_new=0), ARG, "max_new"),
    (attn, dict(max_kv=0), ARG, "max_kv"),
    (attn, dict(pages=-1), ARG, "pages"),
    (attn, dict(q=None), ARG, "null"),
    (attn, dict(table=None), ARG, "null"),
    (attn, dict(out=ADDR["out"] + 8), ALIGN, "out="),
    (attn, dict(cu=ADDR["cu"] + 2), ALIGN, "cu_new"),
    (attn, dict(out=ADDR["q"] + 1024), ARG, "out overlaps q"),
    (attn, dict(max_kv=1 << 20), CAP, "workspace of 0 bytes"),
    (attn, dict(max_kv=1 << 20, ws=None, ws_bytes=1 << 40), CAP, "workspace of 0 bytes"),
    (attn, dict(max_kv=1 << 20, ws=ADDR["ws"] + 8, ws_bytes=1 << 40), ALIGN, "workspace="),
    (attn, dict(max_kv=1 << 20, ws=ADDR["out"], ws_bytes=1 << 40), ARG, "workspace overlaps"),
])
def test_refused_before_launch(call, kw, status, msg):
    ret = call(**kw)
    err = kq.kq_last_error()
    assert ret == status, (ret, err)
    assert msg in err and err.startswith("[kq_"), err


def test_empty_calls_do_nothing():
    assert store(tokens=0, k=None, v=None, slots=None) == 0
    assert load(tokens=0, k=None, v=None, slots=None) == 0
    assert attn(tokens=0, q=None, out=None) == 0
    assert attn(n=0, cu=None, lens=None, table=None) == 0


def test_sizes():
    assert kq.kq_kv_page_bytes("q4_0", 64, 128) == 64 * 4 * 18
    with pytest.raises(kq.KQError) as e:
        kq.kq_kv_page_bytes("q8_0", 64, 128)
    assert e.value.status == CODEC
    assert kq.kq_kv_attention_workspace(0, 0, 8, 8, 64, 1, 1) == 0
    assert kq.kq_kv_attention_workspace(1, 1, 32, 8, 128, 1, 100) == 0
    assert kq.kq_kv_attention_workspace(4, 4, 32, 8, 128, 1, 131072) > 0
    with pytest.raises(kq.KQError):
        kq.kq_kv_attention_workspace(1, 1, 6, 4, 64, 1, 1)


def test_binding_checks_shapes():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    kc, vc = (torch.zeros((4, 2, kq.kq_kv_page_bytes("q4_0", 16, 64)), dtype=torch.uint8) for _ in range(2))
    k = torch.zeros((3, 2, 64), dtype=torch.float16)
    with pytest.raises(ValueError, match="slots has 2"):
        kq.kq_kv_store("q4_0", k, k, i32(2), kc, vc, 16)
    with pytest.raises(ValueError, match="dense"):
        kq.kq_kv_store("q4_0", k.transpose(0, 1), k.transpose(0, 1), i32(2), kc, vc, 16)
    with pytest.raises(ValueError, match="cache of 2"):
        kq.kq_kv_store("q4_0", k[:, :1], k[:, :1], i32(3), kc, vc, 16)
    with pytest.raises(ValueError, match="pages hold"):
        kq.kq_kv_load("q4_0", kc, vc, i32(3), 32, k, k.clone())
    with pytest.raises(TypeError, match="int32"):
        kq.kq_kv_load("q4_0", kc, vc, torch.zeros(3, dtype=torch.int64), 16, k, k.clone())
    q = torch.zeros((3, 4, 64), dtype=torch.float16)
    with pytest.raises(ValueError, match="cu_new has 2"):
        kq.kq_kv_attention("q4_0", q, i32(2), i32(2), i32(2, 4), kc, vc, 16, q.clone())
    with pytest.raises(ValueError, match="table"):
        kq.kq_kv_attention("q4_0", q, i32(3), i32(2), i32(8), kc, vc, 16, q.clone())
    with pytest.raises(ValueError, match="contiguous"):
        kq.kq_kv_attention("q4_0", q, i32(3), i32(2), i32(4, 2).T, kc, vc, 16, q.clone())
    with pytest.raises(ValueError, match="table"):
        kq.kq_block_tables(i32(2), i32(2), i32(4), i32(1), 16, i32(3, 2), i32(5), i32(3), i32(2), i32(1))
