"""GPU calls of the 4-bit cache operators through both Python paths: the host module and ctypes."""

import numpy as np
import pytest

from _gpu import dev

pytestmark = pytest.mark.gpu

HQ, KV, D, PAGE, PAGES, TOKENS = 4, 2, 64, 16, 12, 40


@pytest.fixture(scope="module")
def kq():
    from gguf_quant_matmul_amd import kq as mod

    return mod


def _inputs(kq):
    import torch

    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
    rng = np.random.default_rng(31)
    qkv = dev(rng.standard_normal((TOKENS + 2, HQ + 2 * KV, D)).astype(np.float16))
    kc, vc = kq.kv_cache("q4_0", PAGES, KV, PAGE, D)
    fill = lambda *s: torch.full(s, 55, dtype=torch.int32, device="cuda")
    return dict(ctx=i32(0, 0), new=i32(33, 7), free=i32(*range(PAGES)[::-1]), head=i32(0),
                table=torch.full((2, 4), -1, dtype=torch.int32, device="cuda"), slots=fill(TOKENS + 2), cu=fill(3),
                lens=fill(2), head_out=fill(1), status=fill(1), q=qkv[:, :HQ], k=qkv[:, HQ:HQ + KV],
                v=qkv[:, HQ + KV:], kc=kc, vc=vc, ko=torch.zeros((TOKENS + 2, KV, D), dtype=torch.bfloat16, device="cuda"),
                vo=torch.zeros((TOKENS + 2, KV, D), dtype=torch.bfloat16, device="cuda"),
                out=torch.zeros((TOKENS + 2, HQ, D), dtype=torch.float16, device="cuda"))


def _calls(kq, a):
    return [lambda **kw: kq.kq_block_tables(*(kw.get(n, a[n]) for n in ("ctx", "new", "free", "head")), kw.get("page", PAGE),
                                            *(kw.get(n, a[n]) for n in ("table", "slots", "cu", "lens", "head_out",
                                                                        "status"))),
            lambda **kw: kq.kq_kv_store(kw.get("codec", "q4_0"), *(kw.get(n, a[n]) for n in ("k", "v", "slots", "kc", "vc")),
                                        kw.get("page", PAGE)),
            lambda **kw: kq.kq_kv_load(kw.get("codec", "q4_0"), *(kw.get(n, a[n]) for n in ("kc", "vc", "slots")),
                                       kw.get("page", PAGE), *(kw.get(n, a[n]) for n in ("ko", "vo"))),
            lambda **kw: kq.kq_kv_attention(kw.get("codec", "q4_0"),
                                            *(kw.get(n, a[n]) for n in ("q", "cu", "lens", "table", "kc", "vc")),
                                            kw.get("page", PAGE), kw.get("out", a["out"]), scale=kw.get("scale"),
                                            window=kw.get("window", 0), max_new=33, max_kv=kw.get("max_kv", 33),
                                            workspace=kw.get("workspace"))]


@pytest.mark.parametrize("max_kv", [33, 100000])
def test_both_paths_give_the_same(kq, monkeypatch, max_kv):
    import torch

    assert kq._kqcall is not None
    got = []
    for module in (kq._kqcall, None):
        monkeypatch.setattr(kq, "_kqcall", module)
        a = _inputs(kq)
        for call in _calls(kq, a):
            call(max_kv=max_kv)
        torch.cuda.synchronize()
        got.append([a[n].cpu() for n in ("table", "slots", "cu", "lens", "head_out", "status", "kc", "vc", "ko", "vo", "out")])
    assert got[0][5].item() == 0 and got[0][10][:TOKENS].abs().sum() > 0 and not got[0][10][TOKENS:].any()
    for x, y in zip(*got):
        assert torch.equal(x, y)


def test_both_paths_refuse_the_same(kq, monkeypatch):
    import torch

    a = _inputs(kq)
    tables, store, load, attn = _calls(kq, a)
    i64 = torch.zeros(TOKENS + 2, dtype=torch.int64, device="cuda")
    cases = [(tables, dict(ctx=a["ctx"].float())), (tables, dict(new=a["new"][:1])), (tables, dict(cu=a["cu"][:2])),
             (tables, dict(table=a["table"].T)), (tables, dict(page=24)), (tables, dict(lens=a["ctx"])),
             (tables, dict(free=a["free"].cpu())),
             (store, dict(codec="q8_0")), (store, dict(page=32)), (store, dict(slots=i64)), (store, dict(slots=a["slots"][1:])),
             (store, dict(k=a["k"].float())), (store, dict(k=a["k"][:, :1])), (store, dict(k=a["k"].transpose(0, 1))),
             (store, dict(kc=a["kc"].transpose(0, 1))), (store, dict(kc=a["vc"])), (store, dict(kc=a["kc"].int())),
             (store, dict(v=a["v"][:, :, 1:].expand(-1, -1, -1))), (store, dict(slots=a["slots"].cpu())),
             (store, dict(k=a["k"][:, :, :63], v=a["v"][:, :, :63])), (store, dict(k=a["k"][:1].expand(TOKENS + 2, -1, -1))),
             (load, dict(ko=a["ko"][::2])), (load, dict(ko=a["vo"])), (load, dict(vc=a["vc"][1:])), (load, dict(ko=a["ko"].int())),
             (attn, dict(q=a["q"].float())), (attn, dict(out=a["out"][1:])), (attn, dict(out=a["q"])), (attn, dict(cu=a["lens"])),
             (attn, dict(q=a["q"][:, :3], out=a["out"][:, :3].contiguous())), (attn, dict(scale=float("nan"))),
             (attn, dict(window=-1)), (attn, dict(max_kv=0)), (attn, dict(table=a["table"].long())),
             (attn, dict(max_kv=100000, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))),
             (attn, dict(max_kv=100000, workspace=torch.empty(1 << 26, dtype=torch.uint8))),
             (attn, dict(kc=a["kc"].cpu(), vc=a["vc"].cpu()))]
    want = {n: a[n].clone() for n in a}
    for i, (call, kw) in enumerate(cases):
        errors = []
        for module in (kq._kqcall, None):
            with monkeypatch.context() as m:
                m.setattr(kq, "_kqcall", module)
                with pytest.raises((ValueError, TypeError, kq.KQError)) as e:
                    call(**kw)
                # (the path through ctypes may ask for the workspace first, which names itself)
                errors.append((e.type, str(e.value).replace("_workspace]", "]")))
        assert errors[0] == errors[1], (i, list(kw), errors)
    torch.cuda.synchronize()
    for n in a:
        assert torch.equal(a[n], want[n]), n
