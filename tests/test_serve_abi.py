"""The C ABI of include/q4serve.h on the host, and the binding's refusals:
every invalid argument is rejected before anything is queued.  No compute
call is made; the pointers are placeholders that nothing dereferences."""
import ctypes
import os
import re

import pytest
import torch

import bit_weight_only_int4_amd as q4
from bit_weight_only_int4_amd import serve

HEADER = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "q4serve.h")
OK, INVALID, ALIAS, WORKSPACE = 0, 1, 2, 3


def test_every_declared_symbol_is_exported():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"^\s*[A-Za-z_][\w \*]*?\b(q4_\w+)\s*\(", text, flags=re.M)))
    assert names == sorted(serve.SYMBOLS)
    L = serve._lib()
    for n in names:
        assert hasattr(L, n)


PTR = {n: (i + 1) << 32 for i, n in enumerate(
    ("k", "v", "q", "qo", "kc", "vc", "ks", "vs", "table", "cu", "len", "freq", "ws", "x", "t", "lp",
     "ent", "lse", "ids", "top", "dx", "gl", "ge"))}

APPEND = dict(k=PTR["k"], kt=256, kh=64, v=PTR["v"], vt=256, vh=64, q=PTR["q"], qt=512, qh=64,
              qo=PTR["qo"], qot=512, qoh=64, dtype=0, T=10, B=3, heads=8, kv=4, dim=64, kc=PTR["kc"],
              vc=PTR["vc"], ks=PTR["ks"], vs=PTR["vs"], pages=20, page=16, table=PTR["table"], ld=7,
              cols=7, cu=PTR["cu"], len=PTR["len"], max_new=4, freq=PTR["freq"], rot=64, inter=0, stream=None)
ATTN = dict(q=PTR["q"], qt=512, qh=64, o=PTR["qo"], ot=512, oh=64, dtype=0, T=10, B=3, heads=8, kv=4,
            dim=64, kc=PTR["kc"], vc=PTR["vc"], ks=PTR["ks"], vs=PTR["vs"], pages=20, page=16,
            table=PTR["table"], ld=7, cols=7, cu=PTR["cu"], len=PTR["len"], max_new=4, max_len=100,
            scale=0.125, window=0, ws=None, wsn=0, stream=None)
LOGP = dict(x=PTR["x"], ld=1000, dtype=0, M=300, V=1000, t=PTR["t"], k=5, lp=PTR["lp"], ent=PTR["ent"],
            lse=PTR["lse"], ids=PTR["ids"], top=PTR["top"], ws=None, wsn=0, stream=None)
GRAD = dict(x=PTR["x"], ld=1000, dtype=0, M=300, V=1000, t=PTR["t"], lse=PTR["lse"], ent=PTR["ent"],
            gl=PTR["gl"], ge=PTR["ge"], dx=PTR["dx"], ldd=1000, stream=None)


def call(name, base, **kw):
    assert set(kw) <= set(base)
    return getattr(serve._lib(), name)(*{**base, **kw}.values())


@pytest.mark.parametrize("field,value", [
    ("k", None), ("v", None), ("kc", None), ("vc", None), ("ks", None), ("vs", None), ("table", None),
    ("cu", None), ("len", None), ("qo", None), ("freq", None), ("dtype", 3), ("dtype", -1), ("T", -1),
    ("B", -1), ("T", 1 << 31), ("heads", 6), ("heads", 0), ("kv", 0), ("dim", 8), ("dim", 72), ("dim", 272),
    ("kt", 255), ("kh", 63), ("vh", 63), ("qt", 511), ("qoh", 0), ("pages", 0), ("page", 8), ("page", 48),
    ("page", 256), ("ld", 6), ("cols", 0), ("max_new", 0), ("max_new", -1), ("rot", 63), ("rot", 66),
    ("rot", -2), ("inter", 2), ("kc", PTR["kc"] + 8), ("vc", PTR["vc"] + 4), ("k", PTR["k"] + 2),
    ("ks", PTR["ks"] + 1), ("table", PTR["table"] + 2)])
def test_append_refusals(field, value):
    assert call("q4_kv_append", APPEND, **{field: value}) == INVALID


def test_append_aliases_and_noops():
    for f, p in (("qo", "k"), ("qo", "q"), ("qo", "kc"), ("k", "kc"), ("v", "vc"), ("ks", "vs"), ("freq", "ks")):
        assert call("q4_kv_append", APPEND, **{f: PTR[p] + (64 if f == "qo" and p == "q" else 0)}) == ALIAS, (f, p)
    assert call("q4_kv_append", APPEND, T=0, k=None, v=None) == OK
    assert call("q4_kv_append", APPEND, B=0) == OK


@pytest.mark.parametrize("field,value", [
    ("q", None), ("o", None), ("kc", None), ("vs", None), ("table", None), ("cu", None), ("len", None),
    ("dtype", 3), ("T", -1), ("B", -1), ("heads", 6), ("kv", 3), ("dim", 264), ("dim", 0), ("qt", 511),
    ("oh", 32), ("pages", 0), ("page", 0), ("ld", 6), ("cols", 0), ("max_new", 0), ("max_new", -1),
    ("max_len", -1), ("max_len", 1 << 31), ("window", -1), ("scale", float("nan")), ("scale", float("inf")),
    ("q", PTR["q"] + 2), ("o", PTR["qo"] + 1), ("kc", PTR["kc"] + 1)])
def test_attention_refusals(field, value):
    assert call("q4_attention", ATTN, **{field: value}) == INVALID


def test_attention_aliases_workspace_and_noops():
    for p in ("q", "kc", "vc", "ks", "vs", "table", "cu", "len"):
        assert call("q4_attention", ATTN, o=PTR[p]) == ALIAS, p
    need = serve._lib().q4_attention_workspace_bytes(0, 10, 3, 8, 4, 64, 16, 4, 100000, 0)
    assert need > 0
    long = dict(max_len=100000, ws=PTR["ws"])
    assert call("q4_attention", ATTN, max_len=100000) == WORKSPACE
    assert call("q4_attention", ATTN, **long, wsn=need - 1) == WORKSPACE
    assert call("q4_attention", ATTN, max_len=100000, ws=PTR["ws"] + 4, wsn=need) == WORKSPACE
    assert call("q4_attention", ATTN, max_len=100000, ws=PTR["kc"], wsn=need) == ALIAS
    assert call("q4_attention", ATTN, max_len=100000, ws=PTR["qo"], wsn=need) == ALIAS
    assert call("q4_attention", ATTN, T=0) == OK and call("q4_attention", ATTN, B=0) == OK
    for bad in ((0, -1, 3, 8, 4, 64, 16, 4, 100, 0), (9, 10, 3, 8, 4, 64, 16, 4, 100, 0), (0, 10, 3, 8, 0, 64, 16, 4, 100, 0)):
        assert serve._lib().q4_attention_workspace_bytes(*bad) == 0


@pytest.mark.parametrize("field,value", [
    ("x", None), ("ent", None), ("lse", None), ("lp", None), ("ids", None), ("top", None), ("ld", 999),
    ("ld", -1), ("dtype", 4), ("M", -1), ("V", 0), ("V", 1 << 31), ("k", -1), ("k", 33), ("x", PTR["x"] + 2),
    ("t", PTR["t"] + 4), ("ids", PTR["ids"] + 4), ("lse", PTR["lse"] + 2)])
def test_logprob_refusals(field, value):
    assert call("q4_token_logprobs", LOGP, **{field: value}) == INVALID


def test_logprob_aliases_workspace_and_noops():
    for f in ("lp", "ent", "lse", "ids", "top"):
        assert call("q4_token_logprobs", LOGP, **{f: PTR["x"] + 8}) == ALIAS
    assert call("q4_token_logprobs", LOGP, ent=PTR["lse"]) == ALIAS
    assert call("q4_token_logprobs", LOGP, V=3, ld=1000, k=4) == INVALID
    assert call("q4_token_logprobs", LOGP, M=0, x=None) == OK
    big = dict(M=2, V=100000, ld=100000)
    need = serve._lib().q4_token_logprobs_workspace_bytes(2, 100000, 5, 0)
    assert need > 0 and call("q4_token_logprobs", LOGP, **big) == WORKSPACE
    assert call("q4_token_logprobs", LOGP, **big, ws=PTR["ws"], wsn=need - 1) == WORKSPACE
    assert call("q4_token_logprobs", LOGP, **big, ws=PTR["x"], wsn=need) == ALIAS


@pytest.mark.parametrize("field,value", [
    ("x", None), ("lse", None), ("ent", None), ("dx", None), ("t", None), ("ld", 999), ("ldd", 999),
    ("dtype", 3), ("M", -1), ("V", 0), ("dx", PTR["dx"] + 1), ("gl", PTR["gl"] + 2)])
def test_gradient_refusals(field, value):
    assert call("q4_token_logprobs_backward", GRAD, **{field: value}) == INVALID


def test_gradient_aliases_and_noops():
    assert call("q4_token_logprobs_backward", GRAD, gl=None, ge=None) == INVALID
    for p in ("t", "lse", "ent", "gl", "ge"):
        assert call("q4_token_logprobs_backward", GRAD, dx=PTR[p]) == ALIAS
    # in place needs the same pitch
    assert call("q4_token_logprobs_backward", GRAD, dx=PTR["x"], ldd=1001) == ALIAS
    assert call("q4_token_logprobs_backward", GRAD, dx=PTR["x"] + 4) == ALIAS
    assert call("q4_token_logprobs_backward", GRAD, M=0, x=None) == OK


def test_dequant_refusals():
    base = dict(kc=PTR["kc"], vc=PTR["vc"], ks=PTR["ks"], vs=PTR["vs"], pages=4, kv=2, page=16, dim=64,
                dtype=0, k=PTR["k"], v=PTR["v"], stream=None)
    for f, v in (("kc", None), ("v", None), ("page", 24), ("dim", 24), ("dtype", 7), ("kv", 0), ("pages", -1),
                 ("k", PTR["k"] + 8)):
        assert call("q4_kv_dequant", base, **{f: v}) == INVALID, f
    assert call("q4_kv_dequant", base, k=PTR["kc"]) == ALIAS and call("q4_kv_dequant", base, k=PTR["v"]) == ALIAS
    assert call("q4_kv_dequant", base, pages=0) == OK


def i32(*v):
    return torch.tensor(v, dtype=torch.int32)


def binding_args(op, **kw):
    """Arguments that pass every check but the last, that they are on a GPU."""
    c = dict(zip(("k_cache", "v_cache", "k_scale", "v_scale"), q4.new_cache(4, 2, 64, 16, device="cpu")))
    tables = dict(page_table=i32(0, 1)[None], cu_new=i32(0, 3), lengths=i32(5))
    x = torch.zeros((2, 9))
    a = {"kv_append": dict(k=torch.zeros((3, 2, 64)), v=torch.zeros((3, 2, 64)), **c, **tables,
                           q=torch.zeros((3, 4, 64)), inv_freq=torch.ones(32)),
         "attention": dict(q=torch.zeros((3, 4, 64)), **c, **tables),
         "kv_dequant": c,
         "token_logprobs": dict(logits=x, targets=torch.zeros(2, dtype=torch.int64), top_k=3),
         "token_logprobs_backward": dict(logits=x, targets=torch.zeros(2, dtype=torch.int64), lse=torch.zeros(2),
                                         entropy=torch.zeros(2), g_logprob=torch.zeros(2))}[op]
    return {**a, **kw}


@pytest.mark.parametrize("op", ["kv_append", "attention", "kv_dequant", "token_logprobs", "token_logprobs_backward"])
def test_the_binding_refuses_host_tensors(op):
    with pytest.raises(ValueError, match="must be a device tensor"):
        getattr(q4, op)(**binding_args(op))


CACHE = [("k_cache", torch.zeros((4, 2, 8, 64), dtype=torch.int8)), ("k_cache", torch.zeros((4, 2, 16, 64))),
         ("k_cache", torch.zeros((2, 16, 64), dtype=torch.int8)), ("v_cache", torch.zeros((4, 2, 16, 64), dtype=torch.int8)),
         ("v_cache", torch.zeros((4, 2, 16, 64), dtype=torch.int8).transpose(2, 3)),
         ("v_cache", torch.zeros((5, 2, 64, 16), dtype=torch.int8)), ("k_scale", torch.zeros((4, 2), dtype=torch.float64)),
         ("v_scale", torch.zeros((4, 1))), ("v_scale", torch.zeros((2, 4)).t())]
TABLES = [("page_table", i32(0, 1)), ("page_table", torch.zeros((1, 2), dtype=torch.int64)),
          ("page_table", torch.zeros((4, 1), dtype=torch.int32).t()[:, ::2]), ("page_table", torch.zeros((2, 2), dtype=torch.int32)),
          ("cu_new", i32(0)), ("cu_new", torch.tensor([0, 3])), ("lengths", i32(5, 5)), ("lengths", torch.tensor([5.0])),
          ("lengths", [5])]


@pytest.mark.parametrize("op,name,value", [
    *(("kv_append", *b) for b in CACHE + TABLES), *(("attention", *b) for b in CACHE + TABLES),
    *(("kv_dequant", *b) for b in CACHE), ("kv_dequant", "dtype", torch.int8),
    ("kv_append", "k", torch.zeros((3, 3, 64))), ("kv_append", "k", torch.zeros((3, 2, 64), dtype=torch.float64)),
    ("kv_append", "v", torch.zeros((2, 2, 64))), ("kv_append", "v", torch.zeros((3, 2, 64), dtype=torch.float16)),
    ("kv_append", "k", torch.zeros((3, 64, 2)).transpose(1, 2)), ("kv_append", "q", torch.zeros((3, 5, 64))),
    ("kv_append", "q", torch.zeros((2, 4, 64))), ("kv_append", "q_out", torch.zeros((3, 2, 64))),
    ("kv_append", "inv_freq", torch.ones(33)), ("kv_append", "inv_freq", torch.ones(32, dtype=torch.float64)),
    ("kv_append", "inv_freq", torch.ones(64)[::2]),
    ("attention", "q", torch.zeros((3, 3, 64))), ("attention", "q", torch.zeros((3, 4, 32))),
    ("attention", "q", torch.zeros((3, 4, 64), dtype=torch.int32)), ("attention", "q", torch.zeros((3, 256))),
    ("attention", "out", torch.zeros((3, 4, 64), dtype=torch.float16)), ("attention", "out", torch.zeros((2, 4, 64))),
    ("token_logprobs", "logits", torch.zeros(9)), ("token_logprobs", "logits", torch.zeros((9, 2)).t()),
    ("token_logprobs", "logits", torch.zeros((2, 0))), ("token_logprobs", "logits", torch.zeros((2, 9), dtype=torch.int32)),
    ("token_logprobs", "targets", torch.zeros(3, dtype=torch.int64)), ("token_logprobs", "targets", i32(0, 0)),
    ("token_logprobs", "top_k", 10), ("token_logprobs", "top_k", -1), ("token_logprobs", "top_k", 33),
    ("token_logprobs_backward", "lse", torch.zeros(3)), ("token_logprobs_backward", "entropy", torch.zeros(2).double()),
    ("token_logprobs_backward", "g_logprob", torch.zeros((2, 1))), ("token_logprobs_backward", "g_entropy", torch.zeros(1)),
    ("token_logprobs_backward", "dlogits", torch.zeros((2, 8))),
    ("token_logprobs_backward", "dlogits", torch.zeros((2, 9), dtype=torch.float16))])
def test_the_binding_refuses(op, name, value):
    with pytest.raises(ValueError) as e:
        getattr(q4, op)(**binding_args(op, **{name: value}))
    assert "device tensor" not in str(e.value)


def test_the_binding_refuses_q_out_without_q_and_cache_sizes():
    with pytest.raises(ValueError, match="without q"):
        q4.kv_append(**binding_args("kv_append", q=None, q_out=torch.zeros((3, 4, 64))))
    for page, dim in ((8, 64), (16, 40), (256, 64), (16, 272)):
        with pytest.raises(ValueError):
            q4.new_cache(4, 2, dim, page, device="cpu")


def test_a_status_becomes_q4error():
    """What the library refuses and the binding does not look at."""
    with pytest.raises(q4.Q4Error) as e:
        raise q4.Q4Error(3, "q4_attention")
    assert e.value.status == 3


def test_native_half_and_sources_have_to_match(monkeypatch):
    monkeypatch.setattr(serve, "_module", None)
    monkeypatch.setattr(serve._build, "source_digest", lambda: "0" * 64)
    with pytest.raises(RuntimeError, match="does not match the sources"):
        serve._native()
