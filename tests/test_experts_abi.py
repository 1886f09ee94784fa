"""The C ABI of include/q4experts.h on the host, and the binding's refusals:
every invalid argument is rejected before anything is queued.  No compute call
is made; the pointers are placeholders that nothing dereferences."""
import os
import re

import pytest
import torch

import bit_weight_only_int4_amd as q4
from bit_weight_only_int4_amd import mixture

HEADER = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "q4experts.h")
OK, INVALID, ALIAS, WORKSPACE, UNSUPPORTED = 0, 1, 2, 3, 4
PTR = {n: (i + 1) << 36 for i, n in enumerate(
    ("z", "bias", "ids", "w", "g", "dz", "x", "gu", "gus", "dn", "dns", "out", "pre", "ws", "dx", "dw",
     "qw", "s", "t", "loss", "lse"))}


def test_every_declared_symbol_is_exported():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"^\s*[A-Za-z_][\w \*]*?\b(q4_\w+)\s*\(", text, flags=re.M)))
    assert names == sorted(mixture.SYMBOLS)
    for n in names:
        assert hasattr(mixture._lib(), n)


ROUTE = dict(z=PTR["z"], ld=64, dtype=0, T=10, E=64, k=8, score=0, bias=PTR["bias"], groups=8, top=4, renorm=1,
             scale=1.0, ids=PTR["ids"], w=PTR["w"], stream=None)
ROUTE_BACK = dict(z=PTR["z"], ld=64, dtype=0, T=10, E=64, k=8, ids=PTR["ids"], score=0, renorm=1, scale=1.0,
                  g=PTR["g"], dz=PTR["dz"], ldd=64, stream=None)
EXPERTS = dict(x=PTR["x"], ldx=256, dtype=0, T=10, H=256, W=128, E=8, k=2, ids=PTR["ids"], w=PTR["w"], gu=PTR["gu"],
               gus=PTR["gus"], dn=PTR["dn"], dns=PTR["dns"], gs=32, order=0, out=PTR["out"], ldo=256, pre=PTR["pre"],
               ws=PTR["ws"], wsn=1 << 30, stream=None)
EXPERTS_BACK = dict(d=PTR["x"], ldd=256, dtype=0, T=10, H=256, W=128, E=8, k=2, ids=PTR["ids"], w=PTR["w"],
                    pre=PTR["pre"], gu=PTR["gu"], gus=PTR["gus"], dn=PTR["dn"], dns=PTR["dns"], gs=32, order=0,
                    dx=PTR["dx"], lddx=256, dw=PTR["dw"], ws=PTR["ws"], wsn=1 << 30, stream=None)
HEAD = dict(x=PTR["x"], ldx=256, dtype=0, M=10, V=1000, K=256, qw=PTR["qw"], s=PTR["s"], gs=32, order=0, t=PTR["t"],
            loss=PTR["loss"], lse=PTR["lse"], ws=PTR["ws"], wsn=1 << 30, stream=None)
HEAD_BACK = dict(x=PTR["x"], ldx=256, dtype=0, M=10, V=1000, K=256, qw=PTR["qw"], s=PTR["s"], gs=32, order=0,
                 t=PTR["t"], lse=PTR["lse"], g=PTR["g"], dx=PTR["dx"], lddx=256, ws=PTR["ws"], wsn=1 << 30, stream=None)
CALLS = {"q4_route": ROUTE, "q4_route_backward": ROUTE_BACK, "q4_experts": EXPERTS, "q4_experts_backward": EXPERTS_BACK,
         "q4_head_cross_entropy": HEAD, "q4_head_cross_entropy_backward": HEAD_BACK}


def call(name, **kw):
    assert set(kw) <= set(CALLS[name])
    return getattr(mixture._lib(), name)(*{**CALLS[name], **kw}.values())


@pytest.mark.parametrize("name", list(CALLS))
def test_missing_and_misaligned_pointers(name):
    optional = {"bias", "pre"} if name in ("q4_route", "q4_experts") else set()
    for field, value in CALLS[name].items():
        if field in PTR and value == PTR[field] or field == "d":
            if field == "ws":
                assert call(name, ws=None) == WORKSPACE and call(name, ws=PTR["ws"] + 8) == WORKSPACE
                continue
            if field not in optional:
                assert call(name, **{field: None}) == INVALID, field
            assert call(name, **{field: value + 1}) == INVALID, field


@pytest.mark.parametrize("field,value", [
    ("dtype", 3), ("dtype", -1), ("T", -1), ("T", 1 << 24), ("E", 0), ("E", 1025), ("k", 0), ("k", 33), ("score", 2),
    ("score", -1), ("renorm", 2), ("groups", 0), ("groups", 7), ("top", 0), ("top", 9), ("ld", 63), ("ld", -1),
    ("scale", float("nan")), ("scale", float("inf"))])
def test_route_refusals(field, value):
    assert call("q4_route", **{field: value}) == INVALID
    if field in ROUTE_BACK:
        assert call("q4_route_backward", **{field: value}) == INVALID


def test_route_group_and_alias_refusals():
    assert call("q4_route", groups=16, top=1, k=5) == INVALID  # 4 experts are left
    assert call("q4_route_backward", E=4, ld=4, ldd=4, k=5) == INVALID
    assert call("q4_route_backward", ldd=63) == INVALID
    assert call("q4_route", w=PTR["ids"] + 16) == ALIAS
    assert call("q4_route", ids=PTR["z"] + 64) == ALIAS
    assert call("q4_route_backward", dz=PTR["z"], ldd=65) == ALIAS
    assert call("q4_route_backward", dz=PTR["g"]) == ALIAS


@pytest.mark.parametrize("name", ["q4_experts", "q4_experts_backward"])
@pytest.mark.parametrize("field,value,status", [
    ("dtype", 3, INVALID), ("T", -1, INVALID), ("T", 1 << 24, INVALID), ("T", 1 << 23, INVALID), ("H", 0, INVALID),
    ("H", 252, INVALID), ("H", 1 << 17, INVALID), ("W", 4, INVALID), ("W", 132, INVALID), ("E", 0, INVALID),
    ("E", 1025, INVALID), ("k", 0, INVALID), ("k", 33, INVALID), ("gs", -1, INVALID), ("gs", 16, UNSUPPORTED),
    ("gs", 96, UNSUPPORTED), ("gs", 100, UNSUPPORTED), ("order", 2, INVALID), ("wsn", 1000, WORKSPACE)])
def test_experts_refusals(name, field, value, status):
    assert call(name, **{field: value}) == status


def test_experts_alias_refusals():
    for f in ("x", "ids", "w", "gu", "gus", "dn", "dns", "pre", "ws"):
        assert call("q4_experts", out=PTR[f]) == ALIAS, f
    assert call("q4_experts", ws=PTR["x"] + 64) == ALIAS
    assert call("q4_experts", ldx=255) == INVALID and call("q4_experts", ldo=200) == INVALID
    for f in ("x", "ids", "w", "pre", "gu", "gus", "dn", "dns", "ws", "dw"):
        assert call("q4_experts_backward", dx=PTR[f]) == ALIAS, f
    assert call("q4_experts_backward", ldd=255) == INVALID and call("q4_experts_backward", lddx=9) == INVALID


@pytest.mark.parametrize("name", ["q4_head_cross_entropy", "q4_head_cross_entropy_backward"])
@pytest.mark.parametrize("field,value,status", [
    ("dtype", 3, INVALID), ("M", -1, INVALID), ("M", 1 << 24, INVALID), ("V", 0, INVALID), ("V", 1 << 31, INVALID),
    ("K", 0, INVALID), ("K", 252, INVALID), ("gs", -32, INVALID), ("gs", 48, UNSUPPORTED), ("order", -1, INVALID),
    ("ldx", 255, INVALID), ("wsn", 1000, WORKSPACE)])
def test_head_refusals(name, field, value, status):
    assert call(name, **{field: value}) == status


def test_head_alias_refusals():
    assert call("q4_head_cross_entropy", loss=PTR["lse"]) == ALIAS
    assert call("q4_head_cross_entropy", lse=PTR["t"]) == ALIAS
    assert call("q4_head_cross_entropy", ws=PTR["qw"]) == ALIAS
    for f in ("x", "qw", "s", "t", "lse", "g", "ws"):
        assert call("q4_head_cross_entropy_backward", dx=PTR[f]) == ALIAS, f
    assert call("q4_head_cross_entropy_backward", lddx=255) == INVALID


def test_nothing_to_do():
    """No tokens or rows: valid without any array."""
    none = {f: None for f in PTR}
    assert call("q4_route", **{**{f: None for f in ("z", "bias", "ids", "w")}, "T": 0}) == OK
    assert call("q4_experts", T=0, x=None, ids=None, w=None, out=None, pre=None, ws=None) == OK
    assert call("q4_experts_backward", T=0, d=None, dx=None, dw=None, ws=None) == OK
    assert call("q4_head_cross_entropy", M=0, **{f: none[f] for f in ("x", "t", "loss", "lse", "ws")}) == OK
    assert call("q4_head_cross_entropy_backward", M=0, x=None, dx=None, ws=None) == OK


def test_workspace_sizes():
    f, b = q4.experts_workspace_bytes, q4.experts_backward_workspace_bytes
    assert f(10, 256, 128, 8, 2, group_size=32) >= 10 * 2 * (256 + 128) * 4
    assert f(0, 256, 128, 8, 2, group_size=32) == 0 and f(10, 250, 128, 8, 2, group_size=32) == 0
    assert f(10, 256, 128, 8, 2, group_size=48) == 0 and b(10, 256, 128, 8, 2, group_size=48) == 0
    assert b(10, 256, 128, 8, 2, group_size=0) >= 10 * 2 * (2 * 128 + 256) * 4
    h = q4.head_cross_entropy_workspace_bytes
    # statistics of tiles, not logits
    assert 0 < h(2048, 128257, 2048, group_size=0) < 2048 * 128257 // 4
    # rows are taken 8192 at a time
    assert h(1 << 20, 128257, 2048, group_size=0) == h(8192, 128257, 2048, group_size=0)
    hb = q4.head_cross_entropy_backward_workspace_bytes
    assert 0 < hb(2048, 128257, 2048, group_size=0) < 2048 * 128257 * 4
    assert hb(1 << 20, 128257, 2048, group_size=0) == hb(8192, 128257, 2048, group_size=0)


X, IDS, WT = torch.zeros(4, 64), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
WEIGHTS = [torch.zeros(3, 64, 32, dtype=torch.uint8), torch.zeros(3, 2, 64), torch.zeros(3, 64, 16, dtype=torch.uint8),
           torch.zeros(3, 1, 64)]


def experts(x=X, ids=IDS, w=WT, weights=WEIGHTS, **kw):
    return q4.experts(x, ids, w, *weights, **{"group_size": 32, **kw})


def swapped(i, t):
    return [t if j == i else w for j, w in enumerate(WEIGHTS)]


@pytest.mark.parametrize("kw,text", [
    (dict(x=X.double()), "float32, float16 or bfloat16"), (dict(x=X[0]), "2-D|hidden"), (dict(x="x"), "must be a tensor"),
    (dict(x=X.t()), "unit stride|gate_up|ids"), (dict(ids=IDS.long()), "ids"), (dict(ids=IDS[:3]), "ids"),
    (dict(ids=IDS[:, 0]), "ids"), (dict(w=WT.half()), "weights"), (dict(w=WT[:, :1]), "weights"),
    (dict(weights=swapped(0, WEIGHTS[0][:, :63])), "gate_up"), (dict(weights=swapped(0, WEIGHTS[0].int())), "gate_up"),
    (dict(weights=swapped(0, WEIGHTS[0][:, :, :31])), "gate_up"), (dict(weights=swapped(1, torch.zeros(3, 64))), "gate_up_scales"),
    (dict(weights=swapped(2, WEIGHTS[2][:2])), "down"), (dict(weights=swapped(3, torch.zeros(3, 1, 64).half())), "down_scales"),
    (dict(group_size=-1), "group_size"), (dict(nibble_order="both"), "nibble_order"), (dict(out=torch.zeros(4, 63)), "out"),
    (dict(out=torch.zeros(4, 64).half()), "out"), (dict(), "device tensor")])
def test_experts_binding_refusals(kw, text):
    with pytest.raises(ValueError, match=text):
        experts(**kw)


def test_other_binding_refusals():
    z = torch.zeros(3, 16)
    for kw, text in ((dict(score="relu"), "score"), (dict(groups=3), "groups"), (dict(groups=4, top_groups=5), "top_groups"),
                     (dict(bias=torch.zeros(15)), "bias"), (dict(), "device tensor")):
        with pytest.raises(ValueError, match=text):
            q4.route(z, 4, **kw)
    for k in (0, 17, 33):
        with pytest.raises(ValueError, match="top_k"):
            q4.route(z, k)
    with pytest.raises(ValueError, match="top_k"):
        q4.route(z, 5, groups=4, top_groups=1)
    with pytest.raises(ValueError, match="float32, float16"):
        q4.route(z.int(), 4)
    with pytest.raises(ValueError, match="g_weights"):
        q4.route_backward(z, torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, 5))
    with pytest.raises(ValueError, match="dlogits"):
        q4.route_backward(z, torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, 4), dlogits=torch.zeros(3, 15))
    with pytest.raises(ValueError, match="pre"):
        q4.experts_backward(X, IDS, WT, torch.zeros(4, 2, 63), *WEIGHTS, group_size=32)
    with pytest.raises(ValueError, match="device tensor"):
        q4.experts_backward(X, IDS, WT, torch.zeros(4, 2, 64), *WEIGHTS, group_size=32)
    qw, s, t = torch.zeros(10, 32, dtype=torch.uint8), torch.zeros(2, 10), torch.zeros(4, dtype=torch.int64)
    for args, text in (((X[:, :60], qw, s, t), "multiple of 8"), ((X, qw[:, :31], s, t), "qw"), ((X, qw, s[:1], t), "scales"),
                       ((X, qw, s, t[:3]), "targets"), ((X, qw, s, t.int()), "targets"), ((X, qw, s, t), "device tensor")):
        with pytest.raises(ValueError, match=text):
            q4.head_cross_entropy(*args, group_size=32)
    with pytest.raises(ValueError, match="g_loss"):
        q4.head_cross_entropy_backward(X, qw, s, t, torch.zeros(4), torch.zeros(3), group_size=32)
    with pytest.raises(ValueError, match="lse"):
        q4.head_cross_entropy_backward(X, qw, s, t, None, torch.zeros(4), group_size=32)
