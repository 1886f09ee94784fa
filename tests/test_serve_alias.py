"""Queries turned in place beside keys and values: the refusal of shared
elements (csrc/q4_kv.h, compiled for the host) against a brute-force search,
and through the C ABI."""
import ctypes
import itertools
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import bit_weight_only_int4_amd as q4
from tests.gpu_util import need_gpu
from tests.test_serve_abi import ALIAS, APPEND, PTR, call
from tests.test_serve_index import CSRC

SHIM = """
#include "q4_kv.h"
extern "C" int share(int64_t delta, int64_t T, int64_t dim, int64_t ats, int64_t ahs, int64_t ah, int64_t bts, int64_t bhs,
                     int64_t bh) {
  return q4::rows_share(delta, T, dim, ats, ahs, ah, bts, bhs, bh);
}
"""


@pytest.fixture(scope="module")
def share(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("alias")
    (d / "shim.cpp").write_text(SHIM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", f"-I{CSRC}", str(d / "shim.cpp"), "-o", str(d / "shim.so")],
                   check=True)
    f = ctypes.CDLL(os.path.join(str(d), "shim.so")).share
    f.argtypes = [ctypes.c_int64] * 9
    return lambda *a: bool(f(*a))


def elements(at, T, dim, ts, hs, heads):
    return {at + t * ts + h * hs + e for t in range(T) for h in range(heads) for e in range(dim)}


def test_layouts_of_a_fused_projection(share):
    D, Hq, Hk = 64, 8, 2
    row = (Hq + 2 * Hk) * D
    for T in (1, 2, 50):
        assert not share(Hq * D, T, D, row, D, Hq, row, D, Hk)                # q heads, then k, then v
        assert not share((Hq + Hk) * D, T, D, row, D, Hq, row, D, Hk)
        assert not share(-2 * Hk * D, T, D, row, D, Hq, row, D, Hk)           # q last
        assert not share(D, T, D, 3 * Hk * D, 3 * D, Hk, 3 * Hk * D, 3 * D, Hk)  # q, k, v of each head in turn
        assert share(0, T, D, row, D, Hq, row, D, Hk)                         # keys among the queries
        assert share((Hq - 1) * D, T, D, row, D, Hq, row, D, Hk)
        assert share((Hq - 1) * D + D // 2, T, D, row, D, Hq, row, D, 1)
    assert share(row, 2, D, row, D, Hq, row, D, Hk) and not share(row, 1, D, row, D, Hq, row, D, Hk)


def test_against_a_search(share):
    g = np.random.default_rng(0)
    seen = [0, 0]
    for _ in range(4000):
        dim, T, ah, bh = int(g.integers(1, 4)), int(g.integers(1, 5)), int(g.integers(1, 4)), int(g.integers(1, 4))
        ahs, bhs = (int(dim + g.integers(0, 9)) for _ in range(2))
        ts = int(dim + g.integers(0, 40))
        delta = int(g.integers(-60, 60))
        want = bool(elements(0, T, dim, ts, ahs, ah) & elements(delta, T, dim, ts, bhs, bh))
        assert share(delta, T, dim, ts, ahs, ah, ts, bhs, bh) == want, (delta, T, dim, ts, ahs, ah, bhs, bh)
        seen[want] += 1
    assert min(seen) > 500


def test_the_abi_refuses_keys_among_the_queries():
    fused = dict(qt=768, qot=768, kt=768, vt=768, q=PTR["q"], qo=PTR["q"])
    for (at, name), head in itertools.product((("k", "v"), ("v", "k")), (0, 3, 7)):
        place = {at: PTR["q"] + 4 * 64 * head, name: PTR["q"] + 4 * 64 * 8}
        assert call("q4_kv_append", APPEND, **fused, **place) == ALIAS, (at, head)
    # all three the same tensor
    same = dict(q=PTR["q"], qo=PTR["q"], k=PTR["q"], v=PTR["q"], heads=4, qt=256, qot=256)
    assert call("q4_kv_append", APPEND, **same) == ALIAS
    # other token strides
    assert call("q4_kv_append", APPEND, **{**fused, "kt": 512}, k=PTR["q"] + 4 * 64 * 8, v=PTR["v"]) == ALIAS


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["q k v", "k v q", "q k v of each head"])
def test_queries_turned_in_place_beside_keys_and_values(layout):
    need_gpu()
    T, H, D = 21, 3, 64
    G = 1 if "each" in layout else 4
    if G == 1:
        q, k, v = torch.randn((T, H, 3, D), device="cuda").unbind(2)
    elif layout == "q k v":
        q, k, v = torch.randn((T, (G + 2) * H, D), device="cuda").split([G * H, H, H], 1)
    else:
        k, v, q = torch.randn((T, (G + 2) * H, D), device="cuda").split([H, H, G * H], 1)
    freq = (10000.0 ** (-torch.arange(0, D, 2, device="cuda") / D))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    tables = i32([[1, 2, 0]]), i32([0, T]), i32([T + 9])
    apart, beside = q4.new_cache(3, H, D, 16), q4.new_cache(3, H, D, 16)
    want = q4.kv_append(k.clone(), v.clone(), *apart, *tables, q=q.clone(), inv_freq=freq)
    got = q4.kv_append(k, v, *beside, *tables, q=q, q_out=q, inv_freq=freq)
    assert got.data_ptr() == q.data_ptr() and torch.equal(got, want)
    assert all(torch.equal(a, b) for a, b in zip(apart, beside))
    with pytest.raises(q4.Q4Error):
        q4.kv_append(k, v, *beside, *tables, q=k, q_out=k, inv_freq=freq)
