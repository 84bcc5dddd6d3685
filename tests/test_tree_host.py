"""Host-side checks of the operators for drafted tokens (no GPU needed): every bad
argument is refused before anything is enqueued; the binding's own checks."""
import ctypes

import pytest
import torch

import sparse_head_attention_gb300 as ea
from sparse_head_attention_gb300 import build as ea_build
from test_cache_ops_host import ALL_BAD, BF16, INVALID, P, UNSUPPORTED, WORKSPACE, _str, cache, paged


@pytest.fixture(scope="module")
def L():
    ea_build.build()
    return ea.lib()


Q4, K4 = _str(8 * 32 * 128, 32 * 128, 128, 1), _str(8 * 8 * 128, 8 * 128, 128, 1)


def _rope(L, **kw):
    a = dict(Q=P, Qo=P, qs=Q4, qos=Q4, Hq=32, K=P, Ko=P, ks=K4, kos=K4, Hkv=8, B=4, T=8, d=128, f=P, rot=128, pos=P, n=None, ws=P, wsb=256)
    a.update(kw)
    return L.ea_rope(a["Q"], a["Qo"], a["qs"], a["qos"], a["Hq"], a["K"], a["Ko"], a["ks"], a["kos"], a["Hkv"], a["B"], a["T"], a["d"], a["f"],
                     a["rot"], 0, ctypes.c_float(1.0), a["pos"], a["n"], a["ws"], a["wsb"], None)


BAD_STRIDES = [_str(8 * 4096, 4096, 128, 2), _str(8 * 4096, 4096, 132, 1), _str(0, 4096, 128, 1), _str(8 * 4096, -4096, 128, 1)]


@pytest.mark.parametrize("kw,expect", [
    (dict(Q=None), INVALID), (dict(Qo=None), INVALID), (dict(K=None), INVALID), (dict(Ko=None), INVALID), (dict(qs=None), INVALID),
    (dict(kos=None), INVALID), (dict(Hq=0, Hkv=0), INVALID), (dict(Hq=-1), INVALID), (dict(Hkv=-1), INVALID), (dict(B=0), INVALID),
    (dict(T=0), INVALID), (dict(f=None), INVALID), (dict(f=P + 4), INVALID), (dict(pos=None), INVALID), (dict(rot=0), INVALID),
    (dict(rot=8), INVALID), (dict(rot=144), INVALID), (dict(rot=72), INVALID), (dict(Q=P + 8), INVALID), (dict(Ko=P + 2), INVALID),
    (dict(d=64), UNSUPPORTED), (dict(B=65536), UNSUPPORTED), (dict(ws=None), WORKSPACE), (dict(ws=P + 64), WORKSPACE),
    (dict(wsb=255), WORKSPACE),
] + [(dict(**{k: s}), INVALID) for s in BAD_STRIDES for k in ("qs", "qos", "ks", "kos")])
def test_rope_refuses_bad_arguments(L, kw, expect):
    assert _rope(L, **kw) == expect


def _append(L, c, **kw):
    a = dict(K=P, V=P, s=K4, Q=P, Qo=P, qs=Q4, qos=Q4, Hq=32, f=P, rot=128, pos=None, start=P, n=None, rows=None, B=4, T=8, ws=P, wsb=256)
    a.update(kw)
    return L.ea_cache_write_rope(None if c is None else ctypes.byref(c), a["K"], a["V"], a["s"], a["Q"], a["Qo"], a["qs"], a["qos"], a["Hq"],
                                 a["f"], a["rot"], 0, ctypes.c_float(1.0), a["pos"], a["start"], a["n"], a["rows"], a["B"], a["T"], a["ws"],
                                 a["wsb"], None)


@pytest.mark.parametrize("make,kw,expect", ALL_BAD)
def test_append_refuses_bad_caches(L, make, kw, expect):
    assert _append(L, make(**kw)) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(K=None), INVALID), (dict(V=None), INVALID), (dict(s=None), INVALID), (dict(Q=None), INVALID), (dict(Qo=None), INVALID),
    (dict(qs=None), INVALID), (dict(qos=None), INVALID), (dict(Hq=-1), INVALID), (dict(rows=P), INVALID), (dict(T=0), INVALID),
    (dict(B=0), INVALID), (dict(B=3), INVALID), (dict(f=None), INVALID), (dict(f=P + 8), INVALID), (dict(rot=24), INVALID),
    (dict(rot=160), INVALID), (dict(K=P + 4), INVALID), (dict(Q=P + 4), INVALID), (dict(ws=None), WORKSPACE), (dict(ws=P + 1), WORKSPACE),
    (dict(wsb=0), WORKSPACE),
] + [(dict(**{k: s}), INVALID) for s in BAD_STRIDES for k in ("s", "qs", "qos")])
def test_append_refuses_bad_arguments(L, kw, expect):
    assert _append(L, cache(), **kw) == expect


def test_append_refuses_no_cache_and_bf16_pages_of_odd_size(L):
    assert _append(L, None) == INVALID
    assert _append(L, paged(format=BF16, rows=80, k_scale=None, v_scale=None)) == UNSUPPORTED


def _plan(L, **kw):
    a = dict(p=P, n=None, B=4, T=16, d=P, m=P, ws=P, wsb=256)
    a.update(kw)
    return L.ea_tree_plan(a["p"], a["n"], a["B"], a["T"], a["d"], a["m"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(p=None), INVALID), (dict(d=None), INVALID), (dict(m=None), INVALID), (dict(m=P + 4), INVALID), (dict(B=0), INVALID),
    (dict(T=0), INVALID), (dict(T=129), UNSUPPORTED), (dict(ws=None), WORKSPACE), (dict(ws=P + 16), WORKSPACE), (dict(wsb=8), WORKSPACE),
])
def test_plan_refuses_bad_arguments(L, kw, expect):
    assert _plan(L, **kw) == expect


def _accept(L, **kw):
    a = dict(t=P, p=P, g=P, n=None, B=4, T=16, path=P, k=P, x=P, ws=P, wsb=256)
    a.update(kw)
    return L.ea_tree_accept(a["t"], a["p"], a["g"], a["n"], a["B"], a["T"], a["path"], a["k"], a["x"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(t=None), INVALID), (dict(p=None), INVALID), (dict(g=None), INVALID), (dict(path=None), INVALID), (dict(k=None), INVALID),
    (dict(x=None), INVALID), (dict(B=0), INVALID), (dict(T=0), INVALID), (dict(T=129), UNSUPPORTED), (dict(ws=None), WORKSPACE),
    (dict(ws=P + 16), WORKSPACE), (dict(wsb=8), WORKSPACE),
])
def test_accept_refuses_bad_arguments(L, kw, expect):
    assert _accept(L, **kw) == expect


def test_binding_refuses_host_tensors():
    x = torch.zeros(1, 4, 2, 128, dtype=torch.bfloat16)
    i = torch.zeros(1, 4, dtype=torch.int32)
    f = torch.ones(64)
    for call in (lambda: ea.ea_rope(x, x, i, f), lambda: ea.ea_rope(None, None, i, f), lambda: ea.ea_tree_plan(i),
                 lambda: ea.ea_tree_accept(i, i, i), lambda: ea.ea_cache_write_rope(None, x, x, f)):
        with pytest.raises(ValueError):
            call()


def _attn(L, c, **kw):
    a = dict(Q=P, K=P, V=P, O=P, LSE=None, qs=Q4, ks=K4, os=Q4, sl=P, n=None, d=P, mk=P, B=4, T=8, Hq=32, scale=0.1, m=P, sink=4, window=64,
             bm=None, bs=128, ws=P, wsb=1 << 40)
    a.update(kw)
    return L.ea_hybrid_attn_tree(a["Q"], a["K"], a["V"], None if c is None else ctypes.byref(c), a["O"], a["LSE"], a["qs"], a["ks"], a["os"],
                                 a["sl"], a["n"], a["d"], a["mk"], a["B"], a["T"], a["Hq"], ctypes.c_float(a["scale"]), a["m"], a["sink"],
                                 a["window"], a["bm"], a["bs"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("make,kw,expect", ALL_BAD)
def test_attention_refuses_bad_caches(L, make, kw, expect):
    assert _attn(L, make(**kw)) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(Q=None), INVALID), (dict(K=None), INVALID), (dict(V=None), INVALID), (dict(O=None), INVALID), (dict(sl=None), INVALID),
    (dict(d=None), INVALID), (dict(mk=None), INVALID), (dict(mk=P + 8), INVALID), (dict(m=None), INVALID), (dict(qs=None), INVALID),
    (dict(ks=None), INVALID), (dict(os=None), INVALID), (dict(B=0), INVALID), (dict(B=3), INVALID), (dict(T=0), INVALID),
    (dict(Hq=0), INVALID), (dict(Hq=31), INVALID), (dict(sink=-1), INVALID), (dict(window=0), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(bs=64), INVALID), (dict(Q=P + 8), INVALID),
    (dict(K=P + 2), INVALID), (dict(O=P + 4), INVALID), (dict(T=129), UNSUPPORTED), (dict(Hq=8 * 65), UNSUPPORTED),
    (dict(ws=None), WORKSPACE), (dict(ws=P + 128), WORKSPACE), (dict(wsb=1000), WORKSPACE),
] + [(dict(**{k: s}), INVALID) for s in BAD_STRIDES for k in ("qs", "ks", "os")])
def test_attention_refuses_bad_arguments(L, kw, expect):
    assert _attn(L, cache(), **kw) == expect


def test_attention_refuses_no_cache_and_pages_of_odd_size(L):
    assert _attn(L, None) == INVALID
    assert _attn(L, paged(format=BF16, rows=80, k_scale=None, v_scale=None)) == UNSUPPORTED
    assert _attn(L, paged(scale_block=32, rows=96, kv_str=_str(96 * 1024, 1024, 128, 1))) == UNSUPPORTED
    # more tiles than are counted in 32 bits; block masks whose rows are not numbered
    assert _attn(L, cache(outer=60000, rows=1 << 20), B=60000) == UNSUPPORTED
    assert _attn(L, cache(rows=128 * 65536), bm=P) == UNSUPPORTED


@pytest.mark.parametrize("sizes", [(0, 8, 32, 8, 128, 4096), (4, 0, 32, 8, 128, 4096), (4, 129, 32, 8, 128, 4096), (4, 8, 31, 8, 128, 4096),
                                   (4, 8, 0, 8, 128, 4096), (4, 8, 32, 0, 128, 4096), (4, 8, 520, 8, 128, 4096), (4, 8, 32, 8, 64, 4096),
                                   (4, 8, 32, 8, 128, 0), (60000, 8, 32, 8, 128, 1 << 30)])
def test_attention_workspace_of_bad_sizes(L, sizes):
    assert L.ea_tree_workspace_size(*sizes) == 0


def test_attention_workspace_sizes(L):
    # the partial results are bounded by the grid, not by the batch or the lengths
    small, large = (L.ea_tree_workspace_size(*s) for s in ((1, 8, 32, 8, 128, 4096), (64, 8, 32, 8, 128, 131072)))
    assert 256 < small < large < small + 4 * 64 * 8 * (1024 + 4)
    assert L.ea_tree_workspace_size(1, 33, 32, 8, 128, 4096) > 1.9 * small          # two M tiles


def test_attention_binding_refuses():
    x = torch.zeros(1, 4, 2, 128, dtype=torch.bfloat16)
    i = torch.zeros(1, 4, dtype=torch.int32)
    with pytest.raises(ValueError):
        ea.ea_hybrid_attn_tree(x, x, x, None, i[0], i, i, i, sink=1, window=1)
