"""Host-side checks of the KV cache operators (no GPU needed): workspace sizes and
the refusal of every bad argument before anything is enqueued; the binding's own
checks on CPU tensors."""
import ctypes

import pytest
import torch

import sparse_head_attention_gb300 as ea
from sparse_head_attention_gb300 import build as ea_build

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
E4M3, INT8, BF16 = 1, 2, 0


@pytest.fixture(scope="module")
def L():
    ea_build.build()
    return ea.lib()


def _str(*v):
    return (ctypes.c_int64 * len(v))(*v)


P = 0x100000        # an address that is never dereferenced: every call here is refused on the host


def cache(**kw):
    """4 sequences of 4096 rows and 8 heads, e4m3."""
    a = dict(K=P, V=P, k_scale=P, v_scale=P, kv_str=_str(4096 * 8 * 128, 8 * 128, 128, 1), block_table=None, bt_stride=0, outer=4,
             rows=4096, max_pages=0, Hkv=8, d=128, format=E4M3, scale_block=64)
    a.update(kw)
    return ea._Cache(a["K"], a["V"], a["k_scale"], a["v_scale"], a["kv_str"], a["block_table"], a["bt_stride"], a["outer"],
                     a["rows"], a["max_pages"], a["Hkv"], a["d"], a["format"], a["scale_block"])


def paged(**kw):
    a = dict(block_table=P, bt_stride=16, outer=100, rows=256, max_pages=16, kv_str=_str(256 * 8 * 128, 8 * 128, 128, 1))
    a.update(kw)
    return cache(**a)


BAD_CACHES = [
    (dict(K=None), INVALID), (dict(V=None), INVALID), (dict(k_scale=None), INVALID), (dict(v_scale=None), INVALID),
    (dict(format=3), INVALID), (dict(format=-1), INVALID), (dict(outer=0), INVALID), (dict(rows=0), INVALID), (dict(Hkv=0), INVALID),
    (dict(d=64), UNSUPPORTED), (dict(scale_block=8), UNSUPPORTED), (dict(scale_block=48), UNSUPPORTED), (dict(scale_block=0), UNSUPPORTED),
    (dict(K=P + 8), INVALID), (dict(V=P + 4), INVALID), (dict(kv_str=_str(4096 * 8 * 128, 8 * 128, 128, 2)), INVALID),
    (dict(kv_str=_str(4096 * 8 * 128, 8 * 128 + 8, 128, 1)), INVALID), (dict(kv_str=_str(0, 8 * 128, 128, 1)), INVALID),
    (dict(kv_str=_str(4096 * 8 * 128, -1024, 128, 1)), INVALID), (dict(outer=5), INVALID),          # B is 4
    (dict(rows=(1 << 31) - 128), UNSUPPORTED),
]
BAD_PAGES = [
    (dict(max_pages=0), INVALID), (dict(bt_stride=15), INVALID), (dict(rows=96), UNSUPPORTED),           # not a multiple of 64
    (dict(max_pages=1 << 23, bt_stride=1 << 23), UNSUPPORTED),
]
ALL_BAD = [(cache, kw, e) for kw, e in BAD_CACHES] + [(paged, kw, e) for kw, e in BAD_PAGES]


def _write(L, c, **kw):
    a = dict(K=P, V=P, s=_str(8 * 1024, 8 * 128, 128, 1), start=None, n=None, B=4, T=8, ws=P, wsb=256)
    a.update(kw)
    return L.ea_cache_write(None if c is None else ctypes.byref(c), a["K"], a["V"], a["s"], a["start"], a["n"], a["B"], a["T"], a["ws"],
                            a["wsb"], None)


@pytest.mark.parametrize("make,kw,expect", ALL_BAD)
def test_write_refuses_bad_caches(L, make, kw, expect):
    assert _write(L, make(**kw)) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(K=None), INVALID), (dict(V=None), INVALID), (dict(s=None), INVALID), (dict(T=0), INVALID), (dict(B=0), INVALID), (dict(B=3), INVALID),
    (dict(K=P + 2), INVALID), (dict(s=_str(8 * 1024, 8 * 128, 128, 2)), INVALID), (dict(s=_str(8 * 1024, 8 * 128 + 4, 128, 1)), INVALID),
    (dict(ws=None), WORKSPACE), (dict(ws=P + 128), WORKSPACE), (dict(wsb=255), WORKSPACE),
])
def test_write_refuses_bad_arguments(L, kw, expect):
    assert _write(L, cache(), **kw) == expect


def test_write_refuses_no_cache_and_bf16_pages_of_odd_size(L):
    assert _write(L, None) == INVALID
    assert _write(L, paged(format=BF16, rows=80, k_scale=None, v_scale=None)) == UNSUPPORTED
    assert _write(L, cache(format=BF16, kv_str=_str(4096 * 8 * 128, 8 * 128 + 4, 128, 1))) == INVALID


def _select(L, **kw):
    a = dict(w=P, sl=P, B=4, Hkv=8, Lmax=4096, keep=100, sink=10, recent=20, idx=P, new=P, ws=P, wsb=256)
    a.update(kw)
    return L.ea_evict_select(a["w"], a["sl"], a["B"], a["Hkv"], a["Lmax"], a["keep"], a["sink"], a["recent"], a["idx"], a["new"], a["ws"],
                             a["wsb"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(w=None), INVALID), (dict(sl=None), INVALID), (dict(idx=None), INVALID), (dict(new=None), INVALID), (dict(B=0), INVALID),
    (dict(Hkv=0), INVALID), (dict(Lmax=0), INVALID), (dict(keep=0), INVALID), (dict(sink=-1), INVALID), (dict(recent=-1), INVALID),
    (dict(sink=60, recent=41), INVALID), (dict(sink=(1 << 31) - 1, recent=(1 << 31) - 1), INVALID), (dict(Lmax=(1 << 21) + 1), UNSUPPORTED),
    (dict(B=65536), UNSUPPORTED), (dict(ws=None), WORKSPACE), (dict(wsb=0), WORKSPACE), (dict(ws=P + 1), WORKSPACE),
])
def test_select_refuses_bad_arguments(L, kw, expect):
    assert _select(L, **kw) == expect


def _compact(L, src, dst, **kw):
    a = dict(idx=P, n=P, B=4, keep=100, w=None, wo=None, ws=P, wsb=256)
    a.update(kw)
    return L.ea_cache_compact(ctypes.byref(src), ctypes.byref(dst), a["idx"], a["n"], a["B"], a["keep"], a["w"], a["wo"], a["ws"], a["wsb"],
                              None)


FAR = dict(K=1 << 40, V=1 << 41)        # a destination away from P


@pytest.mark.parametrize("make,kw,expect", ALL_BAD)
def test_compact_refuses_bad_caches(L, make, kw, expect):
    assert _compact(L, make(**kw), cache(**FAR)) == expect
    assert _compact(L, cache(**FAR), make(**kw)) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(idx=None), INVALID), (dict(n=None), INVALID), (dict(keep=0), INVALID), (dict(keep=4097), INVALID), (dict(B=3), INVALID),
    (dict(w=P), INVALID), (dict(wo=P), INVALID), (dict(w=P, wo=P), INVALID), (dict(ws=None), WORKSPACE), (dict(wsb=100), WORKSPACE),
])
def test_compact_refuses_bad_arguments(L, kw, expect):
    assert _compact(L, cache(), cache(**FAR), **kw) == expect


def test_compact_refuses_overlap_and_other_heads(L):
    assert _compact(L, cache(), cache()) == INVALID                                  # in place
    assert _compact(L, cache(), cache(K=P + 4096 * 1024, V=1 << 41)) == INVALID      # dst K begins inside src K
    assert _compact(L, cache(V=1 << 40), cache(K=(1 << 40) + 1024, V=1 << 42)) == INVALID
    assert _compact(L, paged(), cache(K=P + 1024, V=1 << 41)) == INVALID             # a pool against a contiguous cache
    assert _compact(L, cache(), cache(Hkv=4, **FAR)) == INVALID


def _decode(L, c, **kw):
    a = dict(q=P, O=P, LSE=None, qs=_str(32 * 128, 128, 1), os_=_str(32 * 128, 128, 1), sl=P, B=4, Hq=32, scale=0.088, m=P, sink=16,
             window=64, bm=None, bs=128, ns=0, kw=None, acc=1, ws=P, wsb=1 << 34)
    a.update(kw)
    return L.ea_hybrid_attn_decode_q8(a["q"], None if c is None else ctypes.byref(c), a["O"], a["LSE"], a["qs"], a["os_"], a["sl"], a["B"],
                                      a["Hq"], a["scale"], a["m"], a["sink"], a["window"], a["bm"], a["bs"], a["ns"], a["kw"], a["acc"],
                                      a["ws"], a["wsb"], None)


@pytest.mark.parametrize("make,kw,expect", ALL_BAD)
def test_decode_refuses_bad_caches(L, make, kw, expect):
    assert _decode(L, make(**kw)) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), INVALID), (dict(O=None), INVALID), (dict(sl=None), INVALID), (dict(m=None), INVALID), (dict(qs=None), INVALID),
    (dict(Hq=0), INVALID), (dict(Hq=36), INVALID), (dict(Hq=72), UNSUPPORTED), (dict(B=3), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(sink=-1), INVALID), (dict(window=0), INVALID), (dict(ns=-1), INVALID), (dict(ns=1025), INVALID),
    (dict(bs=64), INVALID), (dict(qs=_str(32 * 128, 128, 2)), INVALID), (dict(qs=_str(32 * 128 + 4, 128, 1)), INVALID),
    (dict(os_=_str(0, 128, 1)), INVALID), (dict(q=P + 8), INVALID), (dict(O=P + 2), INVALID), (dict(ws=None), WORKSPACE),
    (dict(ws=P + 64), WORKSPACE), (dict(wsb=1024), WORKSPACE),
])
def test_decode_refuses_bad_arguments(L, kw, expect):
    assert _decode(L, cache(), **kw) == expect


def test_decode_refuses_bf16_caches_and_short_pages(L):
    assert _decode(L, None) == INVALID
    assert _decode(L, cache(format=BF16)) == UNSUPPORTED
    assert _decode(L, paged(rows=32, scale_block=32)) == UNSUPPORTED
    assert _decode(L, cache(rows=65536 * 128, kv_str=_str(65536 * 128 * 1024, 1024, 128, 1)), bm=P) == UNSUPPORTED


def test_decode_workspace(L):
    size = lambda *a: L.ea_decode_q8_workspace_size(*a)  # noqa: E731
    assert size(32, 32, 8, 128, 131072, 0, 0) > 256
    assert size(32, 32, 8, 128, 131072, 0, 1) >= size(32, 32, 8, 128, 131072, 0, 0) + 4 * 32 * 32 * 131072
    for bad in [(0, 32, 8, 128, 4096, 0, 0), (1, 32, 8, 64, 4096, 0, 0), (1, 30, 8, 128, 4096, 0, 0), (1, 72, 8, 128, 4096, 0, 0),
                (1, 32, 8, 128, 0, 0, 0), (1, 32, 8, 128, 4096, 1025, 0), (1, 32, 8, 128, 4096, -1, 0)]:
        assert size(*bad) == 0, bad
    need = size(4, 32, 8, 128, 4096, 0, 1)
    assert _decode(L, cache(), kw=P, wsb=need - 1) == WORKSPACE
    assert _decode(L, cache(), wsb=size(4, 32, 8, 128, 4096, 0, 0) - 1) == WORKSPACE


def _weights(L, **kw):
    a = dict(Q=P, K=P, LSE=P, qs=_str(64 * 32 * 128, 32 * 128, 128, 1), ks=_str(4096 * 8 * 128, 8 * 128, 128, 1), ls=_str(32 * 64, 64),
             sl=None, B=2, Tq=64, Lmax=4096, Hq=32, Hkv=8, d=128, scale=0.088, m=P, sink=16, window=64, bm=None, bs=128, w=P, acc=0, ws=P,
             wsb=1 << 34)
    a.update(kw)
    return L.ea_key_weights(a["Q"], a["K"], a["LSE"], a["qs"], a["ks"], a["ls"], a["sl"], a["B"], a["Tq"], a["Lmax"], a["Hq"], a["Hkv"], a["d"],
                            a["scale"], a["m"], a["sink"], a["window"], a["bm"], a["bs"], a["w"], a["acc"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(Q=None), INVALID), (dict(K=None), INVALID), (dict(LSE=None), INVALID), (dict(m=None), INVALID), (dict(w=None), INVALID),
    (dict(qs=None), INVALID), (dict(ls=None), INVALID), (dict(B=0), INVALID), (dict(Tq=0), INVALID), (dict(Lmax=0), INVALID),
    (dict(Hq=30), INVALID), (dict(scale=0.0), INVALID), (dict(sink=-1), INVALID), (dict(window=0), INVALID), (dict(bs=64), INVALID),
    (dict(d=64), UNSUPPORTED), (dict(Lmax=(1 << 21) + 1), UNSUPPORTED), (dict(Hq=8 * 65), UNSUPPORTED), (dict(B=8192), UNSUPPORTED),
    (dict(qs=_str(64 * 32 * 128, 32 * 128, 128, 2)), INVALID), (dict(ks=_str(4096 * 8 * 128, 8 * 128, 127, 1)), INVALID),
    (dict(ls=_str(-1, 64)), INVALID), (dict(Q=P + 2), INVALID), (dict(ws=None), WORKSPACE), (dict(ws=P + 16), WORKSPACE), (dict(wsb=128), WORKSPACE),
])
def test_key_weights_refuses_bad_arguments(L, kw, expect):
    assert _weights(L, **kw) == expect


def test_key_weights_workspace(L):
    size = lambda *a: L.ea_key_weights_workspace_size(*a)  # noqa: E731
    assert size(1, 1, 32768, 32, 8, 128) == 256                            # one query row: no shares to join
    one = size(1, 4096, 4096, 8, 1, 128)                                   # few key tiles: their queries are cut
    assert one > 256 and _weights(L, B=1, Tq=4096, Hq=8, Hkv=1, wsb=one - 1) == WORKSPACE
    for bad in [(0, 1, 10, 8, 8, 128), (1, 0, 10, 8, 8, 128), (1, 1, 0, 8, 8, 128), (1, 1, 10, 9, 8, 128), (1, 1, 10, 8, 8, 64),
                (1, 1, (1 << 21) + 1, 8, 8, 128)]:
        assert size(*bad) == 0, bad


def test_binding_refuses_cpu_tensors_and_wrong_types():
    K = torch.zeros(2, 64, 4, 128, dtype=torch.int8)
    s = torch.ones(2, 4, 1)
    with pytest.raises(ValueError, match="CUDA"):
        ea.KVCache(K, K.clone(), s, s.clone())
    x = torch.zeros(2, 8, 4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ea.ea_key_weights(x, x, torch.zeros(2, 4, 8), torch.zeros(2, 4, dtype=torch.uint8), sink=0, window=1)
    with pytest.raises(ValueError, match="CUDA"):
        ea.ea_evict_select(torch.zeros(1, 1, 8), torch.zeros(1, dtype=torch.int32), keep=4)


def test_compact_refuses_weights_that_overlap(L):
    # [4][8][4096] floats each (the caches' own sizes): 4 MB a byte short of apart, and one in the other's middle
    n = 4 * 8 * 4096 * 4
    W = 1 << 43
    assert _compact(L, cache(), cache(**FAR), w=W, wo=W + n - 4) == INVALID
    assert _compact(L, cache(), cache(**FAR), w=W, wo=W - n + 4) == INVALID
    assert _compact(L, cache(), cache(**FAR), w=W, wo=W + n // 2) == INVALID


def test_decode_refuses_splits_that_are_too_long(L):
    long = dict(rows=1 << 20, max_pages=64, bt_stride=64, scale_block=64)
    assert _decode(L, paged(**long), ns=3) == UNSUPPORTED
    assert _decode(L, paged(**long), ns=4, wsb=1024) == WORKSPACE       # 2^24 rows each: as far as the workspace


def _pages_on_the_cpu(monkeypatch, table):
    # the handle alone, over CPU tensors: nothing is launched
    monkeypatch.setattr(ea, "_dev", lambda t, name, dtype=None: t)
    K = torch.zeros(8, 64, 2, 128, dtype=torch.int8)
    s = torch.ones(8, 2, 1)
    return ea.KVCache(K, K.clone(), s, s.clone(), block_table=table)


@pytest.mark.parametrize("B,pages", [(2, 4), (3, 1), (5, 2)])
def test_binding_refuses_block_tables_whose_rows_overlap(monkeypatch, B, pages):
    # one prompt's row for all sequences (row stride 0), and rows that begin inside the one before them: sequence b's
    # row is not b * max_pages entries on, and reading there leaves the tensor
    row = torch.arange(pages, dtype=torch.int32)
    with pytest.raises(ValueError, match="block_table"):
        _pages_on_the_cpu(monkeypatch, row[None].expand(B, -1))
    if pages > 1:
        with pytest.raises(ValueError, match="block_table"):
            _pages_on_the_cpu(monkeypatch, torch.arange(B + pages, dtype=torch.int32).as_strided((B, pages), (1, 1)))


def test_binding_passes_the_block_tables_row_stride(monkeypatch):
    wide = torch.zeros(6, 9, dtype=torch.int32)
    for table, stride in ((wide, 9), (wide[:, :4], 9), (wide[::2, 3:], 18), (wide[:, :1], 9), (wide.new_zeros(6, 1), 1),
                          (wide.new_zeros(4)[None], 4), (wide.new_zeros(4).expand(1, -1), 4),
                          (wide.as_strided((1, 4), (0, 1)), 4), (wide.new_zeros(1, 1).expand(1, 1), 1)):
        c = _pages_on_the_cpu(monkeypatch, table)
        assert c._c.bt_stride == stride and c._c.max_pages == table.shape[1]
        assert all(c._c.bt_stride * b == table[b].storage_offset() - table.storage_offset() for b in range(c.B))


@pytest.mark.parametrize("rows", [16, 80, 96])
def test_bf16_pages_of_odd_size_are_read_but_not_written(L, rows):
    odd = dict(format=BF16, rows=rows, k_scale=None, v_scale=None, max_pages=100, bt_stride=100,
               kv_str=_str(rows * 8 * 128, 8 * 128, 128, 1))
    assert _write(L, paged(**odd)) == UNSUPPORTED
    assert _compact(L, cache(), paged(**odd, **FAR)) == UNSUPPORTED
    assert _compact(L, paged(**odd), cache(**FAR), ws=None) == WORKSPACE      # accepted as a source, as far as the workspace
