"""The KV cache operators against plain implementations in 64 bits: writing an
8-bit cache, choosing the tokens that stay, and gathering them into another
cache.  Codes, scales and indices are whole results: they have to be equal."""
import numpy as np
import pytest
import torch

import sparse_head_attention_gb300 as ea
from cache_reference import compact_ref, make_cache, select_ref, tokens, values, write_ref
from gpu_helpers import check_no_device_error, gpu_device

pytestmark = pytest.mark.gpu
E4M3, INT8, BF16 = torch.float8_e4m3fn, torch.int8, torch.bfloat16


@pytest.fixture(scope="module")
def dev():
    return gpu_device()


def handle(c, dev):
    """A KVCache on the device with the reference cache's contents."""
    t = {k: None if v is None else v.to(dev) for k, v in c.items() if k in ("K", "V", "ks", "vs", "table")}
    return ea.KVCache(t["K"], t["V"], t["ks"], t["vs"], scale_block=c["sb"], block_table=t["table"])


def same_cache(h, c):
    for got, want in ((h.K, c["K"]), (h.V, c["V"])):
        size = torch.int16 if want.dtype == BF16 else torch.uint8
        assert torch.equal(got.cpu().view(size), want.view(size))
    for got, want in ((h.k_scale, c["ks"]), (h.v_scale, c["vs"])):
        if want is not None:
            np.testing.assert_array_equal(got.cpu().numpy(), want.numpy())


@pytest.mark.parametrize("dtype", [E4M3, INT8, BF16])
@pytest.mark.parametrize("sb,page", [(16, 0), (32, 64), (64, 0), (64, 64), (128, 128), (128, 0)])
def test_write_appends_at_any_row(dev, dtype, sb, page):
    B, Hkv, cap, T = 7, 3, 384, 150
    c = make_cache(B, cap, Hkv, dtype, sb, page, seed=sb + page)
    h = handle(c, dev)
    # block starts, block ends, a single token, nothing, the last row, everything
    start = [0, 64, 127, 383, 129, 200, 234]
    n = [150, 64, 2, 1, 0, 129, 150]
    K, V = tokens((B, T, Hkv, 128), seed=1), tokens((B, T, Hkv, 128), seed=2)
    V = V * 64.0                                # scales grow: earlier rows are rounded again
    ws = ea.cache_workspace(dev)
    ea.ea_cache_write(h, K.to(dev), V.to(dev), torch.tensor(start, dtype=torch.int32, device=dev),
                      torch.tensor(n, dtype=torch.int32, device=dev), workspace=ws)
    check_no_device_error(ws)
    write_ref(c, K, V, start, n)
    same_cache(h, c)


@pytest.mark.parametrize("dtype", [E4M3, INT8])
def test_write_token_by_token_then_whole(dev, dtype):
    # tokens appended one at a time with growing magnitude, then a second pass over the same rows in one call
    B, Hkv, T = 2, 2, 70
    c = make_cache(B, 128, Hkv, dtype, 32, 0, seed=3)
    h = handle(c, dev)
    K, V = tokens((B, T, Hkv, 128), seed=4), tokens((B, T, Hkv, 128), seed=5)
    K = (K.float() * torch.exp2(torch.arange(T) % 7).view(1, T, 1, 1)).to(BF16)
    Kd, Vd = K.to(dev), V.to(dev)
    for t in range(T):
        at = torch.full((B,), t, dtype=torch.int32, device=dev)
        ea.ea_cache_write(h, Kd[:, t:t + 1], Vd[:, t:t + 1], at)
        write_ref(c, K[:, t:t + 1], V[:, t:t + 1], [t] * B, [1] * B)
    same_cache(h, c)
    ea.ea_cache_write(h, Kd, Vd)
    write_ref(c, K, V, [0] * B, [T] * B)
    same_cache(h, c)


@pytest.mark.parametrize("dtype", [E4M3, INT8])
def test_write_scale_borders(dev, dtype):
    # a block's largest value at, just above and just below each power of two times qmax, zeros, subnormals, the largest bf16
    qmax = 448.0 if dtype == E4M3 else 127.0
    vals = []
    for e in (-70, -65, -64, -63, -8, 0, 3, 118):
        for m in (1.0, 1.75, 1.7578125, 1.984375, 1.9921875):
            vals.append(m * 2.0 ** e)
    vals += [0.0, qmax, 2.0 ** -133, float(torch.finfo(BF16).max)]
    n = len(vals)
    x = torch.zeros(1, 16 * n, 1, 128)
    x[0, ::16, 0, 5] = torch.tensor(vals, dtype=torch.float64).float()
    x[0, 1::16, 0, 6] = -0.37 * x[0, ::16, 0, 5]
    x[0, 2::16, 0, 7] = 0.011 * x[0, ::16, 0, 5]
    x = x.to(BF16)
    c = make_cache(1, 16 * n, 1, dtype, 16, 0, seed=6)
    h = handle(c, dev)
    ea.ea_cache_write(h, x.to(dev), (-x).to(dev))
    write_ref(c, x, -x, [0], [16 * n])
    same_cache(h, c)
    # |value - code * scale| <= half a step of the code, or of the smallest scale's grid
    got = values(h.K.cpu(), h.k_scale.cpu(), 16)
    want = x.double()
    half = (torch.finfo(E4M3).eps / 2 * want.abs()).clamp(min=2.0 ** -10 * 2.0 ** -64) if dtype == E4M3 else None
    s = h.k_scale.cpu().double().repeat_interleave(16, -1).transpose(1, 2)[..., None]
    half = torch.maximum(half, 2.0 ** -10 * s) if dtype == E4M3 else 0.5 * s
    assert (got - want).abs().le(half).all()


@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_write_non_finite_poisons_its_block_only(dev, dtype, bad):
    c = make_cache(1, 256, 2, dtype, 64, 0, seed=7)
    h = handle(c, dev)
    K, V = tokens((1, 100, 2, 128), seed=8), tokens((1, 100, 2, 128), seed=9)
    K[0, 20, 1, 77] = bad                       # row 50: block 0 of head 1
    ea.ea_cache_write(h, K.to(dev), V.to(dev), torch.tensor([30], dtype=torch.int32, device=dev))
    write_ref(c, K, V, [30], [100])
    same_cache(h, c)
    nan = np.isnan(h.k_scale.cpu().numpy())
    assert nan[0, 1, 0] and nan.sum() == 1
    # it stays NaN while rows are appended behind, and ends when the block is written from its first row
    one = tokens((1, 1, 2, 128), seed=10)
    ea.ea_cache_write(h, one.to(dev), one.to(dev), torch.tensor([40], dtype=torch.int32, device=dev))
    assert np.isnan(h.k_scale.cpu().numpy()[0, 1, 0])
    ea.ea_cache_write(h, V.to(dev), V.to(dev))
    assert np.isfinite(h.k_scale.cpu().numpy()[0, 1, 0])


def test_write_strided_inputs_and_cache_views(dev):
    # K and V as slices of one projection [B, T, Hq + 2 Hkv, 128]; the cache a view of a wider one
    B, T, Hkv = 2, 90, 2
    x = tokens((B, T, 8, 128), seed=11)
    K, V = x[:, :, 3:5], x[:, :, 6:8]
    c = make_cache(B, 192, Hkv, E4M3, 64, 0, seed=12)
    wide = {k: torch.zeros(B, 192, 5, 128, dtype=E4M3, device=dev) for k in "KV"}
    wk, wv = (wide[k][:, :, 1:3] for k in "KV")
    wk.copy_(c["K"]), wv.copy_(c["V"])
    h = ea.KVCache(wk, wv, c["ks"].to(dev), c["vs"].to(dev), scale_block=64)
    xd = x.to(dev)
    ea.ea_cache_write(h, xd[:, :, 3:5], xd[:, :, 6:8], torch.tensor([5, 70], dtype=torch.int32, device=dev))
    write_ref(c, K, V, [5, 70], [T, T])
    same_cache(h, c)
    for k in "KV":
        assert not wide[k][:, :, 0].view(torch.uint8).any() and not wide[k][:, :, 3:].view(torch.uint8).any()


def test_write_reports_bad_rows_and_pages(dev):
    c = make_cache(4, 256, 2, INT8, 64, 64, seed=13)
    c["table"][2, 1] = 999                      # rows 64 .. 127 of sequence 2 have no page
    c["table"][3, 0] = -1
    h = handle(c, dev)
    K, V = tokens((4, 100, 2, 128), seed=14), tokens((4, 100, 2, 128), seed=15)
    ws = ea.cache_workspace(dev)
    start = torch.tensor([200, -1, 10, 64], dtype=torch.int32, device=dev)
    ea.ea_cache_write(h, K.to(dev), V.to(dev), start, workspace=ws)
    assert ea.ea_check_errors(ws) == 6 and ea.ea_check_errors(ws) == 0
    # sequence 0 does not fit, 1 starts below 0, 2 loses the block without a page, 3 is written
    write_ref(c, K, V, [None, None, 10, 64], [0, 0, 100, 100])
    same_cache(h, c)
    ea.ea_cache_write(h, K.to(dev), V.to(dev), n_new=torch.tensor([1, 101, 0, -5], dtype=torch.int32, device=dev),
                      workspace=ws)
    assert ea.ea_check_errors(ws) == 6
    write_ref(c, K, V, [0, None, None, None], [1, 0, 0, 0])
    same_cache(h, c)


# ---------------------------------------------------------------- selection
@pytest.mark.parametrize("L,keep,sink,recent", [
    (1, 1, 0, 0), (5, 5, 1, 1), (5, 4, 0, 0), (1000, 100, 10, 20), (1000, 30, 10, 20), (1000, 999, 0, 0),
    (1025, 1, 0, 0), (4097, 2048, 1, 0), (20000, 511, 0, 511), (20000, 511, 511, 0), (20000, 10000, 3, 5),
    (70001, 4096, 128, 1000)])
def test_select_keeps_the_heaviest(dev, L, keep, sink, recent):
    g = torch.Generator().manual_seed(L + keep)
    Lmax, lens = L + 3, [L, L // 2, 0]
    w = torch.rand(3, 2, Lmax, generator=g) ** 9
    w[:, 1] = (w[:, 1] * 8).round() / 8           # many ties, most of them at zero
    w[0, 0, ::7] = w[0, 0, 0]
    ws = ea.cache_workspace(dev)
    idx, new = ea.ea_evict_select(w.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev), keep=keep, sink=sink,
                                  recent=recent, workspace=ws)
    check_no_device_error(ws)
    want, n = select_ref(w.numpy(), lens, keep, sink, recent)
    np.testing.assert_array_equal(idx.cpu().numpy(), want)
    np.testing.assert_array_equal(new.cpu().numpy(), n)


def test_select_unusual_weights(dev):
    # signs, infinities, both zeros, NaN (below everything), subnormals, all equal
    L, keep = 5000, 1234
    g = torch.Generator().manual_seed(1)
    w = torch.randn(1, 6, L, generator=g)
    w[0, 1] = torch.where(torch.rand(L, generator=g) < 0.5, 0.0, -0.0)
    w[0, 2, ::3] = float("nan")
    w[0, 2, 1::3] = -float("inf")
    w[0, 3] = float("nan")
    w[0, 4] *= 1e-40
    w[0, 5, 100:2000] = float("inf")
    lens = [L]
    idx, _ = ea.ea_evict_select(w.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev), keep=keep, sink=2, recent=7)
    want, _ = select_ref(w.numpy(), lens, keep, 2, 7)
    np.testing.assert_array_equal(idx.cpu().numpy(), want)


def test_select_long_sequences_and_bad_lengths(dev):
    L = 1 << 20
    w = torch.rand(1, 2, L, generator=torch.Generator().manual_seed(2))
    idx, _ = ea.ea_evict_select(w.to(dev), torch.tensor([L], dtype=torch.int32, device=dev), keep=100000, sink=4, recent=9)
    want, _ = select_ref(w.numpy(), [L], 100000, 4, 9)
    np.testing.assert_array_equal(idx.cpu().numpy(), want)
    ws = ea.cache_workspace(dev)
    w = torch.rand(3, 1, 100, device=dev)
    idx, new = ea.ea_evict_select(w, torch.tensor([101, -1, 100], dtype=torch.int32, device=dev), keep=10, workspace=ws)
    assert ea.ea_check_errors(ws) == 6
    assert new.tolist() == [0, 0, 10] and (idx[:2] == -1).all() and (idx[2] >= 0).all()


# ---------------------------------------------------------------- compaction
@pytest.mark.parametrize("src", [BF16, E4M3, INT8])
@pytest.mark.parametrize("dst", [BF16, E4M3, INT8])
@pytest.mark.parametrize("paged", [(0, 0), (64, 0), (128, 256)])
def test_compact_gathers_and_requantises(dev, src, dst, paged):
    B, Hkv, keep = 4, 3, 200
    sb_src, sb_dst = 32, 64
    s = make_cache(B, 512, Hkv, src, sb_src, paged[0], seed=20)
    d = make_cache(B, 256, Hkv, dst, sb_dst, paged[1], seed=21)
    g = torch.Generator().manual_seed(22)
    index = torch.stack([torch.randperm(512, generator=g)[:keep].sort().values for _ in range(B * Hkv)])
    index = index.view(B, Hkv, keep).to(torch.int32)
    index[1, 1] = index[1, 1].flip(0)             # any order, and a row taken twice
    index[1, 2, 5] = index[1, 2, 4]
    counts = [200, 129, 0, 1]
    index[1, :, 129:] = -1
    w, w_out = torch.rand(B, Hkv, 512, generator=g), torch.full((B, Hkv, 256), 7.0)
    hs, hd, wo = handle(s, dev), handle(d, dev), w_out.to(dev)
    ws = ea.cache_workspace(dev)
    ea.ea_cache_compact(hs, hd, index.to(dev), torch.tensor(counts, dtype=torch.int32, device=dev), weights=w.to(dev),
                        weights_out=wo, workspace=ws)
    check_no_device_error(ws)
    compact_ref(s, d, index, counts, w, w_out)
    same_cache(hd, d)
    np.testing.assert_array_equal(wo.cpu().numpy(), w_out.numpy())


@pytest.mark.parametrize("sb", [16, 32, 128])
def test_compact_scale_blocks(dev, sb):
    s, d = make_cache(2, 300, 2, E4M3, sb, 0, seed=30), make_cache(2, 300, 2, INT8, sb, 0, seed=31)
    index = torch.arange(299, -1, -1, dtype=torch.int32).expand(2, 2, 300).contiguous()
    hs, hd = handle(s, dev), handle(d, dev)
    ea.ea_cache_compact(hs, hd, index.to(dev), torch.tensor([300, 17], dtype=torch.int32, device=dev))
    compact_ref(s, d, index, [300, 17], None, None)
    same_cache(hd, d)


@pytest.mark.parametrize("src", [E4M3, INT8])
@pytest.mark.parametrize("dst", [E4M3, INT8, BF16])
@pytest.mark.parametrize("outlier", [600.0, 2000.0, 1e4, 3e4, 2e5])
@pytest.mark.parametrize("sb_dst", [16, 64])
def test_compact_of_rows_far_below_their_blocks_largest(dev, src, dst, outlier, sb_dst):
    # every block of the source holds one row `outlier` times larger than the others, which from 3e4 on are all below
    # e4m3's normal codes and at 2e5 its least one: gathered without that row, their block's scale is up to 2^17 smaller
    B, Hkv, sb, L = 3, 3, 32, 256
    s, d = make_cache(B, L, Hkv, src, sb, 64, seed=23), make_cache(B, L, Hkv, dst, sb_dst, 0, seed=24)
    g = torch.Generator().manual_seed(25)
    K, V = (torch.randn(B, L, Hkv, 128, generator=g) for _ in range(2))
    for x in (K, V):
        x[:, sb - 1 :: sb] *= outlier
    write_ref(s, K.to(BF16), V.to(BF16), [0] * B, [L] * B)
    small = torch.arange(L)[torch.arange(L) % sb != sb - 1]
    index = torch.full((B, Hkv, 193), -1, dtype=torch.int32)
    index[:] = small[:193]                        # the small rows alone
    index[1] = small[torch.randperm(len(small), generator=g)[:193]]
    index[:, 1, 70] = 2 * sb - 1                  # head 1: one block with a large row among them
    # counts: the last block of a single small row, whole blocks, one row in all
    counts = [193, 128, 1]
    hs, hd = handle(s, dev), handle(d, dev)
    ws = ea.cache_workspace(dev)
    ea.ea_cache_compact(hs, hd, index.to(dev), torch.tensor(counts, dtype=torch.int32, device=dev), workspace=ws)
    check_no_device_error(ws)
    compact_ref(s, d, index, counts, None, None)
    same_cache(hd, d)


@pytest.mark.parametrize("src", [E4M3, INT8])
@pytest.mark.parametrize("dst", [E4M3, INT8, BF16])
def test_compact_of_values_that_rounded_up_to_two_to_the_128(dev, src, dst):
    # the largest bf16 is 255 / 256 of 2^128 and its code stands for 2^128, beyond fp32, with a finite scale: the block of
    # the destination gets one too (bf16 has no such number and rounds it to infinity)
    top = float(torch.finfo(BF16).max)
    s, d = make_cache(1, 64, 2, src, 32, 0, seed=26), make_cache(1, 64, 2, dst, 16, 0, seed=27)
    K, V = tokens((1, 64, 2, 128), seed=28), tokens((1, 64, 2, 128), seed=29)
    K[0, 3, 0, 5], V[0, 40, 1, 6] = top, -top
    write_ref(s, K, V, [0], [64])
    code = s["K"][0, 3, 0, 5].double() * s["ks"][0, 0, 0].double()
    assert code == 2.0 ** 128 and torch.isfinite(s["ks"]).all()
    index = torch.randperm(64, generator=torch.Generator().manual_seed(30)).to(torch.int32).expand(1, 2, 64).contiguous()
    hs, hd = handle(s, dev), handle(d, dev)
    ea.ea_cache_compact(hs, hd, index.to(dev), torch.tensor([64], dtype=torch.int32, device=dev))
    compact_ref(s, d, index, [64], None, None)
    same_cache(hd, d)


def test_compact_of_everything_keeps_the_values(dev):
    # an e4m3 block whose largest value was rounded down to 224 * s gets half the scale: other codes, the same values
    for dtype in (E4M3, INT8):
        s, d = make_cache(2, 256, 2, dtype, 64, 0, seed=40), make_cache(2, 256, 2, dtype, 64, 0, seed=41)
        hs, hd = handle(s, dev), handle(d, dev)
        index = torch.arange(256, dtype=torch.int32).expand(2, 2, 256).contiguous()
        ea.ea_cache_compact(hs, hd, index.to(dev), torch.tensor([256, 256], dtype=torch.int32, device=dev))
        for got, sc, was, was_s in ((hd.K, hd.k_scale, s["K"], s["ks"]), (hd.V, hd.v_scale, s["V"], s["vs"])):
            assert torch.equal(values(got.cpu(), sc.cpu(), 64), values(was, was_s, 64))


def test_compact_reports_bad_indices_counts_and_pages(dev):
    s, d = make_cache(3, 256, 1, BF16, 64, 64, seed=50), make_cache(3, 128, 1, E4M3, 64, 64, seed=51)
    s["table"][0, 3] = 5000
    d["table"][2, 0] = -7
    index = torch.arange(128, dtype=torch.int32).expand(3, 1, 128).contiguous()
    index[0, 0, 3], index[0, 0, 4], index[0, 0, 5] = -1, 256, 255
    hs, hd = handle(s, dev), handle(d, dev)
    ws = ea.cache_workspace(dev)
    ea.ea_cache_compact(hs, hd, index.to(dev), torch.tensor([128, 129, 128], dtype=torch.int32, device=dev), workspace=ws)
    assert ea.ea_check_errors(ws) == 6
    compact_ref(s, d, index, [128, 0, 128], None, None)
    same_cache(hd, d)


def test_compact_within_one_pool(dev):
    # src and dst are sequences of the same pages, read and written through different tables
    pool = make_cache(1, 1024, 2, INT8, 64, 128, seed=60, spare=4)
    used = set(pool["table"].view(-1).tolist())
    free = [p for p in range(pool["K"].shape[0]) if p not in used][:2]
    d = dict(pool, table=torch.tensor([free], dtype=torch.int32))
    index = torch.arange(0, 1024, 5, dtype=torch.int32).expand(1, 2, 205).contiguous()
    hs = handle(pool, dev)
    hd = ea.KVCache(hs.K, hs.V, hs.k_scale, hs.v_scale, scale_block=64, block_table=d["table"].to(dev))
    ea.ea_cache_compact(hs, hd, index.to(dev), torch.tensor([205], dtype=torch.int32, device=dev))
    compact_ref(pool, d, index, [205], None, None)
    same_cache(hs, pool)


def test_cache_ops_in_a_captured_graph(dev):
    # select, compact and an append captured once, replayed on new contents: equal to eager calls
    B, Hkv, L = 2, 2, 3000
    w = torch.rand(B, Hkv, L, device=dev)
    lens = torch.tensor([3000, 1700], dtype=torch.int32, device=dev)
    s, d = handle(make_cache(B, L, Hkv, E4M3, 64, 0, seed=70), dev), handle(make_cache(B, 512, Hkv, E4M3, 64, 0, seed=71), dev)
    e = handle(make_cache(B, 512, Hkv, E4M3, 64, 0, seed=71), dev)
    one = tokens((B, 1, Hkv, 128), seed=72).to(dev)
    ws = ea.cache_workspace(dev)
    idx, new = torch.empty(B, Hkv, 500, dtype=torch.int32, device=dev), torch.empty(B, dtype=torch.int32, device=dev)

    def step(dst):
        ea.ea_evict_select(w, lens, keep=500, sink=4, recent=100, index=idx, new_seqlens=new, workspace=ws)
        ea.ea_cache_compact(s, dst, idx, new, workspace=ws)
        ea.ea_cache_write(dst, one, one, new, workspace=ws)

    step(d)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(d)
    w.copy_(torch.rand(B, Hkv, L, device=dev))
    lens.copy_(torch.tensor([400, 2999]))
    g.replay()
    torch.cuda.synchronize()
    for a, b in ((e.K, d.K), (e.V, d.V)):         # rows behind the kept ones stay: start from d's
        a.view(torch.uint8).copy_(b.view(torch.uint8))
    e.k_scale.copy_(d.k_scale), e.v_scale.copy_(d.v_scale)
    step(e)
    check_no_device_error(ws)
    for a, b in ((e.K, d.K), (e.V, d.V)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert torch.equal(e.k_scale, d.k_scale) and torch.equal(e.v_scale, d.v_scale)


def test_cache_ops_on_another_stream(dev):
    c = make_cache(2, 256, 2, E4M3, 64, 0, seed=80)
    h = handle(c, dev)
    K, V = tokens((2, 100, 2, 128), seed=81), tokens((2, 100, 2, 128), seed=82)
    Kd, Vd = K.to(dev), V.to(dev)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    ea.ea_cache_write(h, Kd, Vd, stream=side)
    side.synchronize()
    write_ref(c, K, V, [0, 0], [100, 100])
    same_cache(h, c)
