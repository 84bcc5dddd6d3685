"""The decode over an 8-bit cache against a plain implementation in 64 bits:
formats, scale blocks, pages, head groups, modes, lengths from none on, what lies
behind a sequence, and the keys' attention weights.  The tolerances are derived
in cache_reference.decode_ref."""
import numpy as np
import pytest
import torch

import sparse_head_attention_gb300 as ea
from cache_reference import decode_ref, logical, make_cache, rows_of, tokens, value_scales
from gpu_helpers import check_no_device_error, gpu_device
from sparse_head_attention_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
E4M3, INT8, BF16 = torch.float8_e4m3fn, torch.int8, torch.bfloat16
FULL, SSA, BLOCK = ea.FULL, ea.SSA, ea.BLOCK
SCALE = 128 ** -0.5


@pytest.fixture(scope="module")
def dev():
    return gpu_device()


def handle(c, dev):
    t = {k: None if v is None else v.to(dev) for k, v in c.items() if k in ("K", "V", "ks", "vs", "table")}
    return ea.KVCache(t["K"], t["V"], t["ks"], t["vs"], scale_block=c["sb"], block_table=t["table"])


def spoil(c, lens):
    """NaN codes and scales behind every sequence's end (blocks that hold none of its tokens get NaN scales)."""
    page = c["K"].shape[1]
    cap = page if c["table"] is None else page * c["table"].shape[1]
    bad = 0x7f if c["K"].dtype == E4M3 else 0x80
    for b, L in enumerate(lens):
        for p in range(L, cap):
            o, r = rows_of(c, b, p)
            for kv in "KV":
                c[kv].view(torch.uint8)[o, r] = bad
            if p % c["sb"] == 0:
                for sc in ("ks", "vs"):
                    c[sc][o, :, r // c["sb"]] = float("nan")


def check(dev, c, q, lens, modes, sink, window, bm=None, num_splits=0, scale=None, spoiled=True):
    K, V = logical(c)
    O, LSE, W, (tO, tL, tW) = decode_ref(q, K, V, value_scales(c), lens, modes, sink, window, SCALE if scale is None else scale, bm)
    if spoiled:
        spoil(c, lens)
    h = handle(c, dev)
    B, Hq, _ = q.shape
    m = torch.tensor(modes, dtype=torch.uint8, device=dev)
    sl = torch.tensor(lens, dtype=torch.int32, device=dev)
    bmd = None if bm is None else torch.as_tensor(bm).to(dev)
    ws = ea.decode_q8_workspace(B, Hq, h.Hkv, h.capacity, num_splits, True, device=dev)
    kw = torch.full((B, h.Hkv, h.capacity), 0.5, device=dev)
    qd = q.to(dev)
    run = lambda **k: ea.ea_hybrid_attn_decode_q8(qd, h, sl, m, sink=sink, window=window, block_mask=bmd,
                                                  num_splits=num_splits, scale=scale, workspace=ws, **k)
    o1, l1 = run(key_weights=kw, accumulate=True)
    o2, l2 = run()
    kw2 = torch.full_like(kw, 0.25)
    run(key_weights=kw2, accumulate=False)
    check_no_device_error(ws)
    assert torch.equal(o1, o2) and torch.equal(l1, l2)        # with and without the weights
    got = o1.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all()
    assert (np.abs(got - O) <= tO).all(), float((np.abs(got - O) / np.maximum(tO, 1e-30)).max())
    gl = l1.cpu().numpy().astype(np.float64)
    assert (np.isneginf(gl) == np.isneginf(LSE)).all()
    fin = np.isfinite(LSE)
    assert (np.abs(gl[fin] - LSE[fin]) <= tL[fin]).all(), float((np.abs(gl[fin] - LSE[fin]) / tL[fin]).max())
    live = np.arange(h.capacity)[None, None, :] < np.array(lens)[:, None, None]
    w1, w2 = kw.cpu().numpy().astype(np.float64), kw2.cpu().numpy().astype(np.float64)
    live = np.broadcast_to(live, w1.shape)
    assert (w1[~live] == 0.5).all() and (w2[~live] == 0.25).all()
    assert (np.abs(w2 - W) <= tW + 2.0 ** -23 * W)[live].all()
    assert (np.abs(w1 - (W + 0.5)) <= tW + 2.0 ** -23 * (W + 0.5))[live].all()
    return o1, l1, kw2


LENS = [700, 0, 1, 15, 16, 17, 63, 64, 65, 128, 129, 640, 191]


def all_modes(B, Hkv):
    return [[(FULL, SSA, BLOCK)[(b + h) % 3] for h in range(Hkv)] for b in range(B)]


@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("sb,page", [(16, 0), (32, 64), (64, 0), (64, 192), (128, 128), (128, 0)])
@pytest.mark.parametrize("num_splits", [0, 3])
def test_ragged_batch_all_modes(dev, dtype, sb, page, num_splits):
    B, Hkv, g = len(LENS), 3, 4
    cap = 704 if page != 192 else 768
    cap = -(-cap // 128) * 128 if page == 128 else cap
    c = make_cache(B, cap, Hkv, dtype, sb, page, seed=sb + page)
    q = tokens((B, Hkv * g, 128), seed=5)
    bm = wl.block_mask(B, Hkv, cap, density=0.4, seed=6).numpy()
    bm[3] = 0                                     # sequence 3: its block head keeps nothing
    bm[0, :, 5, 5] = 0                            # sequence 0: the diagonal block dropped
    check(dev, c, q, LENS, all_modes(B, Hkv), 20, 90, bm, num_splits)


@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("g", [1, 2, 3, 5, 6, 7, 8])
def test_head_groups(dev, dtype, g):
    c = make_cache(2, 333, 2, dtype, 32, 0, seed=g)
    q = tokens((2, 2 * g, 128), seed=g)
    check(dev, c, q, [333, 200], [[FULL, SSA], [SSA, FULL]], 7, 100)


@pytest.mark.parametrize("dtype", [E4M3, INT8])
def test_one_row_cache(dev, dtype):
    c = make_cache(1, 1, 1, dtype, 16, 0, seed=1)
    check(dev, c, tokens((1, 4, 128), seed=2), [1], [[FULL]], 0, 1)


@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("B,Hkv", [(1, 2), (3, 8)])
def test_long_sequences_of_many_chunks(dev, dtype, B, Hkv):
    L = 9000
    c = make_cache(B, L, Hkv, dtype, 64, 0, seed=11)
    q = tokens((B, 2 * Hkv, 128), seed=12)
    check(dev, c, q, [L - 77 * b for b in range(B)], [[FULL, SSA] * (Hkv // 2)] * B, 64, 1000, spoiled=False)


@pytest.mark.parametrize("dtype", [E4M3, INT8])
def test_peaked_and_uneven_blocks(dev, dtype):
    # blocks of V differ in scale by 2^20, the keys by 2^6; logits of several hundred: a few keys hold all the weight
    B, Hkv, L = 2, 1, 640
    c = make_cache(B, L, Hkv, dtype, 64, 0, seed=21)
    c["vs"] *= torch.exp2(torch.tensor([0., 10, -10, 4, 0, -3, 7, -10, 1, 2]))
    c["ks"] *= torch.exp2(torch.tensor([0., 3, -3, 2, 0, -1, 1, 2, -2, 0]))
    q = (tokens((B, 8, 128), seed=22).float() * 4).to(BF16)
    check(dev, c, q, [640, 500], [[FULL], [SSA]], 100, 400)


def test_queries_of_any_magnitude(dev):
    # rows of q from 2^-100 to 2^100 (scale makes up for it), one of zeros: q enters the products as f16 after a power of two
    for k in (-100, -20, 20, 100):
        c = make_cache(1, 200, 1, E4M3, 64, 0, seed=31)
        q = tokens((1, 4, 128), seed=32)
        q[0, 3] = 0
        q = (q.float() * 2.0 ** k).to(BF16)
        check(dev, c, q, [200], [[FULL]], 0, 1, scale=SCALE * 2.0 ** -k)


def test_strided_queries_outputs_and_cache_views(dev):
    c = make_cache(2, 256, 2, INT8, 64, 0, seed=41)
    q = tokens((2, 8, 128), seed=42)
    wide = {k: torch.zeros(2, 256, 5, 128, dtype=INT8, device=dev) for k in "KV"}
    wk, wv = (wide[k][:, :, 1:3] for k in "KV")
    wk.copy_(c["K"]), wv.copy_(c["V"])
    h = ea.KVCache(wk, wv, c["ks"].to(dev), c["vs"].to(dev))
    wq = torch.zeros(2, 11, 128, dtype=BF16, device=dev)
    wq[:, 2:10] = q.to(dev)
    wo = torch.full((2, 9, 256), 3.0, dtype=BF16, device=dev)
    sl = torch.tensor([256, 100], dtype=torch.int32, device=dev)
    m = torch.tensor([[FULL, SSA], [SSA, FULL]], dtype=torch.uint8, device=dev)
    o, l = ea.ea_hybrid_attn_decode_q8(wq[:, 2:10], h, sl, m, sink=4, window=50, O=wo[:, :8, 128:])
    o2, l2 = ea.ea_hybrid_attn_decode_q8(q.to(dev), handle(c, dev), sl, m, sink=4, window=50)
    assert torch.equal(o, o2) and torch.equal(l, l2)
    assert (wo[:, 8] == 3).all() and (wo[:, :, :128] == 3).all()


def test_equals_the_bf16_decode_on_the_same_values(dev):
    # code * scale is a bf16 value: both decodes read the same numbers
    B, Hq, Hkv, L = 3, 16, 4, 5000
    c = make_cache(B, L, Hkv, E4M3, 64, 0, seed=51)
    K, V = (torch.from_numpy(x).to(BF16) for x in logical(c))
    q = tokens((B, Hq, 128), seed=52).to(dev)
    sl = torch.tensor([5000, 4097, 130], dtype=torch.int32, device=dev)
    m = torch.tensor([[FULL, SSA, SSA, FULL]] * B, dtype=torch.uint8, device=dev)
    o8, l8 = ea.ea_hybrid_attn_decode_q8(q, handle(c, dev), sl, m, sink=100, window=1000)
    o, l = ea.ea_hybrid_attn_decode(q, K.to(dev), V.to(dev), sl, m, sink=100, window=1000)
    assert (l8 - l).abs().max() < 1e-4
    # bf16 rounding on both sides, the other's bf16 probabilities
    assert (o8.float() - o.float()).abs().max() <= (2 * 2.0 ** -8 + 2.0 ** -8) * o.float().abs().max() + 2.0 ** -8


def test_nan_scales_reach_the_heads_that_keep_the_block(dev):
    c = make_cache(2, 256, 2, E4M3, 64, 0, seed=61)
    c["ks"][0, 0, 1] = float("nan")
    c["vs"][1, 1, 3] = float("nan")
    q = tokens((2, 4, 128), seed=62).to(dev)
    sl = torch.tensor([256, 256], dtype=torch.int32, device=dev)
    m = torch.tensor([[FULL, FULL], [FULL, SSA]], dtype=torch.uint8, device=dev)
    o, l = ea.ea_hybrid_attn_decode_q8(q, handle(c, dev), sl, m, sink=4, window=10)
    nan_o, nan_l = o.isnan(), l.isnan()
    assert nan_o[0, :2].all() and nan_l[0, :2].all() and nan_o[1, 2:].all() and nan_l[1, 2:].all()
    assert not nan_o[0, 2:].any() and not nan_o[1, :2].any()
    # a block that the mode does not keep does not matter; one that is all a row keeps is not an empty row
    m = torch.tensor([[SSA, FULL], [FULL, SSA]], dtype=torch.uint8, device=dev)
    o, l = ea.ea_hybrid_attn_decode_q8(q, handle(c, dev), torch.tensor([256, 100], dtype=torch.int32, device=dev), m, sink=4,
                                       window=10)
    assert not o.isnan().any() and not l.isnan().any()
    o, l = ea.ea_hybrid_attn_decode_q8(q, handle(c, dev), torch.tensor([128, 1], dtype=torch.int32, device=dev), m, sink=0,
                                       window=64)
    assert o[0, :2].isnan().all() and l[0, :2].isnan().all()


def test_bad_modes_lengths_and_pages_are_reported(dev):
    c = make_cache(4, 256, 1, INT8, 64, 64, seed=71)
    c["table"][3, 1] = 12345
    q = tokens((4, 4, 128), seed=72)
    ws = ea.decode_q8_workspace(4, 4, 1, 256, 0, True, device=dev)
    kw = torch.zeros(4, 1, 256, device=dev)
    lens, modes = [257, 100, 50, 200], [[FULL], [7], [BLOCK], [FULL]]
    o, l = ea.ea_hybrid_attn_decode_q8(q.to(dev), handle(c, dev), torch.tensor(lens, dtype=torch.int32, device=dev),
                                       torch.tensor(modes, dtype=torch.uint8, device=dev), sink=1, window=5,
                                       key_weights=kw, workspace=ws)
    assert ea.ea_check_errors(ws) == 6 and ea.ea_check_errors(ws) == 0
    assert (o[:3] == 0).all() and torch.isneginf(l[:3]).all() and (kw[:3] == 0).all()
    assert torch.isfinite(l[3]).all() or l[3].isnan().all()


def test_rows_beyond_two_to_the_32_bytes(dev):
    B, Lmax, Hkv = 5, 1 << 20, 8
    h = ea.kv_cache(B, Lmax, Hkv, dtype=E4M3, device=dev)
    K, V = tokens((B, 200, Hkv, 128), seed=81), tokens((B, 200, Hkv, 128), seed=82)
    start = [0, 0, 0, 0, Lmax - 200]
    ea.ea_cache_write(h, K.to(dev), V.to(dev), torch.tensor(start, dtype=torch.int32, device=dev))
    q = tokens((B, 8, 128), seed=83)
    sl = torch.tensor([200, 0, 1, 200, Lmax], dtype=torch.int32, device=dev)
    m = torch.full((B, Hkv), SSA, dtype=torch.uint8, device=dev)
    o, l = ea.ea_hybrid_attn_decode_q8(q.to(dev), h, sl, m, sink=0, window=200)
    small = ea.kv_cache(B, 256, Hkv, dtype=E4M3, device=dev)
    # the same tokens at the same places of their blocks in a small cache
    off = (Lmax - 200) % 64
    ea.ea_cache_write(small, K.to(dev), V.to(dev), torch.tensor([0, 0, 0, 0, off], dtype=torch.int32, device=dev))
    o2, l2 = ea.ea_hybrid_attn_decode_q8(q.to(dev), small, torch.tensor([200, 0, 1, 200, 200 + off], dtype=torch.int32, device=dev), m,
                                         sink=0, window=200)
    assert torch.equal(o, o2) and torch.equal(l, l2)


def test_captured_step_with_weights(dev):
    # append + decode with weights captured once, replayed with new queries, tokens and lengths
    B, Hkv, g = 12, 2, 4
    c = make_cache(B, 512, Hkv, E4M3, 64, 64, seed=91)
    h, h2 = handle(c, dev), handle(c, dev)
    lens = torch.tensor([5 * b for b in range(B)], dtype=torch.int32, device=dev)
    lens1 = lens + 1
    q = tokens((B, Hkv * g, 128), seed=92).to(dev)
    k1, v1 = tokens((B, 1, Hkv, 128), seed=93).to(dev), tokens((B, 1, Hkv, 128), seed=94).to(dev)
    m = torch.tensor(all_modes(B, Hkv), dtype=torch.uint8, device=dev)
    bm = torch.as_tensor(wl.block_mask(B, Hkv, 512, seed=95)).to(dev)
    ws = ea.decode_q8_workspace(B, Hkv * g, Hkv, 512, weights=True, device=dev)
    kw, kw2 = (torch.zeros(B, Hkv, 512, device=dev) for _ in range(2))
    O, LSE = torch.empty(B, Hkv * g, 128, dtype=BF16, device=dev), torch.empty(B, Hkv * g, device=dev)

    def step(cache, w, O, LSE, ws):
        ea.ea_cache_write(cache, k1, v1, lens, workspace=ws)
        ea.ea_hybrid_attn_decode_q8(q, cache, lens1, m, sink=8, window=64, block_mask=bm, key_weights=w, O=O, LSE=LSE,
                                    workspace=ws)

    step(h, kw, O, LSE, ws)
    step(h2, kw2, O, LSE, ws)
    torch.cuda.synchronize()
    g_ = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g_):
        step(h, kw, O, LSE, ws)
    O2, LSE2, ws2 = torch.empty_like(O), torch.empty_like(LSE), torch.zeros_like(ws)
    for i in range(3):
        q.copy_(tokens(tuple(q.shape), seed=100 + i))
        k1.copy_(tokens(tuple(k1.shape), seed=200 + i))
        lens.add_(37)
        lens1.copy_(lens + 1)
        g_.replay()
        step(h2, kw2, O2, LSE2, ws2)
        torch.cuda.synchronize()
        assert torch.equal(O, O2) and torch.equal(LSE, LSE2) and torch.equal(kw, kw2)
        assert torch.equal(h.K.view(torch.uint8), h2.K.view(torch.uint8)) and torch.equal(h.k_scale, h2.k_scale)
    check_no_device_error(ws)


def test_two_streams_with_their_own_workspaces(dev):
    c = make_cache(4, 2000, 2, INT8, 64, 0, seed=111)
    h = handle(c, dev)
    sl = torch.tensor([2000, 1000, 500, 1], dtype=torch.int32, device=dev)
    m = torch.full((4, 2), FULL, dtype=torch.uint8, device=dev)
    qs = [tokens((4, 8, 128), seed=112 + i).to(dev) for i in range(2)]
    want = [ea.ea_hybrid_attn_decode_q8(q, h, sl, m, sink=0, window=1)[0].clone() for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            got[i].append(ea.ea_hybrid_attn_decode_q8(qs[i], h, sl, m, sink=0, window=1, stream=streams[i])[0])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])


@pytest.mark.parametrize("dtype", [E4M3, INT8])
def test_many_short_sequences_beside_a_few_long_ones(dev, dtype):
    # more units than the planner has threads, most of them a chunk of one tile, some none
    B, Hkv, cap = 150, 2, 4096
    c = make_cache(B, cap, Hkv, dtype, 64, 64, seed=121)
    rng = np.random.default_rng(122)
    lens = [int(x) for x in rng.integers(0, 130, B)]
    lens[0], lens[70], lens[149] = 4096, 4001, 3000
    check(dev, c, tokens((B, 2 * Hkv, 128), seed=123), lens, [[FULL, SSA]] * B, 3, 60)


def test_steps_one_after_another_share_a_workspace(dev):
    # three steps with key weights, then without, in one stream and one graph: no step starts before the one before it has
    # read its results
    B, Hkv, g, L = 6, 4, 4, 3000
    c = make_cache(B, L, Hkv, INT8, 32, 0, seed=131)
    h = handle(c, dev)
    sl = torch.tensor([3000, 0, 1, 64, 2111, 999], dtype=torch.int32, device=dev)
    m = torch.tensor(all_modes(B, Hkv), dtype=torch.uint8, device=dev)
    bm = torch.as_tensor(wl.block_mask(B, Hkv, L, density=0.3, seed=132)).to(dev)
    qs = [tokens((B, Hkv * g, 128), seed=133 + i).to(dev) for i in range(3)]

    def steps(ws):
        out = []
        for q in qs:
            w = torch.zeros(B, Hkv, L, device=dev)
            out += list(ea.ea_hybrid_attn_decode_q8(q, h, sl, m, sink=9, window=300, block_mask=bm, key_weights=w,
                                                    workspace=None if ws is None else ws)) + [w]
            out += list(ea.ea_hybrid_attn_decode_q8(q, h, sl, m, sink=9, window=300, block_mask=bm, num_splits=2,
                                                    workspace=None if ws is None else ws))
        return out

    want = []
    for q in qs:                                    # each alone, with workspaces of their own
        w = torch.zeros(B, Hkv, L, device=dev)
        want += list(ea.ea_hybrid_attn_decode_q8(q, h, sl, m, sink=9, window=300, block_mask=bm, key_weights=w)) + [w]
        torch.cuda.synchronize()
        want += list(ea.ea_hybrid_attn_decode_q8(q, h, sl, m, sink=9, window=300, block_mask=bm, num_splits=2))
        torch.cuda.synchronize()
    ws = torch.zeros(max(ea.ea_decode_q8_workspace_size(B, Hkv * g, Hkv, L, n, w) for n, w in ((0, True), (2, False))),
                     dtype=torch.uint8, device=dev)
    got = steps(ws)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = steps(ws)
    for _ in range(3):
        for t in captured:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, want))
    check_no_device_error(ws)


def test_equal_calls_give_equal_bits_whatever_cta_takes_a_chunk(dev):
    # several chunks of many lengths for each SM, taken from a queue in another order every time
    B, Hkv, g, L = 7, 8, 2, 20000
    gen = torch.Generator(device=dev).manual_seed(141)
    c = ea.kv_cache(B, L, Hkv, dtype=INT8, scale_block=32, device=dev)
    for x in (c.K, c.V):
        x.copy_(torch.randint(-127, 128, x.shape, generator=gen, device=dev, dtype=torch.int8))
    for x in (c.k_scale, c.v_scale):
        x.copy_(torch.exp2(torch.randint(-9, -5, x.shape, generator=gen, device=dev).float()))
    sl = torch.tensor([20000, 19999, 17777, 12345, 9000, 64, 15001], dtype=torch.int32, device=dev)
    m = torch.tensor(all_modes(B, Hkv), dtype=torch.uint8, device=dev)
    bm = torch.as_tensor(wl.block_mask(B, Hkv, L, density=0.5, seed=142)).to(dev)
    q = tokens((B, Hkv * g, 128), seed=143).to(dev)
    ws = ea.decode_q8_workspace(B, Hkv * g, Hkv, L, device=dev)
    run = lambda: ea.ea_hybrid_attn_decode_q8(q, c, sl, m, sink=100, window=5000, block_mask=bm, workspace=ws)
    o, l = run()
    for _ in range(60):
        got = [run() for _ in range(10)]
        assert all(torch.equal(o, a) and torch.equal(l, b) for a, b in got)
    check_no_device_error(ws)


@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("page", [64, 192])
def test_keys_of_missing_pages_count_as_zeros(dev, dtype, page):
    # reported, and read as zeros with a scale of 1: logits of 0, nothing added to the output
    B, Hkv, g, cap = 5, 3, 4, 768
    c = make_cache(B, cap, Hkv, dtype, 32, page, seed=151)
    n = c["table"].shape[1]
    c["table"][0, 1], c["table"][1, n - 1], c["table"][2] = 12345, -1, c["K"].shape[0]
    c["table"][3, 0] = -(1 << 31)
    lens, modes = [768, 768, 700, 200, 500], all_modes(B, Hkv)
    q = tokens((B, Hkv * g, 128), seed=152)
    bm = wl.block_mask(B, Hkv, cap, density=0.5, seed=153).numpy()
    K, V = logical(c)
    O, LSE, W, (tO, tL, tW) = decode_ref(q, K, V, value_scales(c), lens, modes, 20, 300, SCALE, bm)
    ws = ea.decode_q8_workspace(B, Hkv * g, Hkv, cap, 0, True, device=dev)
    kw = torch.zeros(B, Hkv, cap, device=dev)
    o, l = ea.ea_hybrid_attn_decode_q8(q.to(dev), handle(c, dev), torch.tensor(lens, dtype=torch.int32, device=dev),
                                       torch.tensor(modes, dtype=torch.uint8, device=dev), sink=20, window=300,
                                       block_mask=torch.as_tensor(bm).to(dev), key_weights=kw, workspace=ws)
    assert ea.ea_check_errors(ws) == 6
    assert (np.abs(o.double().cpu().numpy() - O) <= tO).all()
    gl = l.double().cpu().numpy()
    fin = np.isfinite(LSE)
    assert (np.isneginf(gl) == ~fin).all() and (np.abs(gl[fin] - LSE[fin]) <= tL[fin]).all()
    assert (np.abs(kw.double().cpu().numpy() - W) <= tW + 2.0 ** -23 * W).all()
