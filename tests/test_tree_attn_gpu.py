"""Attention of a tree of drafted tokens over a cache against a plain implementation in
64 bits: formats, pages, head groups, modes, lengths and counts from none on, masks,
what lies in masked places, and a whole step as a server runs it."""
import math

import numpy as np
import pytest
import torch

import sparse_head_attention_gb300 as ea
from cache_reference import capacity, logical, make_cache, rows_of, tokens, value_scales
from gpu_helpers import check_no_device_error, gpu_device
from tree_reference import accept, attend, inv_freq, plan, random_tree, rotate, units

pytestmark = pytest.mark.gpu
E4M3, INT8, BF16 = torch.float8_e4m3fn, torch.int8, torch.bfloat16
FULL, SSA, BLOCK = ea.FULL, ea.SSA, ea.BLOCK
SCALE = 128 ** -0.5
KEEP = 7.5                                            # what an output row that must stay holds


@pytest.fixture(scope="module")
def dev():
    return gpu_device()


def handle(c, dev):
    t = {k: None if v is None else v.to(dev) for k, v in c.items() if k in ("K", "V", "ks", "vs", "table")}
    return ea.KVCache(t["K"], t["V"], t["ks"], t["vs"], scale_block=c["sb"], block_table=t["table"])


def spoil(c, lens):
    """NaN behind every sequence's end, codes and scales (of blocks that hold none of its tokens)."""
    for b, L in enumerate(lens):
        for p in range(L, capacity(c)):
            o, r = rows_of(c, b, p)
            for kv, sc in (("K", "ks"), ("V", "vs")):
                if c["ks"] is None:
                    c[kv][o, r] = math.nan
                else:
                    c[kv].view(torch.uint8)[o, r] = 0x7f if c[kv].dtype == E4M3 else 0x80
                    if p % c["sb"] == 0:
                        c[sc][o, :, r // c["sb"]] = math.nan


def i32(v, dev):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=dev)


def near(O, LSE, ref, n, T, what=""):
    O, LSE = O.float().cpu().numpy().astype(np.float64), LSE.cpu().numpy().astype(np.float64)
    rO, rL, tO, tL = ref
    for b in range(len(n)):
        assert (O[b, n[b] :] == KEEP).all() and (LSE[b, :, n[b] :] == KEEP).all(), (what, b, "rows behind the last")
        o, l = O[b, : n[b]], LSE[b, :, : n[b]]
        none = np.isneginf(rL[b, :, : n[b]])
        assert np.array_equal(np.isneginf(l), none), (what, b, "empty rows")
        with np.errstate(invalid="ignore"):
            bad = ~(np.abs(l - rL[b, :, : n[b]]) <= tL[b, :, : n[b]]) & ~none
        assert not bad.any(), (what, b, "LSE", np.argwhere(bad)[:4], l[bad][:4], rL[b, :, : n[b]][bad][:4])
        bad = ~(np.abs(o - rO[b, : n[b]]) <= tO[b, : n[b]] + 2.0 ** -100)
        assert not bad.any(), (what, b, "O", bad.sum(), np.argwhere(bad)[:4], o[bad][:4], rO[b, : n[b]][bad][:4])


def inputs(B, T, Hq, Hkv, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(B, T, Hq, 128, generator=g).to(BF16), tokens((B, T, Hkv, 128), seed + 1), tokens((B, T, Hkv, 128), seed + 2)


def out(B, T, Hq, dev):
    return (torch.full((B, T, Hq, 128), KEEP, dtype=BF16, device=dev), torch.full((B, Hq, T), KEEP, dtype=torch.float32, device=dev))


def check(dev, c, Hq, Hkv, T, lens, n, modes, sink=16, window=100, kind="tree", seed=0, bm=None, scale=None):
    B = len(lens)
    Q, K, V = inputs(B, T, Hq, Hkv, seed)
    p = random_tree(B, T, seed, kind)
    depth, mask = plan(p, n)
    Kc, Vc = logical(c)
    ref = attend(*(x.double().numpy() for x in (Q, K, V)), Kc, Vc, lens, n, depth, mask, modes, sink, window, scale or SCALE, bm,
                 None if c["ks"] is None else units(value_scales(c), lens))
    spoil(c, lens)
    for b in range(B):
        K[b, n[b] :], V[b, n[b] :] = math.nan, math.inf
    h = handle(c, dev)
    ws = ea.tree_workspace(B, T, Hq, Hkv, h.capacity, device=dev)
    args = [x.to(dev) for x in (Q, K, V)] + [h, i32(lens, dev), i32(depth, dev), i32(mask, dev), torch.tensor(modes, dtype=torch.uint8, device=dev)]
    kw = dict(sink=sink, window=window, n_nodes=i32(n, dev), block_mask=None if bm is None else torch.as_tensor(bm).to(dev), scale=scale, workspace=ws)
    O, LSE = out(B, T, Hq, dev)
    ea.ea_hybrid_attn_tree(*args, O=O, LSE=LSE, **kw)
    check_no_device_error(ws)
    near(O, LSE, ref, n, T)
    O2, LSE2 = out(B, T, Hq, dev)
    ea.ea_hybrid_attn_tree(*args, O=O2, LSE=LSE2, **kw)
    assert torch.equal(O, O2) and torch.equal(LSE, LSE2)


FORMATS = [(BF16, 64, 0), (BF16, 64, 64), (BF16, 64, 256), (E4M3, 32, 0), (INT8, 64, 64), (E4M3, 128, 128), (INT8, 16, 0)]


@pytest.mark.parametrize("dtype,sb,page", FORMATS)
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 4, 1), (16, 8, 2), (40, 8, 2)])
def test_full_heads(dev, dtype, sb, page, T, Hq, Hkv):
    lens = [300, 0, 1, 128, 65]
    n = [T, T, max(1, T - 3), 0, (T + 1) // 2]
    check(dev, make_cache(5, 320, Hkv, dtype, sb, page, 11), Hq, Hkv, T, lens, n, [[FULL] * Hkv] * 5, seed=T)


@pytest.mark.parametrize("g", [1, 3, 5, 7, 16, 48, 64])
def test_head_groups(dev, g):
    T = 128 if g < 3 else 50
    lens, n = [200, 33], [T, T // 3]
    check(dev, make_cache(2, 256, 1, BF16, 64, 0, 5), g, 1, T, lens, n, [[FULL], [SSA]], seed=g, sink=7, window=60)


@pytest.mark.parametrize("kind", ["tree", "chain", "star", "forest"])
@pytest.mark.parametrize("dtype,sb,page", [(BF16, 64, 64), (INT8, 32, 0)])
def test_trees(dev, kind, dtype, sb, page):
    T = 128
    check(dev, make_cache(3, 192, 2, dtype, sb, page, 3), 4, 2, T, [190, 64, 0], [128, 99, 33], [[FULL, SSA]] * 3, kind=kind, seed=4, sink=3, window=40)


@pytest.mark.parametrize("dtype,sb,page", FORMATS)
@pytest.mark.parametrize("sink,window", [(0, 1), (5, 2), (128, 256), (200, 130), (0, 5000)])
def test_streaming_heads(dev, dtype, sb, page, sink, window):
    lens, n, T = [1000, 129, 700, 2, 0], [20, 7, 20, 20, 1], 20
    check(dev, make_cache(5, 1024, 1, dtype, sb, page, 8), 4, 1, T, lens, n, [[SSA]] * 5, sink=sink, window=window, kind="chain", seed=3)


def blocks(B, Hkv, cap, seed, share):
    n = -(-cap // 128)
    return (np.random.RandomState(seed).rand(B, Hkv, n, n) < share).astype(np.uint8)


@pytest.mark.parametrize("dtype,sb,page", [(BF16, 64, 0), (BF16, 64, 64), (E4M3, 64, 0), (INT8, 16, 128)])
@pytest.mark.parametrize("share", [0.0, 0.4, 1.0])
def test_block_heads(dev, dtype, sb, page, share):
    # nodes on both sides of a block's border, on one side, without a cache
    lens, n, T = [1020, 640, 900, 0], [64, 64, 9, 64], 64
    cap = 1152
    bm = blocks(4, 2, cap, 6, share)
    check(dev, make_cache(4, cap, 2, dtype, sb, page, 9), 8, 2, T, lens, n, [[BLOCK, FULL], [BLOCK, BLOCK], [SSA, BLOCK], [BLOCK, SSA]], kind="chain", seed=6, bm=bm)


@pytest.mark.parametrize("dtype,sb,page", [(BF16, 64, 0), (E4M3, 64, 256)])
def test_many_short_sequences(dev, dtype, sb, page):
    """More units than CTAs, ranges over several of them."""
    B, T = 45, 3
    r = np.random.RandomState(0)
    lens, n = r.randint(0, 400, B).tolist(), r.randint(0, T + 1, B).tolist()
    check(dev, make_cache(B, 512, 8, dtype, sb, page, 1), 16, 8, T, lens, n, [[(b + h) % 2 for h in range(8)] for b in range(B)], seed=2)


@pytest.mark.parametrize("dtype,sb,page", [(BF16, 64, 0), (INT8, 64, 64)])
def test_one_long_sequence(dev, dtype, sb, page):
    """A unit over many CTAs, two M tiles."""
    check(dev, make_cache(1, 20032, 1, dtype, sb, page, 1), 8, 1, 24, [20000], [24], [[FULL]], seed=2)


def test_extreme_scores(dev):
    """Logits far apart: the running maximum has to follow; a large scale."""
    c = make_cache(1, 600, 1, BF16, 64, 0, 2)
    c["K"][0, 400:] *= 16.0
    check(dev, c, 4, 1, 8, [600], [8], [[FULL]], seed=1, scale=0.3)


def test_non_finite_in_masked_places(dev):
    """Infinities and NaN in keys and values that some rows keep and others do not: only the rows that keep one get it."""
    for dtype in (BF16, E4M3):
        B, T, Hq, lens, n = 2, 6, 4, [500, 3], [6, 6]
        Q, K, V = inputs(B, T, Hq, 1, 3)
        p = np.array([[-1, 0, 1, 1, 0, 4]] * 2, np.int32)
        depth, mask = plan(p, n)
        modes, sink, window = [[SSA], [FULL]], 10, 200
        c = make_cache(B, 512, 1, dtype, 16, 0, 4)
        V[0, 3, 0, 5], V[1, 4, 0, 9], K[1, 2, 0, 1] = math.nan, math.inf, math.nan
        first = 500 - window + 1                                  # depth 0 keeps it, the nodes below do not
        if dtype == BF16:
            c["V"][0, first, 0, 77] = -math.inf
        ref = attend(*(np.nan_to_num(x.double().numpy(), nan=0.0, posinf=0.0) for x in (Q, K, V)),
                     *(np.nan_to_num(x, neginf=0.0) for x in logical(c)), lens, n, depth, mask, modes, sink, window, SCALE,
                     vunit=None if dtype == BF16 else units(value_scales(c), lens))
        h = handle(c, dev)
        ws = ea.tree_workspace(B, T, Hq, 1, 512, device=dev)
        O, LSE = out(B, T, Hq, dev)
        ea.ea_hybrid_attn_tree(Q.to(dev), K.to(dev), V.to(dev), h, i32(lens, dev), i32(depth, dev), i32(mask, dev),
                               torch.tensor(modes, dtype=torch.uint8, device=dev), sink=sink, window=window, O=O, LSE=LSE, workspace=ws)
        check_no_device_error(ws)
        o = O.float().cpu().numpy()
        hit = lambda b, t, d: not np.isfinite(o[b, t, :, d]).any()  # noqa: E731
        assert hit(0, 3, 5) and hit(1, 4, 9) and hit(1, 5, 9) and np.isposinf(o[1, 4, :, 9]).all()
        assert np.isnan(o[1, 2]).all() and torch.isnan(LSE[1, :, 2]).all()
        clean = np.isfinite(o)
        want = np.ones_like(clean)
        want[0, 3, :, 5] = want[1, 4, :, 9] = want[1, 5, :, 9] = want[1, 2] = False
        if dtype == BF16:
            want[0, 0, :, 77] = False
            assert np.isneginf(o[0, 0, :, 77]).all()
        assert np.array_equal(clean, want)
        err = np.abs(o - ref[0])
        assert (err[want] <= ref[2][want]).all()


def test_reports(dev):
    """Bad lengths, counts, depths, modes, masks and pages: reported, nothing out of range is touched."""
    T, Hq = 4, 4
    Q, K, V = (x.to(dev) for x in inputs(2, T, Hq, 1, 3))
    depth, mask = plan(random_tree(2, T, 1, "chain"), [T, T])
    c = handle(make_cache(2, 128, 1, BF16, 64, 0, 4), dev)
    ws = ea.tree_workspace(2, T, Hq, 1, 128, device=dev)
    bm = torch.ones(2, 1, 1, 1, dtype=torch.uint8, device=dev)

    def run(cache=c, lens=(100, 50), n=(4, 4), d=depth, modes=(FULL, FULL), block_mask=None):
        O, LSE = out(2, T, Hq, dev)
        ea.ea_hybrid_attn_tree(Q, K, V, cache, i32(lens, dev), i32(d, dev), i32(mask, dev), torch.tensor(modes, dtype=torch.uint8, device=dev).view(2, 1),
                               sink=4, window=64, n_nodes=i32(n, dev), block_mask=block_mask, O=O, LSE=LSE, workspace=ws)
        return ea.ea_check_errors(ws), O.float().cpu().numpy(), LSE.cpu().numpy()

    st, good, lse = run()
    assert st == 0
    for kw in (dict(lens=(129, 50)), dict(lens=(-1, 50)), dict(modes=(3, FULL)), dict(modes=(BLOCK, FULL)),
               dict(lens=(125, 50), modes=(BLOCK, FULL), block_mask=bm)):
        st, o, l = run(**kw)
        assert st == 6 and not o[0].any() and np.isneginf(l[0]).all() and np.array_equal(o[1], good[1]), kw
    for n in ((5, 4), (-1, 4)):
        st, o, l = run(n=n)
        assert st == 6 and (o[0] == KEEP).all() and (l[0] == KEEP).all() and np.array_equal(o[1], good[1])
    d = depth.copy()
    d[0, 3], d[0, 0] = 4, -1
    st, o, _ = run(d=d)
    assert st == 6 and np.array_equal(o, good)            # (a full head's mask has no use for the depth)
    st, o, _ = run(modes=(BLOCK, FULL), lens=(124, 50), block_mask=bm)
    assert st == 0 and np.isfinite(o).all() and o[0].any()
    table = torch.tensor([[0, 7], [1, -1]], dtype=torch.int32, device=dev)
    p = handle(make_cache(1, 256, 1, BF16, 64, 0, 4), dev)
    pool = ea.KVCache(p.K.view(4, 64, 1, 128), p.V.view(4, 64, 1, 128), block_table=table)
    st, o, _ = run(cache=pool, lens=(100, 64))
    assert st == 6 and np.isfinite(o).all()
    st, o, _ = run(cache=pool, lens=(64, 64))             # pages behind the length are not looked at
    assert st == 0


def test_strides_streams_and_graphs(dev):
    """Parts of one projection's output, another stream, a captured call replayed with new lengths and contents."""
    B, T, Hq, Hkv = 2, 9, 8, 2
    qkv = tokens((B, T, Hq + 2 * Hkv, 128), 5).to(dev)
    q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq : Hq + Hkv], qkv[:, :, Hq + Hkv :]
    p = random_tree(B, T, 3)
    depth, mask = (i32(x, dev) for x in plan(p, [T, T]))
    m = torch.tensor([[FULL, SSA], [SSA, FULL]], dtype=torch.uint8, device=dev)
    c = handle(make_cache(B, 500, Hkv, E4M3, 64, 0, 2), dev)
    lens = i32([400, 30], dev)
    ws = ea.tree_workspace(B, T, Hq, Hkv, 500, device=dev)
    call = lambda a, b, e, **kw: ea.ea_hybrid_attn_tree(a, b, e, c, lens, depth, mask, m, sink=4, window=64, **kw)  # noqa: E731
    ref = call(q.contiguous(), k.contiguous(), v.contiguous())
    O = torch.empty(T, B, Hq, 128, dtype=BF16, device=dev).transpose(0, 1)
    got = call(q, k, v, O=O, workspace=ws)
    assert got[0] is O and torch.equal(O, ref[0]) and torch.equal(got[1], ref[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = call(q, k, v, stream=s)
    s.synchronize()
    assert torch.equal(got[0], ref[0]) and call(q, k, v, want_lse=False)[1] is None
    g = torch.cuda.CUDAGraph()
    LSE = torch.empty(B, Hq, T, device=dev)
    with torch.cuda.graph(g):
        call(q, k, v, O=O, LSE=LSE, workspace=ws)
    for L in ([500, 0], [1, 129], [256, 300]):
        lens.copy_(i32(L, dev))
        qkv.mul_(-1.25)
        g.replay()
        ref = call(q, k, v)
        assert torch.equal(O, ref[0]) and torch.equal(LSE, ref[1])
    check_no_device_error(ws)


@pytest.mark.parametrize("dtype", [BF16, INT8])
def test_single_token_is_the_decode(dev, dtype):
    """T = 1 over a cache equals a decode over the cache with that token in it."""
    B, Hq, Hkv, L = 3, 8, 2, [200, 64, 1]
    c = handle(make_cache(B, 256, Hkv, dtype, 64, 0, 7), dev)
    Q, K, V = (x.to(dev) for x in inputs(B, 1, Hq, Hkv, 1))
    m = torch.tensor([[FULL, SSA]] * B, dtype=torch.uint8, device=dev)
    one = torch.zeros(B, 1, dtype=torch.int32, device=dev)
    depth, mask = ea.ea_tree_plan(one - 1)
    O, LSE = ea.ea_hybrid_attn_tree(Q, K, V, c, i32(L, dev), depth, mask, m, sink=4, window=30)
    ea.ea_cache_write(c, K, V, start=i32(L, dev))
    n = i32(np.array(L) + 1, dev)
    if dtype == BF16:
        o, lse = ea.ea_hybrid_attn_decode(Q[:, 0], c.K, c.V, n, m, sink=4, window=30)
        assert (O[:, 0].float() - o.float()).abs().max() <= 2.0 ** -6 * o.float().abs().max() and (LSE[:, :, 0] - lse).abs().max() < 1e-4
    else:                                               # the token itself is rounded to 8 bits there
        o, lse = ea.ea_hybrid_attn_decode_q8(Q[:, 0], c, n, m, sink=4, window=30)
        assert (LSE[:, :, 0] - lse).abs().max() < 0.2


def test_a_whole_step(dev):
    """Masks, rotation, attention, acceptance and the accepted tokens' way into the cache, as a server runs them twice."""
    B, T, Hq, Hkv, cap = 3, 12, 8, 2, 256
    r = np.random.RandomState(1)
    f = inv_freq(128)
    fd = torch.from_numpy(f).to(dev)
    lens = [100, 0, 37]
    c = make_cache(B, cap, Hkv, BF16, 64, 64, 3)
    h = handle(c, dev)
    Kc, Vc = logical(c)
    ws, cws = ea.tree_workspace(B, T, Hq, Hkv, cap, device=dev), ea.cache_workspace(dev)
    modes = [[FULL, SSA]] * B
    m = torch.tensor(modes, dtype=torch.uint8, device=dev)
    start = i32(lens, dev)
    for step in range(2):
        p = random_tree(B, T, step, "tree")
        n = [T, T - 2, 5]
        Q, K, V = inputs(B, T, Hq, Hkv, 10 * step)
        tok, tgt = r.randint(0, 3, (B, T)), r.randint(0, 3, (B, T))
        nd, pd = i32(n, dev), i32(p, dev)
        depth, mask = ea.ea_tree_plan(pd, nd, workspace=cws)
        qr, kr = ea.ea_rope(Q.to(dev), K.to(dev), start[:, None] + depth, fd, n_new=nd, workspace=cws)
        O, LSE = out(B, T, Hq, dev)
        ea.ea_hybrid_attn_tree(qr, kr, V.to(dev), h, start, depth, mask, m, sink=8, window=64, n_nodes=nd, O=O, LSE=LSE, workspace=ws)
        path, count, nxt = ea.ea_tree_accept(i32(tok, dev), pd, i32(tgt, dev), nd, workspace=cws)
        ea.ea_cache_write_rope(h, K.to(dev), V.to(dev), fd, start=start, n_new=count, rows=path, workspace=cws)
        start = start + count
        check_no_device_error(ws)
        check_no_device_error(cws)
        d, mk = plan(p, n)
        got = [x.double().cpu().numpy() for x in (qr, kr)]
        for b in range(B):
            for x, y in ((Q, got[0]), (K, got[1])):
                w = rotate(x[b, : n[b]].double().numpy(), lens[b] + d[b, : n[b]], f, False)
                assert (np.abs(y[b, : n[b]] - w) <= np.abs(w) * 2.0 ** -8 + 1e-4).all()
        near(O, LSE, attend(got[0], got[1], V.double().numpy(), Kc, Vc, lens, n, d, mk, modes, 8, 64, SCALE), n, T, step)
        rp, rc, rn = accept(tok, p, tgt, n)
        assert np.array_equal(path.cpu().numpy(), rp) and np.array_equal(count.cpu().numpy(), rc) and np.array_equal(nxt.cpu().numpy(), rn)
        for b in range(B):
            for i in range(rc[b]):
                Kc[b, lens[b] + i], Vc[b, lens[b] + i] = got[1][b, rp[b, i]], V[b, rp[b, i]].double().numpy()
            lens[b] += int(rc[b])
        now = logical(dict(c, K=h.K.cpu(), V=h.V.cpu()))
        for b in range(B):                               # the accepted ones alone, with the bits that attended
            assert np.array_equal(now[0][b, : lens[b]], Kc[b, : lens[b]]) and np.array_equal(now[1][b, : lens[b]], Vc[b, : lens[b]])


def test_two_calls_at_once(dev):
    """Two streams, each with a workspace of its own, over one cache and shared pages."""
    B, T, Hq, Hkv = 2, 20, 16, 2
    c = make_cache(1, 512, Hkv, BF16, 64, 64, 4)
    table = c["table"].repeat(B, 1).contiguous()          # both sequences read the same pages, a row each
    h = ea.KVCache(c["K"].to(dev), c["V"].to(dev), block_table=table.to(dev))
    Q, K, V = (x.to(dev) for x in inputs(B, T, Hq, Hkv, 9))
    depth, mask = (i32(x, dev) for x in plan(random_tree(B, T, 3), [T] * B))
    m = torch.tensor([[FULL, SSA]] * B, dtype=torch.uint8, device=dev)
    lens = i32([500, 300], dev)
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [ea.tree_workspace(B, T, Hq, Hkv, h.capacity, device=dev) for _ in streams]
    call = lambda w, s: ea.ea_hybrid_attn_tree(Q, K, V, h, lens, depth, mask, m, sink=4, window=64, workspace=w, stream=s)  # noqa: E731
    ref = call(ws[0], None)
    torch.cuda.synchronize()
    got = [[call(w, s) for w, s in zip(ws, streams)] for _ in range(20)]
    torch.cuda.synchronize()
    for pair in got:
        for o, l in pair:
            assert torch.equal(o, ref[0]) and torch.equal(l, ref[1])
    for w in ws:
        check_no_device_error(w)


def test_masks_that_leave_nothing(dev):
    """No ancestors, no cache: zero and -inf, for some rows and for all."""
    B, T, Hq = 2, 5, 4
    Q, K, V = (x.to(dev) for x in inputs(B, T, Hq, 1, 2))
    depth = torch.zeros(B, T, dtype=torch.int32, device=dev)
    mask = torch.zeros(B, T, 4, dtype=torch.int32, device=dev)
    mask[1, 2, 0] = 1 << 4
    m = torch.zeros(B, 1, dtype=torch.uint8, device=dev)
    for dtype in (BF16, INT8):
        c = handle(make_cache(B, 128, 1, dtype, 64, 0, 1), dev)
        O, LSE = ea.ea_hybrid_attn_tree(Q, K, V, c, i32([0, 0], dev), depth, mask, m, sink=0, window=1)
        none = torch.ones(B, T, dtype=torch.bool, device=dev)
        none[1, 2] = False
        assert not O[none].any() and torch.isneginf(LSE.transpose(1, 2)[none]).all()
        assert (O[1, 2].float() - V[1, 4, 0].float()).abs().max() <= 2.0 ** -8 * V[1, 4].float().abs().max()
