"""The attention weights that queries give their keys against a plain
implementation in 64 bits (its tolerance is derived there), and the whole run
that they serve: prefill, weights, 8-bit cache, eviction, decode."""
import numpy as np
import pytest
import torch

import sparse_head_attention_gb300 as ea
from cache_reference import (decode_ref, key_weights_ref, logical, select_ref, tokens, value_scales,
                             write_ref)
from gpu_helpers import check_no_device_error, gpu_device
from sparse_head_attention_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
E4M3, INT8, BF16 = torch.float8_e4m3fn, torch.int8, torch.bfloat16
FULL, SSA, BLOCK = ea.FULL, ea.SSA, ea.BLOCK
SCALE = 128 ** -0.5


@pytest.fixture(scope="module")
def dev():
    return gpu_device()


def all_modes(B, Hkv):
    return [[(FULL, SSA, BLOCK)[(b + h) % 3] for h in range(Hkv)] for b in range(B)]


def row_lse(Q, K, modes, sink, window, lens, bm):
    """LSE [B, Hq, Tq] of the kept keys of each row, -inf where there are none, 7 for rows before the sequence."""
    Q, K = Q.double().numpy(), K.double().numpy()
    B, Tq, Hq, _ = Q.shape
    g = Hq // K.shape[2]
    out = np.full((B, Hq, Tq), 7.0)
    for b, L in enumerate(lens):
        t = np.arange(max(0, Tq - L), Tq)
        if not len(t):
            continue
        i, j = (L - Tq + t)[:, None], np.arange(L)[None, :]
        for q in range(Hq):
            h = q // g
            keep = j <= i
            if modes[b][h] == SSA:
                keep = keep & ((j < sink) | (i - j < window))
            elif modes[b][h] == BLOCK:
                keep = keep & (bm[b, h][i // 128, j // 128] != 0)
            x = np.where(keep, SCALE * (Q[b, t, q] @ K[b, :L, h].T), -np.inf)
            top = x.max(1)
            with np.errstate(divide="ignore"):
                out[b, q, t] = np.where(np.isinf(top), -np.inf, np.where(np.isinf(top), 0, top) + np.log(
                    np.exp(x - np.where(np.isinf(top), 0, top)[:, None]).sum(1)))
    return torch.from_numpy(out).float()


def check(dev, B, Tq, Lmax, Hq, Hkv, modes, sink, window, lens=None, bm=None, seed=1):
    Q, K = tokens((B, Tq, Hq, 128), seed=seed), tokens((B, Lmax, Hkv, 128), seed=seed + 1)
    use = lens or [Lmax] * B
    LSE = row_lse(Q, K, modes, sink, window, use, bm)
    W, tol = key_weights_ref(Q, K, LSE, modes, sink, window, use, SCALE, bm)
    for b, L in enumerate(use):                     # whatever lies behind the sequence, and the rows before it
        K[b, L:] = float("nan")
        Q[b, : max(0, Tq - L)] = float("nan")
    ws = ea.key_weights_workspace(B, Tq, Lmax, Hq, Hkv, device=dev)
    w0 = torch.rand(B, Hkv, Lmax, generator=torch.Generator().manual_seed(seed))
    w = w0.to(dev)
    kw = dict(sink=sink, window=window, workspace=ws, block_mask=None if bm is None else torch.as_tensor(bm).to(dev),
              seqlens=None if lens is None else torch.tensor(lens, dtype=torch.int32, device=dev))
    args = (Q.to(dev), K.to(dev), LSE.to(dev), torch.tensor(modes, dtype=torch.uint8, device=dev))
    ea.ea_key_weights(*args, weights=w, **kw)
    once = torch.full_like(w, 0.25)
    ea.ea_key_weights(*args, weights=once, accumulate=False, **kw)
    check_no_device_error(ws)
    live = np.broadcast_to(np.arange(Lmax)[None, None] < np.array(use)[:, None, None], W.shape)
    got = once.cpu().numpy().astype(np.float64)
    assert (got[~live] == 0.25).all()
    assert (np.abs(got - W) <= tol)[live].all(), float((np.abs(got - W)[live] / tol[live]).max())
    both = w.cpu().numpy().astype(np.float64)
    s = w0.numpy().astype(np.float64)
    assert (both[~live] == s[~live]).all()
    assert (np.abs(both - (s + W)) <= tol + 2.0 ** -23 * (s + W))[live].all()
    return once


@pytest.mark.parametrize("S", [1, 2, 15, 16, 17, 127, 128, 129, 300, 1000])
def test_whole_prefill(dev, S):
    B, Hkv, g = 3, 3, 2
    bm = wl.block_mask(B, Hkv, S, density=0.3, seed=S).numpy()
    check(dev, B, S, S, Hkv * g, Hkv, all_modes(B, Hkv), 20, 150, bm=bm)


@pytest.mark.parametrize("Tq", [1, 3, 16, 33, 64, 65, 100, 128, 200, 513])
@pytest.mark.parametrize("g", [1, 4, 7])
def test_last_rows_of_ragged_sequences(dev, Tq, g):
    lens = [700, 0, 1, 64, 127, 129, 640, 513]
    B, Hkv, Lmax = len(lens), 3, 701
    bm = wl.block_mask(B, Hkv, Lmax, density=0.3, seed=Tq).numpy()
    bm[6] = 0                                       # block heads that keep nothing: LSE -inf
    check(dev, B, Tq, Lmax, Hkv * g, Hkv, all_modes(B, Hkv), 30, 77, lens, bm, seed=Tq)


@pytest.mark.parametrize("sink,window", [(0, 1), (0, 128), (1, 127), (128, 129), (200, 1), (1000, 1000), (64, 1 << 30)])
def test_streaming_borders(dev, sink, window):
    check(dev, 1, 520, 520, 4, 2, [[SSA, SSA]], sink, window, seed=sink)
    check(dev, 1, 40, 520, 4, 2, [[SSA, SSA]], sink, window, seed=sink + 1)


def test_group_of_many_heads(dev):
    check(dev, 1, 20, 200, 64, 1, [[FULL]], 0, 1)
    check(dev, 1, 200, 200, 20, 1, [[SSA]], 5, 50)


def test_prefill_lse_and_strided_views(dev):
    # the prefill's own LSE; an observation window as views of the prefill's tensors; one projection's slices
    B, S, Hq, Hkv, T = 2, 700, 8, 2, 64
    x = tokens((B, S, Hq + 2 * Hkv, 128), seed=3).to(dev)
    Q, K, V = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
    m = torch.tensor([[FULL, SSA], [SSA, FULL]], dtype=torch.uint8, device=dev)
    _, LSE = ea.ea_hybrid_attn_prefill(Q, K, V, m, sink=16, window=100)
    w = ea.ea_key_weights(Q, K, LSE, m, sink=16, window=100)
    W, tol = key_weights_ref(Q.cpu(), K.cpu(), LSE.cpu(), m.tolist(), 16, 100, [S] * B, SCALE)
    assert (np.abs(w.cpu().numpy() - W) <= tol).all()
    # every row's probabilities sum to 1: g * S in all, up to the prefill's LSE (1e-3 at most)
    assert abs(w.double().sum().item() / (B * Hq * S) - 1) < 1e-3
    w = ea.ea_key_weights(Q[:, -T:], K, LSE[:, :, -T:], m, sink=16, window=100)
    W, tol = key_weights_ref(Q[:, -T:].cpu(), K.cpu(), LSE[:, :, -T:].cpu(), m.tolist(), 16, 100, [S] * B, SCALE)
    assert (np.abs(w.cpu().numpy() - W) <= tol).all()


def test_shares_and_repeats_give_equal_bits(dev):
    # few key tiles: their queries are cut into shares that are joined in order
    B, S, Hq, Hkv = 1, 3000, 8, 1
    Q, K = tokens((B, S, Hq, 128), seed=5).to(dev), tokens((B, S, Hkv, 128), seed=6).to(dev)
    m = torch.zeros(1, 1, dtype=torch.uint8, device=dev)
    V = torch.zeros_like(K)
    _, LSE = ea.ea_hybrid_attn_prefill(Q, K, V, m, sink=0, window=1)
    ws = ea.key_weights_workspace(B, S, S, Hq, Hkv, device=dev)
    assert ws.numel() > 2 * 4 * S
    first = ea.ea_key_weights(Q, K, LSE, m, sink=0, window=1, workspace=ws)
    for _ in range(5):
        assert torch.equal(first, ea.ea_key_weights(Q, K, LSE, m, sink=0, window=1, workspace=ws))
    assert abs(first.double().sum().item() / (Hq * S) - 1) < 1e-3
    check_no_device_error(ws)


def test_bad_modes_and_lengths_are_reported(dev):
    Q, K = tokens((4, 10, 2, 128), seed=7).to(dev), tokens((4, 50, 1, 128), seed=8).to(dev)
    LSE = torch.zeros(4, 2, 10, device=dev)
    ws = ea.key_weights_workspace(4, 10, 50, 2, 1, device=dev)
    m = torch.tensor([[FULL], [9], [BLOCK], [FULL]], dtype=torch.uint8, device=dev)
    w = ea.ea_key_weights(Q, K, LSE, m, sink=0, window=1, workspace=ws, accumulate=False,
                          seqlens=torch.tensor([51, 50, 50, -3], dtype=torch.int32, device=dev))
    assert ea.ea_check_errors(ws) == 6
    assert (w == 0).all()
    good = ea.ea_key_weights(Q, K, LSE, torch.zeros_like(m), sink=0, window=1, workspace=ws)
    check_no_device_error(ws)
    assert (good > 0).all()


def test_captured_and_replayed(dev):
    B, T, L, Hq, Hkv = 2, 32, 500, 8, 2
    Q, K = tokens((B, T, Hq, 128), seed=9).to(dev), tokens((B, L, Hkv, 128), seed=10).to(dev)
    LSE = torch.full((B, Hq, T), 6.0, device=dev)
    sl = torch.tensor([500, 300], dtype=torch.int32, device=dev)
    m = torch.tensor([[FULL, SSA]] * B, dtype=torch.uint8, device=dev)
    ws = ea.key_weights_workspace(B, T, L, Hq, Hkv, device=dev)
    w, w2 = torch.zeros(B, Hkv, L, device=dev), torch.zeros(B, Hkv, L, device=dev)
    step = lambda out: ea.ea_key_weights(Q, K, LSE, m, sink=4, window=99, seqlens=sl, weights=out, workspace=ws)
    step(w)
    step(w2)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(w)
    Q.copy_(tokens((B, T, Hq, 128), seed=11))
    sl.copy_(torch.tensor([33, 499]))
    for _ in range(2):
        g.replay()
        step(w2)
    torch.cuda.synchronize()
    assert torch.equal(w, w2)
    check_no_device_error(ws)


@pytest.mark.parametrize("dtype", [E4M3, INT8])
def test_prefill_evict_and_decode_together(dev, dtype):
    # a prompt is prefilled; the weights of its last 64 queries choose which tokens of each head stay; those become an
    # 8-bit cache; tokens are appended and decoded, their weights accumulate; the cache is cut once more; each result
    # is compared with the plain form on the inputs that the step had
    B, S, Hq, Hkv, keep, sink, recent, steps = 2, 900, 8, 2, 300, 8, 100, 40
    g = Hq // Hkv
    Q, K, V = (t.to(dev) for t in wl.qkv(B, S, Hq, Hkv, 128, seed=12))
    m = torch.tensor([[FULL, SSA], [FULL, FULL]], dtype=torch.uint8, device=dev)
    modes = m.tolist()
    _, LSE = ea.ea_hybrid_attn_prefill(Q, K, V, m, sink=sink, window=100)
    w = ea.ea_key_weights(Q[:, -64:], K, LSE[:, :, -64:], m, sink=sink, window=100)
    W, tol = key_weights_ref(Q[:, -64:].cpu(), K.cpu(), LSE[:, :, -64:].cpu(), modes, sink, 100, [S] * B, SCALE)
    assert (np.abs(w.cpu().numpy() - W) <= tol).all()
    lens = torch.full((B,), S, dtype=torch.int32, device=dev)
    idx, n = ea.ea_evict_select(w, lens, keep=keep, sink=sink, recent=recent)
    want, _ = select_ref(w.cpu().numpy(), [S] * B, keep, sink, recent)
    np.testing.assert_array_equal(idx.cpu().numpy(), want)

    src = ea.KVCache(K, V)
    cache = ea.kv_cache(B, 512, Hkv, dtype=dtype, scale_block=32, device=dev)
    kw = torch.zeros(B, Hkv, 512, device=dev)
    ea.ea_cache_compact(src, cache, idx, n, weights=w, weights_out=kw)
    ref = dict(K=torch.zeros(B, 512, Hkv, 128, dtype=dtype), V=torch.zeros(B, 512, Hkv, 128, dtype=dtype),
               ks=torch.zeros(B, Hkv, 16), vs=torch.zeros(B, Hkv, 16), table=None, sb=32)
    at = torch.from_numpy(want).long().permute(0, 2, 1)[..., None].expand(-1, -1, -1, 128)
    write_ref(ref, K.cpu().gather(1, at), V.cpu().gather(1, at), [0] * B, [keep] * B)

    def same(h, c):
        for a, b in ((h.K, c["K"]), (h.V, c["V"])):
            assert torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8))
        for a, b in ((h.k_scale, c["ks"]), (h.v_scale, c["vs"])):
            assert torch.equal(a.cpu(), b)

    same(cache, ref)
    ws = ea.decode_q8_workspace(B, Hq, Hkv, 512, weights=True, device=dev)
    total = kw.double().cpu().numpy()
    slack = np.zeros_like(total)
    for t in range(steps):
        k1, v1 = tokens((B, 1, Hkv, 128), seed=300 + t), tokens((B, 1, Hkv, 128), seed=400 + t)
        q = tokens((B, Hq, 128), seed=500 + t)
        ea.ea_cache_write(cache, k1.to(dev), v1.to(dev), n)
        write_ref(ref, k1, v1, n.tolist(), [1] * B)
        n = n + 1
        O, L = ea.ea_hybrid_attn_decode_q8(q.to(dev), cache, n, m, sink=sink, window=recent, key_weights=kw, workspace=ws)
        if t % 13 == 0:
            same(cache, ref)
        Kr, Vr = logical(ref)
        Or, Lr, Wr, (tO, tL, tW) = decode_ref(q, Kr, Vr, value_scales(ref), n.tolist(), modes, sink, recent, SCALE)
        assert (np.abs(O.float().cpu().numpy() - Or) <= tO).all() and (np.abs(L.cpu().numpy() - Lr) <= tL).all()
        total += Wr
        slack += tW + 2.0 ** -23 * total
    assert (np.abs(kw.cpu().numpy() - total) <= slack).all()
    check_no_device_error(ws)
    idx, n2 = ea.ea_evict_select(kw, n, keep=200, sink=sink, recent=recent)
    want, _ = select_ref(kw.cpu().numpy(), n.tolist(), 200, sink, recent)
    np.testing.assert_array_equal(idx.cpu().numpy(), want)
    short = ea.kv_cache(B, 256, Hkv, dtype=dtype, scale_block=32, device=dev)
    ea.ea_cache_compact(cache, short, idx, n2)
    q = tokens((B, Hq, 128), seed=999)
    O, L = ea.ea_hybrid_attn_decode_q8(q.to(dev), short, n2, m, sink=sink, window=recent)
    got = {"K": short.K.cpu(), "V": short.V.cpu(), "ks": short.k_scale.cpu(), "vs": short.v_scale.cpu(), "table": None, "sb": 32}
    Ks, Vs = logical(got)
    at = np.transpose(want, (0, 2, 1))[..., None].astype(np.int64)
    Kr, Vr = logical(ref)
    if dtype == E4M3:
        # a token moves to a block of a larger or smaller scale: within e4m3's rounding (2^-4), or the block's smallest step
        np.testing.assert_allclose(Ks[:, :200], np.take_along_axis(Kr, np.broadcast_to(at, (B, 200, Hkv, 128)), 1), rtol=2.0 ** -4,
                                   atol=2.0 ** -10 * got["ks"].max().item())
    Or, Lr, _, (tO, tL, _) = decode_ref(q, Ks, Vs, value_scales(got), n2.tolist(), modes, sink, recent, SCALE)
    assert (np.abs(O.float().cpu().numpy() - Or) <= tO).all() and (np.abs(L.cpu().numpy() - Lr) <= tL).all()


@pytest.mark.parametrize("Tq,Hq", [(1, 32), (64, 32), (17, 8)])
def test_runs_of_key_tiles_that_share_one_query_tile(dev, Tq, Hq):
    # enough key tiles that an item takes several: the query tile and its LSE stay while keys pass; ragged lengths and
    # streaming heads (most of whose key tiles no row sees) between them; against the same formula in torch, float64
    B, Hkv, L, sink, window = 3, 8, 32768 + 77, 100, 300
    lens = [L, 20000, 129]
    Q, K = tokens((B, Tq, Hq, 128), seed=21).to(dev), tokens((B, L, Hkv, 128), seed=22).to(dev)
    LSE = (torch.rand(B, Hq, Tq, generator=torch.Generator().manual_seed(23)) + 12).to(dev)
    modes = [[(FULL, SSA)[(b + h) % 2] for h in range(Hkv)] for b in range(B)]
    ws = ea.key_weights_workspace(B, Tq, L, Hq, Hkv, device=dev)
    w = torch.full((B, Hkv, L), -1.0, device=dev)
    ea.ea_key_weights(Q, K, LSE, torch.tensor(modes, dtype=torch.uint8, device=dev), sink=sink, window=window,
                      seqlens=torch.tensor(lens, dtype=torch.int32, device=dev), weights=w, accumulate=False, workspace=ws)
    check_no_device_error(ws)
    g = Hq // Hkv
    for b, n in enumerate(lens):
        assert (w[b, :, n:] == -1).all()
        t = torch.arange(max(0, Tq - n), Tq, device=dev)
        i, j = (n - Tq + t)[:, None], torch.arange(n, device=dev)[None]
        for h in range(Hkv):
            keep = j <= i
            if modes[b][h] == SSA:
                keep = keep & ((j < sink) | (i - j < window))
            want, tol = torch.zeros(n, dtype=torch.float64, device=dev), torch.zeros(n, dtype=torch.float64, device=dev)
            for q in range(h * g, (h + 1) * g):
                x = Q[b, t, q].double() @ K[b, :n, h].double().T * SCALE
                d = 2.0 ** -16 * SCALE * (Q[b, t, q].double().abs() @ K[b, :n, h].double().abs().T) + 2.0 ** -21 * (x.abs() + 13)
                p = torch.where(keep, torch.exp(x - LSE[b, q, t].double()[:, None]), 0.0)
                want += p.sum(0)
                tol += (p * torch.expm1(d)).sum(0) + 2.0 ** -13 * p.sum(0) + 1e-37
            # (these LSE are not the rows' own: some sums lie above the largest float32, and are infinite there)
            got = w[b, h, :n].double()
            over = got.isinf() & (got > 0) & (want + tol > torch.finfo(torch.float32).max)
            assert (((got - want).abs() <= tol) | over).all()
