"""Attention of a tree of drafted tokens where its arithmetic or its bounds can go wrong:
depths out of range, drafted values of zero, values of any size in places that a row
does not keep, few kept keys, the widest windows."""
import math

import numpy as np
import pytest
import torch

import sparse_head_attention_gb300 as ea
from cache_reference import logical, make_cache, tokens, value_scales, write_ref
from gpu_helpers import bf16_half_ulp, check_no_device_error, gpu_device
from test_tree_attn_gpu import KEEP, handle, i32, inputs, out
from tree_reference import plan, random_tree

pytestmark = pytest.mark.gpu
E4M3, INT8, BF16 = torch.float8_e4m3fn, torch.int8, torch.bfloat16
FULL, SSA, BLOCK = ea.FULL, ea.SSA, ea.BLOCK
SCALE = 128 ** -0.5


@pytest.fixture(scope="module")
def dev():
    return gpu_device()


def unit(x):
    """What a drafted row's f16 numbers of an 8-bit cache's step stand for: the power of two that puts the row's largest
    finite magnitude into [2^14, 2^15), that magnitude taken as 2^-64 at least.  x float64 [..., 128]."""
    top = np.where(np.isfinite(x), np.abs(x), 0.0).max(-1)
    return 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(top, 2.0 ** -126))), -64) - 14)


def attend(Q, K, V, Kc, Vc, lens, n, depth, mask, modes, sink, window, bm=None, vscale=None, few=False):
    """The operator in 64 bits, over the keys that a row keeps alone, and how far it may be off:
      logits: 2^-17 of sum |q k| (128 fp32 terms), and 2^-17 for the exponent's multiply-add and exponential; over 8 bits q's
      elements are f16, off by 2^-36 of their row's largest, and a drafted key's by 2^-27 of its own row's (half of f16's least
      step, 2^-25, where the largest of rows within 2^12 of one another is at least 2^14), or of 2^-64;
      probabilities: bf16, half a step 2^-8; `few`: in two parts, the second less than 2^-7 of it, half a step 2^-15; f16 (8-bit caches) 2^-11, and 2^-25 where below
      2^-14, in units of 2^-7 of the largest kept weight times unit (vscale: of the cache's V), a tile's units standing for
      the largest within 2^12: at most 2^-20 max(u) sum |v| / u, u the units of the kept keys alone; a drafted value as a
      drafted key;
      sums and joins: 2^-16.
    The output's own rounding, half a bf16 step, is left to the caller."""
    B, T, Hq, D = Q.shape
    Hkv = K.shape[2]
    g = Hq // Hkv
    O, LSE = np.zeros((B, T, Hq, D)), np.full((B, Hq, T), -np.inf)
    tO, tL = np.zeros((B, T, Hq, D)), np.zeros((B, Hq, T))
    for b in range(B):
        L, nb = lens[b], n[b]
        pos = L + depth[b, :nb].astype(np.int64)
        at = np.concatenate([np.arange(L), pos])
        up = ((mask[b, :nb].view(np.uint32)[:, :, None] >> np.arange(32, dtype=np.uint32)) & 1).reshape(nb, 128)[:, :nb].astype(bool)
        for h in range(Hkv):
            k, v = np.concatenate([Kc[b, :L, h], K[b, :nb, h]]), np.concatenate([Vc[b, :L, h], V[b, :nb, h]])
            keep = np.concatenate([np.ones((nb, L), bool), up], 1)
            if modes[b][h] == SSA:
                keep &= (at[None] < sink) | (pos[:, None] - at[None] < window)
            elif modes[b][h] == BLOCK:
                keep &= bm[b, h][pos // 128][:, at // 128] != 0
            for t in range(nb):
                j = np.flatnonzero(keep[t])
                if not len(j):
                    continue
                q, hs = Q[b, t, h * g : (h + 1) * g], slice(h * g, (h + 1) * g)
                x = q @ k[j].T * SCALE
                e = (np.abs(q) @ np.abs(k[j]).T * SCALE).max(1) * 2.0 ** -17 + 2.0 ** -17
                if vscale is not None:
                    own = j[j >= L]
                    e += 2.0 ** -36 * np.abs(q).max(1) * np.abs(k[j]).sum(1).max() * SCALE
                    if len(own):
                        e += 2.0 ** -27 * np.abs(q).sum(1) * np.maximum(np.abs(k[own]).max(), 2.0 ** -64) * SCALE
                top = x.max(1, keepdims=True)
                p = np.exp(x - top)
                s = p.sum(1, keepdims=True)
                p /= s
                O[b, t, hs], LSE[b, hs, t] = p @ v[j], (top + np.log(s))[:, 0]
                part = 2.0 ** -11 if vscale is not None else 2.0 ** -15 if few else 2.0 ** -8
                tO[b, t, hs] = (p @ np.abs(v[j])) * (part + 2.0 ** -16 + 2 * e[:, None])
                if vscale is not None:
                    u = np.concatenate([vscale[b, :L, h] / 64, unit(v[L:])])[j]
                    tO[b, t, hs] += 2.0 ** -20 * u.max() * (np.abs(v[j]) / u[:, None]).sum(0)
                    if len(own):
                        tO[b, t, hs] += 2.0 ** -27 * np.maximum(np.abs(v[own]).max(), 2.0 ** -64)
                tL[b, hs, t] = e + np.abs(LSE[b, hs, t]) * 2.0 ** -20
    return O, LSE, tO, tL


def check(dev, c, Q, K, V, lens, n, parents, modes, sink=16, window=100, bm=None, few=False, rows=None):
    """One call against the above; rows: the (sequence, node) pairs that are compared (all)."""
    B, T, Hq, _ = Q.shape
    depth, mask = plan(parents, n)
    q8 = c["ks"] is not None
    ref = attend(*(x.double().numpy() for x in (Q, K, V)), *logical(c), lens, n, depth, mask, modes, sink, window, bm,
                 value_scales(c) if q8 else None, few)
    h = handle(c, dev)
    ws = ea.tree_workspace(B, T, Hq, K.shape[2], h.capacity, device=dev)
    O, LSE = out(B, T, Hq, dev)
    ea.ea_hybrid_attn_tree(*(x.to(dev) for x in (Q, K, V)), h, i32(lens, dev), i32(depth, dev), i32(mask, dev),
                           torch.tensor(modes, dtype=torch.uint8, device=dev), sink=sink, window=window, n_nodes=i32(n, dev),
                           block_mask=None if bm is None else torch.as_tensor(bm).to(dev), O=O, LSE=LSE, workspace=ws)
    check_no_device_error(ws)
    O, LSE = O.float().cpu().numpy().astype(np.float64), LSE.cpu().numpy().astype(np.float64)
    for b, t in rows or [(b, t) for b in range(B) for t in range(n[b])]:
        o, l = O[b, t], LSE[b, :, t]
        assert np.array_equal(np.isneginf(l), np.isneginf(ref[1][b, :, t])), (b, t, "empty rows")
        some = ~np.isneginf(l)
        bad = ~(np.abs(l - ref[1][b, :, t]) <= ref[3][b, :, t]) & some
        assert not bad.any(), (b, t, "LSE", l[bad][:4], ref[1][b, :, t][bad][:4])
        err = np.abs(o - ref[0][b, t])
        bad = ~(err <= bf16_half_ulp(np.maximum(np.abs(o), np.abs(ref[0][b, t]))) + ref[2][b, t] + 2.0 ** -130)
        assert not bad.any(), (b, t, "O", int(bad.sum()), o[bad][:4], ref[0][b, t][bad][:4], err[bad].max())


def _depths(dev, mode, L, sink, window, bm, given, nearest):
    """The call with the depths `given` reports them and equals the one with the nearest valid ones, whose error word is clear."""
    B, T, Hq, Hkv = 1, 6, 4, 1
    Q, K, V = (x.to(dev) for x in inputs(B, T, Hq, Hkv, 5))
    _, mask = plan(random_tree(B, T, 0, "chain"), [T])
    h = handle(make_cache(B, 512, Hkv, BF16, 64, 0, 7), dev)
    ws = ea.tree_workspace(B, T, Hq, Hkv, 512, device=dev)
    got = []
    for d, status in ((given, 6), (nearest, 0)):
        got.append(ea.ea_hybrid_attn_tree(Q, K, V, h, i32([L], dev), i32([d], dev), i32(mask, dev), torch.tensor([[mode]], dtype=torch.uint8, device=dev),
                                          sink=sink, window=window, block_mask=None if bm is None else torch.as_tensor(bm).to(dev), workspace=ws))
        assert ea.ea_check_errors(ws) == status
    for a, b in zip(*got):
        assert torch.equal(a, b)


def _block_rows():
    bm = np.zeros((1, 1, 4, 4), np.uint8)
    bm[0, 0, 1, 1] = bm[0, 0, 2, 2] = bm[0, 0, 2, 0] = 1
    return bm


def test_depths_just_outside_their_range(dev):
    """An ancestor's depth counts as the nearest valid one, as a node's own does."""
    # -1 would lie below the sink's end, 0 does not
    _depths(dev, SSA, 100, 100, 2, None, [-1, 1, 2, 3, 4, 5], [0, 1, 2, 3, 4, 5])
    _depths(dev, SSA, 100, 0, 2, None, [0, 1, 2, 3, 6, 5], [0, 1, 2, 3, 5, 5])
    # positions 250 to 255: block 1, whose row keeps it; 256 would be in block 2
    _depths(dev, BLOCK, 250, 0, 1, _block_rows(), [-1, 1, 2, 3, 4, 5], [0, 1, 2, 3, 4, 5])
    _depths(dev, BLOCK, 250, 0, 1, _block_rows(), [0, 1, 6, 3, 4, 5], [0, 1, 5, 3, 4, 5])


@pytest.mark.parametrize("far", [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 200, -1000000])
def test_depths_far_outside_their_range(dev, far):
    """No sum with such a depth leaves 32 bits, nor the block mask."""
    near = 5 if far > 0 else 0
    _depths(dev, SSA, 100, 100, 2, None, [0, far, 2, 3, 4, 5], [0, near, 2, 3, 4, 5])
    _depths(dev, BLOCK, 250, 0, 1, _block_rows(), [0, far, 2, 3, 4, 5], [0, near, 2, 3, 4, 5])


@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("value", [0.0, 2.0 ** -120, math.inf])
def test_drafted_values_of_nothing(dev, dtype, value):
    """One head's drafted values are all zero (or next to nothing, or, on a node that no other keeps, infinite): the sums stay
    finite, over no cache, over a tile of it, and where a range of tiles begins or ends at the tree's own."""
    T, Hq, Hkv = 6, 8, 2
    p = np.array([[-1, 0, 1, 1, 0, 4]], np.int32)
    for lens in ([0, 100], [128, 1], [20000, 20100], [20161, 20050], [3000, 2900]):
        B = len(lens)
        Q, K, V = inputs(B, T, Hq, Hkv, 3)
        V[:, :, 1] = 0.0 if math.isinf(value) else value
        if math.isinf(value):
            V[:, 5, 1, 7] = value
        rows = [(b, t) for b in range(B) for t in range(T) if not (math.isinf(value) and t == 5)]
        check(dev, make_cache(B, max(lens) + 64, Hkv, dtype, 64, 0, 5), Q, K, V, lens, [T] * B, p.repeat(B, 0), [[FULL] * Hkv] * B, rows=rows)


@pytest.mark.parametrize("dtype", [E4M3, INT8])
def test_some_rows_of_zero(dev, dtype):
    """Blocks of zeros in the cache and drafted rows of zero among others."""
    B, T, Hq, Hkv, lens = 2, 6, 8, 2, [500, 33]
    Q, K, V = inputs(B, T, Hq, Hkv, 3)
    c = make_cache(B, 512, Hkv, dtype, 16, 0, 5)
    zero = torch.zeros(B, 48, Hkv, 128, dtype=BF16)
    for s in (0, 144, 400):
        write_ref(c, zero, tokens((B, 48, Hkv, 128), s) if s == 144 else zero, [s] * B, [48] * B)
    K[:, 1], V[:, 1], V[:, 4] = 0.0, 0.0, 0.0
    check(dev, c, Q, K, V, lens, [T] * B, random_tree(B, T, 1), [[FULL, SSA]] * B)


@pytest.mark.parametrize("dtype,sb,page", [(E4M3, 16, 0), (INT8, 16, 64), (BF16, 64, 0)])
@pytest.mark.parametrize("size", [10, 14, 40, 90, -40])
def test_values_of_another_size_in_places_not_kept(dev, dtype, sb, page, size):
    """Keys and values 2^size times the others', in rows that no node keeps and on a node that keeps its own alone: the others'
    results are as if they were not there.  (-40: the others are the large ones.)"""
    B, T, Hq, Hkv, lens = 2, 6, 8, 2, [500, 0]
    p = np.array([[-1, 0, 1, 1, 0, 4]] * B, np.int32)
    Q, K, V = inputs(B, T, Hq, Hkv, 3)
    c = make_cache(B, 512, Hkv, dtype, sb, page, 4)
    big, small = 2.0 ** max(size, 0), 2.0 ** min(size, 0)
    # a window's end inside a tile, a sink's end inside another: the rows between are kept by none
    kn, vn = tokens((B, 512, Hkv, 128), 50).float(), tokens((B, 512, Hkv, 128), 51).float()
    write_ref(c, (kn * small).to(BF16), (vn * small).to(BF16), [0] * B, [512] * B)
    for s in (256, 16):
        write_ref(c, (kn[:, :32] * big).to(BF16), (vn[:, :32] * big).to(BF16), [s] * B, [32] * B)
    for x in (K, V):
        x.mul_(small)
        x[:, 3] *= big / small
    rows = [(b, t) for b in range(B) for t in range(T) if t != 3]
    check(dev, c, (Q.float() / small).clamp(max=2.0 ** 100).to(BF16) if size < 0 else Q, K, V, lens, [T] * B, p, [[SSA, SSA], [FULL, SSA]], sink=10, window=200, rows=rows)


@pytest.mark.parametrize("dtype", [E4M3, INT8])
def test_large_values_kept_with_others(dev, dtype):
    """Blocks of different scales in a tile and drafted rows of different size, all kept: each within the bits of its own weight."""
    B, T, Hq, Hkv, lens = 2, 9, 4, 1, [300, 40]
    Q, K, V = inputs(B, T, Hq, Hkv, 3)
    c = make_cache(B, 320, Hkv, dtype, 16, 0, 4)
    r = np.random.RandomState(0)
    for s in range(0, 320, 16):
        x = [tokens((B, 16, Hkv, 128), 60 + s + i).float() * 2.0 ** float(r.randint(-6, 7)) * (1.0 if i else 0.25) for i in range(2)]
        write_ref(c, *(y.to(BF16) for y in x), [s] * B, [16] * B)
    V *= torch.from_numpy(2.0 ** r.randint(-6, 7, (B, T, 1, 1))).to(BF16)
    check(dev, c, Q, K, V, lens, [T] * B, random_tree(B, T, 2), [[FULL]] * B)


@pytest.mark.parametrize("dtype", [E4M3, INT8])
def test_single_token_is_the_8bit_decode(dev, dtype):
    """T = 1 equals the 8-bit decode over the cache with that token in it, outputs and log-sum-exps, where the token's numbers
    are 8-bit ones at the scale of the block that it begins."""
    B, Hq, Hkv, L = 3, 8, 2, [192, 64, 128]
    c = make_cache(B, 256, Hkv, dtype, 64, 0, 7)
    Kc, Vc = logical(c)
    Q = inputs(B, 1, Hq, Hkv, 1)[0]
    K, V = (torch.from_numpy(np.stack([x[b, L[b] - 1][None] for b in range(B)])).to(BF16) for x in (Kc, Vc))
    depth, mask = plan(np.full((B, 1), -1, np.int32), [1] * B)
    modes = [[FULL, SSA]] * B
    ref = attend(*(x.double().numpy() for x in (Q, K, V)), Kc, Vc, L, [1] * B, depth, mask, modes, 4, 30, vscale=value_scales(c))
    h = handle(c, dev)
    m = torch.tensor(modes, dtype=torch.uint8, device=dev)
    O, LSE = ea.ea_hybrid_attn_tree(Q.to(dev), K.to(dev), V.to(dev), h, i32(L, dev), i32(depth, dev), i32(mask, dev), m, sink=4, window=30)
    ea.ea_cache_write(h, K.to(dev), V.to(dev), start=i32(L, dev))
    o, lse = ea.ea_hybrid_attn_decode_q8(Q[:, 0].to(dev), h, i32(np.array(L) + 1, dev), m, sink=4, window=30)
    a, b = O[:, 0].double().cpu().numpy(), o.double().cpu().numpy()
    assert (np.abs(a - b) <= 2 * (bf16_half_ulp(np.maximum(np.abs(a), np.abs(b))) + ref[2][:, 0])).all()
    assert (np.abs(LSE[:, :, 0].double().cpu().numpy() - lse.double().cpu().numpy()) <= 2 * ref[3][:, :, 0]).all()


@pytest.mark.parametrize("page", [0, 64])
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 8, 2), (5, 4, 2), (24, 16, 2)])
def test_few_kept_keys(dev, T, Hq, Hkv, page):
    """bf16 caches, rows that keep at most 512 keys of the cache: probabilities in two parts, as the decode has them, so that
    little but the output's own rounding is left.  Values of one sign and a large offset, which each probability's error enters whole."""
    lens = [0, 2, 5, 60, 130, 300, 500, 5000]
    B = len(lens)
    c = make_cache(B, 5056, Hkv, BF16, 64, page, 3)
    g = torch.Generator().manual_seed(1)
    sign = torch.where(torch.rand(128, generator=g) < 0.5, -1.0, 1.0)
    offset = lambda *s: ((2.2 + 1.6 * torch.rand(*s, 128, generator=g)) * sign).to(BF16)  # noqa: E731
    write_ref(c, tokens((B, 5056, Hkv, 128), 9), offset(B, 5056, Hkv), [0] * B, [5056] * B)
    Q, K, _ = inputs(B, T, Hq, Hkv, 3)
    modes = [[FULL, SSA]] * (B - 1) + [[SSA, SSA]]
    check(dev, c, Q, K, offset(B, T, Hkv), lens, [T] * B, random_tree(B, T, 4, "chain" if T == 24 else "tree"), modes, sink=16, window=128, few=True)


def test_infinite_values_over_few_keys(dev):
    """An infinity among values that all rows keep stays one, whatever its probability's parts are."""
    B, T, Hq, lens = 2, 4, 4, [64, 300]
    Q, K, V = inputs(B, T, Hq, 1, 3)
    c = make_cache(B, 320, 1, BF16, 64, 0, 2)
    c["K"][:] = 0.0                                       # equal weights: powers of two, or not
    K.zero_()
    c["V"][0, 5, 0, 17], c["V"][1, 7, 0, 19] = math.inf, -math.inf
    depth, mask = (i32(x, dev) for x in plan(random_tree(B, T, 3, "chain"), [T] * B))
    O, _ = ea.ea_hybrid_attn_tree(*(x.to(dev) for x in (Q, K, V)), handle(c, dev), i32(lens, dev), depth, mask,
                                  torch.zeros(B, 1, dtype=torch.uint8, device=dev), sink=0, window=1)
    assert torch.isposinf(O[0, :, :, 17]).all() and torch.isneginf(O[1, :, :, 19]).all()
    O[0, :, :, 17], O[1, :, :, 19] = 0.0, 0.0
    assert torch.isfinite(O).all()


@pytest.mark.parametrize("dtype", [BF16, INT8])
def test_the_widest_window_and_sink(dev, dtype):
    """Windows and sinks up to 2^31 - 1 keep what any larger than the cache keeps."""
    B, T, Hq = 3, 20, 4
    Q, K, V = (x.to(dev) for x in inputs(B, T, Hq, 1, 2))
    h = handle(make_cache(B, 320, 1, dtype, 64, 0, 1), dev)
    depth, mask = (i32(x, dev) for x in plan(random_tree(B, T, 3, "chain"), [T] * B))
    m = torch.full((B, 1), SSA, dtype=torch.uint8, device=dev)
    call = lambda s, w: ea.ea_hybrid_attn_tree(Q, K, V, h, i32([300, 0, 1], dev), depth, mask, m, sink=s, window=w)  # noqa: E731
    ref = call(0, 1000)
    for s, w in ((0, 2 ** 31 - 1), (2 ** 31 - 1, 1), (2 ** 31 - 1, 2 ** 31 - 1), (0, 2 ** 30)):
        got = call(s, w)
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


