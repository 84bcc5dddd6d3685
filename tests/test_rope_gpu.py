"""Rotation by position, alone and on the way into a cache, against plain forms in 64
bits: both pairings, partial rotation, far and negative positions, strides, formats,
pages, blocks begun before, gathered rows, and what must stay as it was."""
import numpy as np
import pytest
import torch

import sparse_head_attention_gb300 as ea
from cache_reference import block_scale, capacity, make_cache, rows_of, tokens
from gpu_helpers import check_no_device_error, gpu_device
from tree_reference import inv_freq, rotate, rotate_error

pytestmark = pytest.mark.gpu
E4M3, INT8, BF16 = torch.float8_e4m3fn, torch.int8, torch.bfloat16
KEEP = 7.5                                            # what an output row that must stay holds


@pytest.fixture(scope="module")
def dev():
    return gpu_device()


def near_bf16(got, want, err, what):
    """bf16 rounding: half a step, 2^-8 relative; err: the fp32 value's own."""
    got = got.float().cpu().numpy().astype(np.float64)
    tol = np.abs(want) * 2.0 ** -8 + 1.01 * err + 2.0 ** -133
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])


@pytest.mark.parametrize("rot,interleaved,scale", [(128, False, 1.0), (128, True, 1.0), (64, False, 1.0), (64, True, 0.5),
                                                   (16, False, 1.0), (96, True, 1.0), (112, False, 1.25)])
@pytest.mark.parametrize("B,T,Hq,Hkv", [(1, 1, 1, 1), (3, 17, 10, 2), (2, 40, 5, 1)])
def test_rope(dev, rot, interleaved, scale, B, T, Hq, Hkv):
    Q, K = tokens((B, T, Hq, 128), 1), tokens((B, T, Hkv, 128), 2)
    f = inv_freq(rot)
    r = np.random.RandomState(3)
    pos = r.randint(0, 1 << 20, (B, T)).astype(np.int32)
    pos.flat[0] = 0
    pos.flat[-1] = 2 ** 31 - 1
    if T > 2:
        pos[0, 1], pos[0, 2] = -5, -2 ** 31
    n = [T, T - 3, 0][:B] if T > 3 else [T] * B
    ws = ea.cache_workspace(dev)
    nd = torch.tensor(n, dtype=torch.int32, device=dev)
    fd, pd = torch.from_numpy(f).to(dev), torch.from_numpy(pos).to(dev)
    qo, ko = (torch.full(x.shape, KEEP, dtype=BF16, device=dev) for x in (Q, K))
    ea.ea_rope(Q.to(dev), K.to(dev), pd, fd, n_new=nd, interleaved=interleaved, rope_scale=scale, Q_out=qo, K_out=ko, workspace=ws)
    check_no_device_error(ws)
    for x, o, nm in ((Q, qo, "Q"), (K, ko, "K")):
        for b in range(B):
            v = x[b, : n[b]].double().numpy()
            near_bf16(o[b, : n[b]], rotate(v, pos[b, : n[b]], f, interleaved, scale), rotate_error(v, f, interleaved, scale), nm)
            assert (o[b, n[b] :].float() == KEEP).all(), nm
            assert torch.equal(o[b, : n[b], :, rot:].cpu(), x[b, : n[b], :, rot:])
    # in place, one of the two alone, on another stream: the same bits
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    qi = Q.to(dev)
    torch.cuda.synchronize()
    a, none = ea.ea_rope(qi, None, pd, fd, n_new=nd, interleaved=interleaved, rope_scale=scale, Q_out=qi, stream=s)
    torch.cuda.synchronize()
    assert none is None and a is qi
    for b in range(B):
        assert torch.equal(qi[b, : n[b]], qo[b, : n[b]]) and torch.equal(qi[b, n[b] :].cpu(), Q[b, n[b] :])
    _, ki = ea.ea_rope(None, K.to(dev), pd, fd, interleaved=interleaved, rope_scale=scale)
    for b in range(B):
        assert torch.equal(ki[b, : n[b]], ko[b, : n[b]])


def test_rope_strided_views(dev):
    """Queries and keys as parts of one projection's output."""
    B, T, Hq, Hkv = 2, 33, 6, 2
    qkv = tokens((B, T, Hq + 2 * Hkv, 128), 5).to(dev)
    q, k = qkv[:, :, :Hq], qkv[:, :, Hq : Hq + Hkv]
    pos = torch.arange(B * T, dtype=torch.int32, device=dev).view(B, T)
    f = torch.from_numpy(inv_freq(128)).to(dev)
    out = torch.empty(T, B, Hq, 128, dtype=BF16, device=dev).transpose(0, 1)
    a, b = ea.ea_rope(q, k, pos, f, Q_out=out)
    c, d = ea.ea_rope(q.contiguous(), k.contiguous(), pos, f)
    assert a is out and torch.equal(a, c) and torch.equal(b, d)


def test_rope_bad_count_and_frequency(dev):
    x = tokens((2, 4, 1, 128), 6).to(dev)
    pos = torch.zeros(2, 4, dtype=torch.int32, device=dev)
    pos[1] = 3
    f = torch.from_numpy(inv_freq(16)).to(dev)
    f[3], f[4], f[5] = float("inf"), 2.0 ** 24, float("nan")
    ws = ea.cache_workspace(dev)
    out = torch.full_like(x, KEEP)
    ea.ea_rope(x, None, pos, f, n_new=torch.tensor([5, 4], dtype=torch.int32, device=dev), Q_out=out, workspace=ws)
    assert ea.ea_check_errors(ws) == 6 and ea.ea_check_errors(ws) == 0
    assert (out[0].float() == KEEP).all()
    bad = torch.isnan(out[1, 0, 0].float()).cpu().numpy()
    assert sorted(np.flatnonzero(bad)) == [3, 4, 5, 11, 12, 13]
    # the largest frequency below the limit, against whole numbers of 1 / 2 pi
    f2 = np.full(8, np.nextafter(np.float32(2.0 ** 24), np.float32(0)), np.float32)
    f2[1], f2[2], f2[3] = np.float32(1e-30), np.float32(2.0 ** -149), np.float32(-0.75)
    y = x[1:2].clone()
    o, _ = ea.ea_rope(y, None, pos[1:2], torch.from_numpy(f2).to(dev))
    v = y[0].double().cpu().numpy()
    near_bf16(o[0], rotate(v, [3] * 4, f2, False), rotate_error(v, f2, False), "f")


def handle(c, dev):
    t = {k: None if v is None else v.to(dev) for k, v in c.items() if k in ("K", "V", "ks", "vs", "table")}
    return ea.KVCache(t["K"], t["V"], t["ks"], t["vs"], scale_block=c["sb"], block_table=t["table"])


def half_step(x, s, dtype):
    """Half the distance of the codes around x, times their scale s."""
    if dtype == INT8:
        return np.full_like(x, 0.5 * s)
    e = np.floor(np.log2(np.maximum(np.abs(x) / s, 2.0 ** -6)))
    return 2.0 ** (e - 4) * s


def check_append(dev, dtype, sb, page, Hkv, T, start, n, rows=None, positions=None, rot=128, interleaved=False, Hq=0, seed=0, cap=None):
    B = len(start)
    cap = cap or -(-(max(s + k for s, k in zip(start, n)) + 40) // 256) * 256
    c = make_cache(B, cap, Hkv, dtype, sb, page, seed)
    cap = capacity(c)
    K, V = tokens((B, T, Hkv, 128), seed + 1), tokens((B, T, Hkv, 128), seed + 2)
    Q = tokens((B, T, Hq, 128), seed + 3) if Hq else None
    f = inv_freq(rot)
    h = handle(c, dev)
    ws = ea.cache_workspace(dev)
    i32 = lambda v: None if v is None else torch.tensor(np.asarray(v), dtype=torch.int32, device=dev)  # noqa: E731
    q = ea.ea_cache_write_rope(h, K.to(dev), V.to(dev), torch.from_numpy(f).to(dev), Q=None if Q is None else Q.to(dev), start=i32(start),
                               n_new=i32(n), rows=i32(rows), positions=i32(positions), interleaved=interleaved,
                               Q_out=None if Q is None else torch.full(Q.shape, KEEP, dtype=BF16, device=dev), workspace=ws)
    check_no_device_error(ws)
    got = dict(K=h.K.cpu(), V=h.V.cpu(), ks=None if dtype == BF16 else h.k_scale.cpu(), vs=None if dtype == BF16 else h.v_scale.cpu())
    touched = {kv: torch.zeros(c[kv].shape[:2], dtype=torch.bool) for kv in "KV"}
    scaled = {kv: None if dtype == BF16 else torch.zeros_like(c["ks"], dtype=torch.bool) for kv in "KV"}
    for b in range(B):
        idx = [int(rows[b][i]) for i in range(n[b])] if rows is not None else list(range(n[b]))
        pos = [int(positions[b][t]) for t in idx] if positions is not None else [start[b] + i for i in range(n[b])]
        for kv, x in (("K", K), ("V", V)):
            v = x[b, idx].double().numpy().reshape(n[b], Hkv, 128)
            err = rotate_error(v, f, interleaved) if kv == "K" else np.zeros_like(v)
            w = rotate(v, pos, f, interleaved) if kv == "K" else v
            p, end = start[b], start[b] + n[b]
            step = sb if dtype != BF16 else 1
            while p < end:
                p0 = p // step * step
                stop = min(p0 + step, end)
                o, r = rows_of(c, b, p0)
                new, e = w[p - start[b] : stop - start[b]], err[p - start[b] : stop - start[b]]
                if dtype == BF16:
                    near_bf16(got[kv][o, r : r + 1], new, e, kv)
                    touched[kv][o, r] = True
                    p = stop
                    continue
                j, m = r // sb, p - p0
                sc = "ks" if kv == "K" else "vs"
                for hh in range(Hkv):
                    s = float(got[sc][o, hh, j])
                    was = float(c[sc][o, hh, j]) if m else 0.0
                    big = np.abs(new[:, hh]).max()
                    # the rotated value is off by a few 2^-24: a largest value that near a border may fall to either side
                    ok = {max(was, block_scale(big * (1 + u), dtype)) for u in (-2.0 ** -20, 0.0, 2.0 ** -20)}
                    assert s in ok, (kv, b, p, hh, s, ok)
                    code = got[kv][o, r + m : r + m + len(new), hh].float().numpy().astype(np.float64)
                    tol = half_step(new[:, hh], s, dtype) + 1.01 * e[:, hh]
                    assert (np.abs(code * s - new[:, hh]) <= tol * (1 + 2.0 ** -20)).all(), (kv, b, p, hh)
                    if m:                               # the tokens before: the same codes, or rounded to the grown scale
                        old = c[kv][o, r : r + m, hh].float().numpy().astype(np.float64) * was
                        now = got[kv][o, r : r + m, hh].float().numpy().astype(np.float64) * s
                        tol = half_step(old, s, dtype) if s != was else np.zeros_like(old)
                        assert (np.abs(now - old) <= tol).all(), (kv, b, p, hh)
                touched[kv][o, r : r + m + len(new)] = True
                scaled[kv][o, :, j] = True
                p = stop
    for kv, sc in (("K", "ks"), ("V", "vs")):
        bits = (lambda t: t.view(torch.int16)) if dtype == BF16 else (lambda t: t.view(torch.uint8))
        same = bits(got[kv]) == bits(c[kv])
        assert same[~touched[kv]].all(), kv
        if dtype != BF16:
            assert (got[sc] == c[sc])[~scaled[kv]].all(), sc
    if Hq:
        for b in range(B):
            pos = positions[b][: n[b]] if positions is not None else start[b] + np.arange(n[b])
            v = Q[b, : n[b]].double().numpy()
            near_bf16(q[b, : n[b]], rotate(v, pos, f, interleaved), rotate_error(v, f, interleaved), "Q")
            assert (q[b, n[b] :].float() == KEEP).all()
    else:
        assert q is None


FORMATS = [(BF16, 64, 0), (BF16, 64, 64), (E4M3, 64, 0), (E4M3, 16, 128), (INT8, 32, 64), (INT8, 128, 0)]


@pytest.mark.parametrize("dtype,sb,page", FORMATS)
def test_append(dev, dtype, sb, page):
    # fresh, inside a block, across blocks and pages, nothing, one token
    check_append(dev, dtype, sb, page, 2, 150, [0, 37, 250, 100, 63], [150, 149, 70, 0, 1], Hq=6)
    check_append(dev, dtype, sb, page, 1, 1, [5, 0, 64], [1, 1, 1], Hq=8, rot=64, interleaved=True, seed=9)


@pytest.mark.parametrize("dtype,sb,page", FORMATS)
def test_append_accepted_rows(dev, dtype, sb, page):
    r = np.random.RandomState(4)
    rows = np.stack([r.permutation(24) for _ in range(3)])
    rows[1, 1] = rows[1, 0]                              # the same row twice
    check_append(dev, dtype, sb, page, 3, 24, [100, 7, 61], [5, 24, 0], rows=rows, seed=2)
    pos = r.randint(0, 1 << 21, (3, 24))
    check_append(dev, dtype, sb, page, 3, 24, [100, 7, 61], [5, 24, 2], rows=rows, positions=pos, seed=3, rot=96, interleaved=True)


@pytest.mark.parametrize("dtype,sb,page", [(BF16, 64, 0), (E4M3, 32, 64)])
def test_append_positions_apart_from_rows(dev, dtype, sb, page):
    """After an eviction a token's position is not its row in the cache."""
    pos = np.arange(30)[None] + np.array([[1000000], [5]])
    check_append(dev, dtype, sb, page, 2, 30, [64, 90], [30, 11], positions=pos, Hq=4)


@pytest.mark.parametrize("dtype,sb,page", [(E4M3, 64, 0), (INT8, 128, 128), (E4M3, 32, 64), (BF16, 64, 64)])
def test_append_few_tokens_into_begun_blocks(dev, dtype, sb, page):
    # up to 16: whole blocks of rows before them, a block's end among them, none
    check_append(dev, dtype, sb, page, 3, 16, [0, 37, 120, 127, 250, 63], [16, 16, 16, 1, 11, 0], Hq=40, seed=30)
    check_append(dev, dtype, sb, page, 9, 3, [126, 31, 64], [3, 2, 3], Hq=18, seed=31)


@pytest.mark.parametrize("dtype,sb", [(E4M3, 64), (INT8, 128), (INT8, 32)])
def test_append_long_with_queries(dev, dtype, sb):
    """Many queries beside an 8-bit cache: the bits of the rotation alone and of the append alone."""
    B, T, Hq, Hkv, cap = 2, 2500, 16, 2, 2816
    Q, K, V = (tokens((B, T, h, 128), 20 + i).to(dev) for i, h in enumerate((Hq, Hkv, Hkv)))
    f = torch.from_numpy(inv_freq(128)).to(dev)
    start, n = (torch.tensor(v, dtype=torch.int32, device=dev) for v in ([0, 77], [2500, 2311]))
    pos = start[:, None] + torch.arange(T, dtype=torch.int32, device=dev)
    a, b = (ea.kv_cache(B, cap, Hkv, dtype=dtype, scale_block=sb, device=dev) for _ in range(2))
    out, alone = (torch.full(Q.shape, KEEP, dtype=BF16, device=dev) for _ in range(2))
    ws = ea.cache_workspace(dev)
    ea.ea_cache_write_rope(a, K, V, f, Q=Q, Q_out=out, start=start, n_new=n, workspace=ws)
    ea.ea_cache_write_rope(b, K, V, f, start=start, n_new=n, workspace=ws)
    ea.ea_rope(Q, None, pos, f, n_new=n, Q_out=alone, workspace=ws)
    check_no_device_error(ws)
    assert torch.equal(out.view(torch.int16), alone.view(torch.int16))
    assert (out[1, 2311:].float() == KEEP).all()
    for x, y in ((a.K, b.K), (a.V, b.V)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert torch.equal(a.k_scale, b.k_scale) and torch.equal(a.v_scale, b.v_scale)


def test_append_equals_rope_then_write(dev):
    """A bf16 cache holds the bits that ea_rope gives."""
    B, T, Hkv = 2, 20, 4
    K, V = tokens((B, T, Hkv, 128), 1).to(dev), tokens((B, T, Hkv, 128), 2).to(dev)
    f = torch.from_numpy(inv_freq(128)).to(dev)
    start = torch.tensor([3, 40], dtype=torch.int32, device=dev)
    pos = start[:, None] + torch.arange(T, dtype=torch.int32, device=dev)
    a, b = (ea.kv_cache(B, 128, Hkv, dtype=BF16, device=dev) for _ in range(2))
    ea.ea_cache_write_rope(a, K, V, f, start=start)
    _, kr = ea.ea_rope(None, K, pos, f)
    ea.ea_cache_write(b, kr, V, start=start)
    assert torch.equal(a.K, b.K) and torch.equal(a.V, b.V)


def test_append_reports_and_leaves(dev):
    """A sequence that does not fit, a page outside the cache, a row outside the input."""
    f = torch.from_numpy(inv_freq(128)).to(dev)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    for dtype in (BF16, E4M3):
        K = tokens((2, 8, 1, 128), 1).to(dev)
        c = ea.kv_cache(2, 64, 1, dtype=dtype, device=dev)
        ws = ea.cache_workspace(dev)
        ea.ea_cache_write_rope(c, K, K, f, start=i32(60, 0), workspace=ws)
        assert ea.ea_check_errors(ws) == 6
        assert not c.K[0].float().any() and c.V[1, :8].float().any()
        table = i32(3, 1, 0, 9).view(2, 2)
        p = ea.kv_cache_paged(4, 64, 1, table, dtype=dtype)
        ea.ea_cache_write_rope(p, K, K, f, start=i32(60, 62), workspace=ws)
        assert ea.ea_check_errors(ws) == 6
        v = p.V.float().abs().amax((2, 3)).cpu()
        assert (v[3, 60:] > 0).all() and (v[1, :4] > 0).all() and (v[0, 62:] > 0).all() and not v[2].any() and not v[1, 4:].any()
        c = ea.kv_cache(2, 64, 1, dtype=dtype, device=dev)
        c.V.view(torch.uint8).fill_(0x11)
        rows = torch.zeros(2, 8, dtype=torch.int32, device=dev)
        rows[0, 1], rows[1, 0] = 8, -1
        ea.ea_cache_write_rope(c, K, K, f, n_new=i32(3, 1), rows=rows, workspace=ws)
        assert ea.ea_check_errors(ws) == 6
        assert not c.V[0, 1].float().any() and not c.V[1, 0].float().any() and c.V[0, 0].float().abs().max() > 0


@pytest.mark.parametrize("dtype", [E4M3, INT8])
def test_append_non_finite(dev, dtype):
    """An infinity or a NaN makes its block NaN; other blocks and heads are as they would be."""
    f = torch.from_numpy(inv_freq(128)).to(dev)
    K = tokens((1, 100, 2, 128), 1).to(dev)
    V = K.clone()
    K[0, 70, 1, 5] = float("inf")
    V[0, 10, 0, 127] = float("nan")
    c = ea.kv_cache(1, 128, 2, dtype=dtype, scale_block=32, device=dev)
    ea.ea_cache_write_rope(c, K, V, f)
    assert torch.isnan(c.k_scale).cpu().numpy().nonzero() is not None
    assert torch.isnan(c.k_scale)[0].nonzero().cpu().tolist() == [[1, 2]] and torch.isnan(c.v_scale)[0].nonzero().cpu().tolist() == [[0, 0]]


def test_append_captured(dev):
    """One graph, replayed with new contents and lengths."""
    B, T, Hkv, Hq = 3, 4, 2, 4
    f = torch.from_numpy(inv_freq(128)).to(dev)
    K, V, Q = (tokens((B, T, h, 128), s).to(dev) for h, s in ((Hkv, 1), (Hkv, 2), (Hq, 3)))
    start = torch.tensor([0, 5, 63], dtype=torch.int32, device=dev)
    n = torch.tensor([4, 2, 3], dtype=torch.int32, device=dev)
    a, b = (ea.kv_cache(B, 128, Hkv, device=dev) for _ in range(2))
    ws = ea.cache_workspace(dev)
    qo = torch.zeros_like(Q)
    call = lambda c, o: ea.ea_cache_write_rope(c, K, V, f, Q=Q, Q_out=o, start=start, n_new=n, workspace=ws)  # noqa: E731
    call(a, qo)
    a.K.zero_()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(a, qo)
    a.K.zero_(), a.V.zero_(), a.k_scale.zero_(), a.v_scale.zero_(), qo.zero_()
    q2 = torch.zeros_like(Q)
    for step in range(3):
        g.replay()
        call(b, q2)
        assert torch.equal(a.K.view(torch.uint8), b.K.view(torch.uint8)) and torch.equal(a.V.view(torch.uint8), b.V.view(torch.uint8))
        assert torch.equal(a.k_scale, b.k_scale) and torch.equal(a.v_scale, b.v_scale) and torch.equal(qo, q2)
        start += n
        K.mul_(1.5)
        Q.neg_()
    check_no_device_error(ws)
