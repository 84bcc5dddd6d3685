"""Plain CPU implementations of the KV cache operators, in 64 bits, written from
their definitions (imported by the tests of those operators).

A reference cache is a dict: K, V (codes or bf16), ks, vs (float32 scales, None
for bf16), table (int32 [B, pages] or None), sb (tokens of a scale block)."""
import math

import numpy as np
import torch

E4M3, INT8, BF16 = torch.float8_e4m3fn, torch.int8, torch.bfloat16
QMAX = {E4M3: 448.0, INT8: 127.0}


def tokens(shape, seed):
    """bf16 N(0, 1), one token in fifty eight times larger."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    big = torch.rand(shape[:-1], generator=g) < 0.02
    return (x * torch.where(big, 8.0, 1.0)[..., None]).to(BF16)


def block_scale(amax, dtype):
    """The least power of two s >= 2^-64 with amax <= qmax * s; NaN for a non-finite amax."""
    if not math.isfinite(amax):
        return math.nan
    e = -64
    if amax > 0:
        e = max(e, math.frexp(amax)[1] - 12)
    while amax > QMAX[dtype] * 2.0 ** e:
        e += 1
    return 2.0 ** e


def encode(x, dtype):
    """float64 values (already divided by the scale) -> the nearest codes, ties to even."""
    x = np.asarray(x, np.float64)
    if dtype == INT8:
        return torch.from_numpy(np.rint(x).astype(np.int8))
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6)))
    step = np.exp2(e - 3)
    y = np.copysign(np.abs(np.rint(x / step) * step), x)      # exactly an e4m3 value
    return torch.from_numpy(y).float().to(E4M3)


def rows_of(c, b, p):
    """(outer index, row) of row p of sequence b; None if its page is outside the cache."""
    if c["table"] is None:
        return b, p
    page = c["K"].shape[1]
    o = int(c["table"][b, p // page])
    return (o, p % page) if 0 <= o < c["K"].shape[0] else None


def values(codes, scales, sb):
    """float64 values of contiguous codes [B, L, H, D] with scales [B, H, n]."""
    if scales is None:
        return codes.double()
    s = scales.double().repeat_interleave(sb, -1)[..., : codes.shape[1]]
    return codes.float().double() * s.transpose(1, 2)[..., None]


def capacity(c):
    return c["K"].shape[1] * (1 if c["table"] is None else c["table"].shape[1])


def make_table(B, n, spare, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randperm(B * n + spare, generator=g)[: B * n].view(B, n).to(torch.int32)


def make_cache(B, cap, Hkv, dtype, sb, page, seed, spare=2):
    """A reference cache whose every row holds a token (written whole)."""
    table = make_table(B, -(-cap // page), spare, seed) if page else None
    outer, rows = (B, cap) if not page else (B * table.shape[1] + spare, page)
    c = dict(K=torch.zeros(outer, rows, Hkv, 128, dtype=dtype), V=torch.zeros(outer, rows, Hkv, 128, dtype=dtype),
             ks=None, vs=None, table=table, sb=sb)
    if dtype != BF16:
        c["ks"] = torch.ones(outer, Hkv, -(-rows // sb))
        c["vs"] = torch.ones_like(c["ks"])
    n = capacity(c)
    write_ref(c, tokens((B, n, Hkv, 128), seed + 1000), tokens((B, n, Hkv, 128), seed + 2000), [0] * B, [n] * B)
    return c


def _write_block(c, kv, sc, b, p0, lo, x):
    """Rows lo .. lo + len(x) of sequence b, all in the block that starts at p0; x float64 [n, Hkv, 128]."""
    at = rows_of(c, b, p0)
    if at is None:
        return
    o, r = at
    codes, dtype = c[kv], c[kv].dtype
    k, n = lo - p0, len(x)
    if dtype == BF16:
        codes[o, r + k : r + k + n] = torch.from_numpy(x).to(BF16)
        return
    i = r // c["sb"]
    for h in range(codes.shape[2]):
        part = x[:, h]
        amax = float(np.abs(part).max()) if np.isfinite(part).all() else math.inf
        s = block_scale(amax, dtype)
        if k:
            was = float(c[sc][o, h, i])
            if math.isnan(was) or math.isnan(s):
                s = math.nan
            elif was > s:
                s = was
            elif was < s:
                old = codes[o, r : r + k, h].float().double().numpy()
                codes[o, r : r + k, h] = encode(old * (was / s), dtype)
        new = torch.zeros(n, 128).to(dtype) if math.isnan(s) else encode(part / s, dtype)
        codes[o, r + k : r + k + n, h] = new
        c[sc][o, h, i] = s


def write_ref(c, K, V, start, n):
    """ea_cache_write; start[b] None: the sequence is refused."""
    sb = c["sb"] if c["ks"] is not None else 64
    for kv, sc, x in (("K", "ks", K), ("V", "vs", V)):
        for b in range(x.shape[0]):
            if start[b] is None or n[b] == 0:
                continue
            p, end = start[b], start[b] + n[b]
            xb = x[b].double().numpy()
            while p < end:
                p0 = p // sb * sb
                stop = min(p0 + sb, end)
                _write_block(c, kv, sc, b, p0, p, xb[p - start[b] : stop - start[b]])
                p = stop


def compact_ref(src, dst, index, counts, w, w_out):
    """ea_cache_compact, into dst (and w_out)."""
    B, Hkv = index.shape[:2]
    sb = dst["sb"] if dst["ks"] is not None else 64
    cap = capacity(src)
    for b in range(B):
        n = counts[b]
        if not n:
            continue
        for kv, sc in (("K", "ks"), ("V", "vs")):
            x = np.zeros((n, Hkv, 128))
            for h in range(Hkv):
                for i in range(n):
                    p = int(index[b, h, i])
                    at = rows_of(src, b, p) if 0 <= p < cap else None
                    if at is None:
                        continue
                    v = src[kv][at[0], at[1], h].float().double().numpy()
                    if src[sc] is not None:
                        v = v * float(src[sc][at[0], h, at[1] // src["sb"]])
                    x[i, h] = v
            for p0 in range(0, n, sb):
                _write_block(dst, kv, sc, b, p0, p0, x[p0 : p0 + sb][: n - p0])
        if w is not None:
            for h in range(Hkv):
                w_out[b, h, :n] = w[b, h, index[b, h, :n].long()]


def select_ref(w, lens, keep, sink, recent):
    """ea_evict_select on float32 weights [B, Hkv, Lmax]."""
    B, Hkv, _ = w.shape
    index = np.full((B, Hkv, keep), -1, np.int32)
    for b, L in enumerate(lens):
        n = min(L, keep)
        for h in range(Hkv):
            if L <= keep:
                index[b, h, :n] = np.arange(n)
                continue
            mid = np.arange(sink, L - recent)
            x = w[b, h, mid].astype(np.float64)
            nan = np.isnan(x)
            order = np.lexsort((mid, -np.where(nan, 0.0, x), nan))       # numbers first, then heavy, then early
            best = mid[order[: keep - sink - recent]]
            index[b, h] = np.sort(np.concatenate([np.arange(sink), best, np.arange(L - recent, L)]))
    return index, np.array([min(L, keep) for L in lens], np.int32)


def logical(c):
    """K, V [B, capacity, Hkv, 128] float64 of a reference cache, its pages in order (pages outside it: zeros)."""
    out = []
    for kv, sc in (("K", "ks"), ("V", "vs")):
        codes, scales, table = c[kv], c[sc], c["table"]
        if table is None:
            out.append(values(codes, scales, c["sb"]).numpy())
            continue
        per = values(codes, scales, c["sb"])
        ok = (table >= 0) & (table < codes.shape[0])
        x = per[table.clamp(0, codes.shape[0] - 1).long()]
        x = torch.where(ok[..., None, None, None], x, 0.0)
        out.append(x.reshape(table.shape[0], -1, *codes.shape[2:]).numpy())
    return out


def value_scales(c):
    """The scale of V of every row, [B, capacity, Hkv] float64 (pages outside the cache: 1)."""
    rows, table = c["K"].shape[1], c["table"]
    per = c["vs"].double().repeat_interleave(c["sb"], -1)[..., :rows].transpose(1, 2)       # [outer, rows, Hkv]
    if table is None:
        return per.numpy()
    ok = (table >= 0) & (table < per.shape[0])
    x = torch.where(ok[..., None, None], per[table.clamp(0, per.shape[0] - 1).long()], 1.0)
    return x.reshape(table.shape[0], -1, per.shape[2]).numpy()


def kept_keys(mode, L, sink, window, mask):
    """Which of the keys 0 .. L - 1 a decode row of a sequence of length L keeps."""
    j = np.arange(L)
    if mode == 1:
        return (j < sink) | (L - 1 - j < window)
    if mode == 2:
        return mask[(L - 1) // 128][j // 128] != 0
    return np.ones(L, bool)


def decode_ref(q, K, V, vs, lens, modes, sink, window, scale, bm=None):
    """float64 (O, LSE, weights, tolerances) of a decode step on K, V [B, cap, Hkv, 128] float64.

    Tolerances, from the arithmetic: a logit is an fp32 sum of 128 products, off by at most 128 * 2^-23 of the sum
    of their magnitudes (each addition may be truncated), plus three fp32 roundings of its size; call that d.  The
    probabilities are off by 2 d + 2^-20 relative (exp2 and the normaliser).  What multiplies V's codes is w_j = p_j s_j
    (s_j the scale of V's block) in units that put the largest at 2^14, rounded to f16: by 2^-11 of itself, or, below
    f16's normal range, by half of f16's smallest step 2^-24, which is 2^-25 / 2^14 = 2^-39 of the largest p s; times
    the code v_j / s_j.  The output is rounded to bf16 (2^-8)."""
    q = q.double().numpy()
    B, Hq, D = q.shape
    cap, Hkv = K.shape[1], K.shape[2]
    g = Hq // Hkv
    O, LSE, W = np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf), np.zeros((B, Hkv, cap))
    tO, tL, tW = np.zeros_like(O), np.zeros_like(LSE), np.zeros_like(W)
    for b, L in enumerate(lens):
        for h in range(Hkv):
            if L == 0:
                continue
            keep = kept_keys(modes[b][h], L, sink, window, None if bm is None else bm[b, h])
            at = np.nonzero(keep)[0]
            if not len(at):
                continue
            k, v = K[b, at, h], V[b, at, h]
            for i in range(h * g, (h + 1) * g):
                x = scale * (k @ q[b, i])
                d = 2.0 ** -16 * scale * (np.abs(k) @ np.abs(q[b, i])) + 2.0 ** -22 * np.abs(x)
                top = x.max()
                p = np.exp(x - top)
                l = p.sum()
                LSE[b, i] = top + np.log(l)
                p /= l
                O[b, i] = p @ v
                W[b, h, at] += p
                rel = 2 * d.max() + 2.0 ** -20
                s = vs[b, at, h]
                floor = 2.0 ** -39 * (p * s).max() * (np.abs(v) / s[:, None]).sum(0)
                tO[b, i] = 2.0 ** -8 * np.abs(O[b, i]) + (rel + 2.0 ** -11) * (p @ np.abs(v)) * 1.01 + 1.01 * floor + 1e-30
                tL[b, i] = d.max() + 2.0 ** -20 * (1 + abs(LSE[b, i]))
                tW[b, h, at] += p * rel + 1e-38
    return O, LSE, W, (tO, tL, tW)


def key_weights_ref(Q, K, LSE, modes, sink, window, lens, scale, bm=None):
    """float64 (weights [B, Hkv, Lmax], tolerance) of ea_key_weights, LSE the float32 rows it is given.

    Tolerance: a logit is an fp32 sum of 128 products, off by at most 128 * 2^-23 of the sum of their magnitudes; it
    and the LSE are rounded a few times at their size (2^-22); exp2 and the sums' own rounding (a few hundred terms
    added one after the other, then the tiles') stay below 2^-13 of the result: n = 1024 additions of 2^-24 each."""
    Q, K, LSE = Q.double().numpy(), K.double().numpy(), LSE.double().numpy()
    B, Tq, Hq, _ = Q.shape
    Lmax, Hkv = K.shape[1], K.shape[2]
    g = Hq // Hkv
    W, tol = np.zeros((B, Hkv, Lmax)), np.zeros((B, Hkv, Lmax))
    for b, L in enumerate(lens):
        t = np.arange(max(0, Tq - L), Tq)
        i, j = (L - Tq + t)[:, None], np.arange(L)[None, :]
        for h in range(Hkv):
            keep = j <= i
            if modes[b][h] == 1:
                keep = keep & ((j < sink) | (i - j < window))
            elif modes[b][h] == 2:
                keep = keep & (bm[b, h][i // 128, j // 128] != 0)
            for q in range(h * g, (h + 1) * g):
                x = scale * (Q[b, t, q] @ K[b, :L, h].T)
                lse = LSE[b, q, t][:, None]
                d = 2.0 ** -16 * scale * (np.abs(Q[b, t, q]) @ np.abs(K[b, :L, h]).T) + 2.0 ** -21 * (
                    np.abs(x) + np.where(np.isfinite(lse), np.abs(lse), 0))
                keep_q = keep & np.isfinite(lse)
                p = np.where(keep_q, np.exp(np.where(keep_q, x - np.where(np.isfinite(lse), lse, 0), 0)), 0)
                W[b, h, :L] += p.sum(0)
                tol[b, h, :L] += (p * np.expm1(d)).sum(0) + 2.0 ** -13 * p.sum(0) + 1e-37
    return W, tol
