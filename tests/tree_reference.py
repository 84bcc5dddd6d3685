"""Plain CPU implementations of the operators for drafted tokens, in 64 bits, written
from their definitions (imported by those operators' tests)."""
import math

import numpy as np

FULL, SSA, BLOCK = 0, 1, 2


def inv_freq(rot, base=500000.0):
    """float32 frequencies of a rotation, as a model holds them."""
    return (base ** (-2.0 * np.arange(rot // 2) / rot)).astype(np.float32)


def turn_fraction(pos, f):
    """pos * f / 2 pi mod 1 of integers and float32 frequencies: exact integers times 1 / 2 pi to 192 bits."""
    inv2pi = 0x28be60db9391054a7f09d5f47d4d377036d8a5664f10e410  # 1 / 2 pi in units of 2^-192
    out = np.zeros((len(pos), len(f)))
    for j, x in enumerate(f):
        m, e = math.frexp(float(x))
        m = int(m * 2 ** 24)                        # x = m 2^(e - 24)
        for i, p in enumerate(pos):
            shift = 192 + 24 - e
            v = (int(p) * m * inv2pi) % (1 << shift)
            out[i, j] = (v >> (shift - 60)) / 2.0 ** 60
    return out


def rotate(x, pos, f, interleaved, scale=1.0):
    """x float64 [n, H, 128] at positions [n]; f float32 [rot / 2]."""
    rot = 2 * len(f)
    a = 2 * math.pi * turn_fraction(pos, f)[:, None, :]
    c, s = np.cos(a) * scale, np.sin(a) * scale
    y = x.copy()
    i = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    j = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., j] * c + x[..., i] * s
    return y


def rotate_error(x, f, interleaved, scale=1.0):
    """How far an fp32 rotation may be off: the angle is off by pi 2^-31 of truncation and pi 2^-24 of rounding, the sine
    and cosine by 2 ulp (2^-23), each product and sum by 2^-24: in all below 2^-21 of |x_i| + |x_j|."""
    rot = 2 * len(f)
    e = np.zeros_like(x)
    i = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    j = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    e[..., i] = e[..., j] = (np.abs(x[..., i]) + np.abs(x[..., j])) * 2.0 ** -21 * abs(scale)
    return e


def plan(parents, n):
    """depth [B, T], mask int32 [B, T, 4]."""
    B, T = parents.shape
    depth, mask = np.zeros((B, T), np.int32), np.zeros((B, T, 4), np.uint32)
    for b in range(B):
        for t in range(n[b]):
            u = t
            while True:
                mask[b, t, u // 32] |= np.uint32(1 << (u % 32))
                p = int(parents[b, u])
                if not 0 <= p < u:
                    break
                u = p
                depth[b, t] += 1
    return depth, mask.view(np.int32)


def accept(tokens, parents, targets, n):
    B, T = parents.shape
    path, count, nxt = np.full((B, T), -1, np.int32), np.zeros(B, np.int32), np.full(B, -1, np.int32)
    for b in range(B):
        at = 0 if n[b] else None
        while at is not None:
            path[b, count[b]] = at
            count[b] += 1
            nxt[b] = targets[b, at]
            kids = [t for t in range(at + 1, n[b]) if parents[b, t] == at and tokens[b, t] == targets[b, at]]
            at = kids[0] if kids else None
    return path, count, nxt


def random_tree(B, T, seed, kind="tree"):
    r = np.random.RandomState(seed)
    p = np.full((B, T), -1, np.int32)
    for b in range(B):
        for t in range(1, T):
            if kind == "chain":
                p[b, t] = t - 1
            elif kind == "star":
                p[b, t] = 0
            elif kind == "forest":
                p[b, t] = r.randint(-1, t)
            else:
                p[b, t] = r.randint(0, t)
    return p


def units(scales, lens):
    """What the f16 numbers of a key's tile of an 8-bit cache stand for: the largest scale of the 128 aligned rows (below the
    sequence's length), over 2^6 (e4m3) or 2^5 (int8; 2^6 here, the smaller).  scales float64 [B, cap, Hkv]."""
    u = np.ones_like(scales)
    for b, L in enumerate(lens):
        for j in range(0, L, 128):
            u[b, j : j + 128] = scales[b, j : min(j + 128, L)].max(0) / 64
    return u


def attend(Q, K, V, Kc, Vc, lens, n, depth, mask, modes, sink, window, scale, bm=None, vunit=None):
    """ea_hybrid_attn_tree in 64 bits.  Q [B, T, Hq, 128], K, V [B, T, Hkv, 128], Kc, Vc [B, cap, Hkv, 128] float64.
    Returns O [B, T, Hq, 128], LSE [B, Hq, T] and how far an fp32 kernel with bf16 probabilities may be off:
      a product q . k sums 128 fp32 terms: 2^-17 of sum |q k|, times scale: a logit's error; its exponent is one fused
      multiply-add of up to 2^6 (2^-18 relative to p) and the exponential 2^-22;
      a probability is rounded to bf16 (2^-8), the output too; sums over keys are fp32 in tiles of 128 (2^-17) that are
      joined by weights of 2^-20.
    8-bit caches (vunit: units() of V's scales): probabilities are f16 instead, w_j = p_j u_j in units of 2^-7 of the largest
    weight M; one that is below 2^-14 is subnormal, off by 2^-25.  The sum of w / u is 2^7 / max u at least, and the f16
    numbers of V are v_j / u_j, so that adds at most 2^-32 max(u) sum |v_j| / u_j to an output.  The tree's own values are f16
    too, times a power of two that puts the largest in [2^14, 2^15), so off by 2^-39 of it at most where subnormal."""
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
            k = np.concatenate([Kc[b, :L, h], K[b, :nb, h]])
            v = np.concatenate([Vc[b, :L, h], V[b, :nb, h]])
            if vunit is not None and nb:
                own = 2.0 ** (np.floor(np.log2(max(np.abs(V[b, :nb, h]).max(), 2.0 ** -126))) - 14)
                u = np.concatenate([vunit[b, :L, h], np.full(nb, own)])
            keep = np.concatenate([np.ones((nb, L), bool), up], 1)
            if modes[b][h] == SSA:
                keep &= (at[None] < sink) | (pos[:, None] - at[None] < window)
            elif modes[b][h] == BLOCK:
                keep &= bm[b, h][pos // 128][:, at // 128] != 0
            for t in range(nb):
                j = np.flatnonzero(keep[t])
                if not len(j):
                    continue
                q = Q[b, t, h * g : (h + 1) * g]
                x = q @ k[j].T * scale
                e = (np.abs(q) @ np.abs(k[j]).T * scale).max(1) * 2.0 ** -17 + 2.0 ** -17
                top = x.max(1, keepdims=True)
                p = np.exp(x - top)
                s = p.sum(1, keepdims=True)
                p /= s
                hs = slice(h * g, (h + 1) * g)
                O[b, t, hs] = p @ v[j]
                LSE[b, hs, t] = (top + np.log(s))[:, 0]
                tO[b, t, hs] = (p @ np.abs(v[j])) * (2.0 ** -8 + 2 * e[:, None]) + np.abs(O[b, t, hs]) * 2.0 ** -8
                if vunit is not None:
                    tO[b, t, hs] += 2.0 ** -32 * u[j].max() * (np.abs(v[j]) / u[j][:, None]).sum(0) + 2.0 ** -39 * np.abs(V[b, :nb, h]).max()
                tL[b, hs, t] = e + np.abs(LSE[b, hs, t]) * 2.0 ** -20
    return O, LSE, tO, tL
