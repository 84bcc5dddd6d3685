"""What is measured of the cache operators: the 8-bit KV cache (writing it, attending to it with one query token) and
the eviction of its tokens by accumulated attention weight (the weights, the selection, the compaction).

Every case has a plain form in torch, and a call of the framework's operator.  Head dim 128 throughout."""
import math

import numpy as np
import torch

own = False

D = 128
FULL, SSA, BLOCK = 0, 1, 2
QMAX = {"e4m3": 448.0, "int8": 127.0}
# qmax = fraction * 2^exponent, fraction in [0.5, 1)
QFRAC = {"e4m3": (0.875, 9), "int8": (0.9921875, 7)}
DTYPE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8, "bf16": torch.bfloat16}
MIN_EXP = -64


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step's new tokens of a serving batch, each somewhere inside a block of its cache
        dict(name="write_step_b32", op="write", B=32, T=1, Hkv=8, Lmax=2048, fmt="e4m3", sblk=64, page=0, ragged=True, fresh=False),
        # a prefilled 32K sequence goes into an empty cache
        dict(name="write_prefill_32k", op="write", B=1, T=32768, Hkv=8, Lmax=32832, fmt="e4m3", sblk=64, page=0, ragged=False, fresh=True),
        # a chunk of prompts of different lengths appended to paged caches that already hold something
        dict(name="write_ragged_paged_int8", op="write", B=8, T=1000, Hkv=8, Lmax=4096, fmt="int8", sblk=32, page=256, ragged=True, fresh=False),
        # the smallest decode step: one sequence, six of eight heads streaming
        dict(name="decode_b1_l32k_int8_paged", op="decode", B=1, Hq=32, Hkv=8, Lmax=32768, fmt="int8", sblk=64, page=64, modes="mix", sink=128, window=2048, ragged=False, weights=False),
        # the largest: sixteen sequences of 64K, every head attending to all of its cache
        dict(name="decode_b16_l64k_full", op="decode", B=16, Hq=32, Hkv=8, Lmax=65536, fmt="e4m3", sblk=64, page=0, modes="full", sink=128, window=4096, ragged=False, weights=False),
        # sequences of all lengths (none, one token, ...), all three kinds of heads, the step's key weights wanted
        dict(name="decode_ragged_all_weights", op="decode", B=9, Hq=32, Hkv=8, Lmax=30000, fmt="e4m3", sblk=16, page=0, modes="all", sink=100, window=1500, ragged=True, weights=True),
        # the weights that the last 64 queries of a prompt give its keys
        dict(name="weights_window64_s32k", op="weights", B=1, Tq=64, Lmax=32768, Hq=32, Hkv=8, modes="full", sink=128, window=2048, ragged=False),
        # the weights of every query of a prefill
        dict(name="weights_prefill_16k", op="weights", B=1, Tq=16384, Lmax=16384, Hq=32, Hkv=8, modes="full", sink=128, window=2048, ragged=False),
        # which tokens of one long sequence stay
        dict(name="select_b1_l128k", op="select", B=1, Hkv=8, Lmax=131072, keep=8192, sink=128, recent=2048, ragged=False),
        # which tokens of a ragged batch stay, some sequences shorter than what is kept
        dict(name="select_b32_ragged", op="select", B=32, Hkv=8, Lmax=20001, keep=2048, sink=16, recent=512, ragged=True),
        # after a prefill: the kept tokens of the bf16 keys and values become the 8-bit cache
        dict(name="compact_bf16_to_e4m3", op="compact", B=1, Hkv=8, Lsrc=32768, Lmax=8192, keep=8192, src="bf16", dst="e4m3", sblk=64, page=0, ragged=False),
        # while serving: 8-bit paged caches are shortened into fresh pages
        dict(name="compact_int8_paged_b16", op="compact", B=16, Hkv=8, Lsrc=16384, Lmax=4096, keep=4000, src="int8", dst="int8", sblk=32, page=128, ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _up(x, m):
    return -(-x // m) * m


def draw(rng):
    op = rng.choice(["write", "decode", "weights", "select", "compact"])
    fmt = rng.choice(["e4m3", "int8"])
    Hkv = rng.choice([1, 2, 4, 8])
    sblk = rng.choice([16, 32, 64, 128])
    page = rng.choice([0, 0, 128, 256])
    ragged = rng.random() < 0.6
    if op == "write":
        B = _log(rng, 1, 64)
        T = min(_log(rng, 1, 32768), max(1, 32768 * 8 // (B * Hkv)))
        Lmax = _up(T + 2 * sblk + rng.randrange(0, 1024), max(256, sblk))
        return dict(op=op, B=B, T=T, Hkv=Hkv, Lmax=Lmax, fmt=fmt, sblk=sblk, page=page, ragged=ragged, fresh=rng.random() < 0.3)
    if op == "decode":
        B = _log(rng, 1, 32)
        Lmax = max(1, min(_log(rng, 1, 131072), 16 * 65536 * 8 // (B * Hkv)))
        if page:
            Lmax = max(page, Lmax // page * page)
        return dict(op=op, B=B, Hq=Hkv * rng.randrange(1, 9), Hkv=Hkv, Lmax=Lmax, fmt=fmt, sblk=sblk, page=page, modes=rng.choice(["full", "mix", "all"]),
                    sink=rng.randrange(0, 200), window=_log(rng, 1, 4096), ragged=ragged, weights=rng.random() < 0.5)
    if op == "weights":
        Lmax = _log(rng, 1, 32768)
        Hq = Hkv * rng.randrange(1, 9)
        Tq = max(1, min(_log(rng, 1, Lmax), 16384 * 16384 * 32 // (2 * Lmax * Hq)))
        B = max(1, min(_log(rng, 1, 8), 16384 * 16384 * 32 // (2 * Lmax * Tq * Hq)))
        return dict(op=op, B=B, Tq=Tq, Lmax=Lmax, Hq=Hq, Hkv=Hkv, modes=rng.choice(["full", "mix", "all"]), sink=rng.randrange(0, 200),
                    window=_log(rng, 1, 4096), ragged=ragged)
    if op == "select":
        B = _log(rng, 1, 64)
        Lmax = max(8, min(_log(rng, 8, 262144), 5000000 // (B * Hkv)))
        keep = rng.randrange(1, Lmax + 1)
        sink = rng.randrange(0, min(keep, 200) + 1)
        return dict(op=op, B=B, Hkv=Hkv, Lmax=Lmax, keep=keep, sink=sink, recent=rng.randrange(0, keep - sink + 1), ragged=ragged)
    B = _log(rng, 1, 32)
    src, dst = rng.choice([("bf16", fmt), (fmt, fmt), ("bf16", "bf16"), ("e4m3", "int8"), (fmt, "bf16")])
    keep = min(_log(rng, 1, 16384), max(1, 262144 // (B * Hkv)))
    Lsrc, Lmax = keep + min(_log(rng, 1, 16384), 1600000 // (B * Hkv)), keep + rng.randrange(0, 300)
    if page:
        Lsrc, Lmax = _up(Lsrc, page), _up(Lmax, page)
    return dict(op=op, B=B, Hkv=Hkv, Lsrc=Lsrc, Lmax=Lmax, keep=keep, src=src, dst=dst, sblk=sblk, page=page, ragged=ragged)


def _lens(B, most, ragged):
    """Lengths of a batch's sequences: all `most`, or spread over 0 .. most with an empty one and one of a single token among them."""
    if not ragged:
        return [most] * B
    v = [int(round(most * ((b * 0.6180339887 + 0.37) % 1.0))) for b in range(B)]
    v[0] = most
    if B > 1:
        v[1] = 0
    if B > 2:
        v[2] = 1
    return v


def _modes(c):
    if c["modes"] == "full":
        pick = lambda i: FULL  # noqa: E731
    elif c["modes"] == "mix":  # a quarter of the heads attends to everything
        pick = lambda i: FULL if i % 4 == 1 else SSA  # noqa: E731
    else:
        pick = lambda i: (BLOCK, FULL, SSA)[i % 3]  # noqa: E731
    return [[pick(b + h) for h in range(c["Hkv"])] for b in range(c["B"])]


def _kept(mode, L, c):
    """About how many keys a decode row of length L keeps (a block mask keeps a fifth)."""
    if mode == SSA:
        return min(L, c["sink"] + c["window"])
    return L if mode == FULL else L / 5


def work(c):
    rows = lambda n: n * c["Hkv"] * D * 2  # noqa: E731  (values of K and V)
    size = {"bf16": 2, "e4m3": 1, "int8": 1}
    if c["op"] == "write":
        n = sum(_new_lens(c))
        return {"bytes": rows(n) * 3, "flops": 0}
    if c["op"] == "decode":
        kept = sum(_kept(m, L, c) for ms, L in zip(_modes(c), _lens(c["B"], c["Lmax"], c["ragged"])) for m in ms)
        g = c["Hq"] // c["Hkv"]
        out = sum(4 * c["Hkv"] * L for L in _lens(c["B"], c["Lmax"], c["ragged"])) if c["weights"] else 0
        return {"bytes": kept * (2 * D + 8 / c["sblk"]) + c["B"] * c["Hq"] * (4 * D + 4) + out, "flops": 4 * D * g * kept}
    if c["op"] == "weights":
        g, pairs = c["Hq"] // c["Hkv"], 0.0
        lens = _lens(c["B"], c["Lmax"], c["ragged"])
        for ms, L in zip(_modes(c), lens):
            n = min(L, c["Tq"])
            for m in ms:
                if m == SSA:
                    pairs += n * min(c["sink"] + c["window"], L - n / 2)
                else:
                    pairs += n * (L - n / 2) * (1 if m == FULL else 0.2)
        return {"bytes": sum(lens) * c["Hkv"] * (2 * D + 4) + c["B"] * min(c["Tq"], c["Lmax"]) * c["Hq"] * (2 * D + 4), "flops": 2 * D * g * pairs + 1}
    if c["op"] == "select":
        lens = _lens(c["B"], c["Lmax"], c["ragged"])
        return {"bytes": 4 * c["Hkv"] * sum(L + min(L, c["keep"]) for L in lens), "flops": 0}
    n = sum(_lens(c["B"], c["keep"], c["ragged"]))
    return {"bytes": rows(n) * (size[c["src"]] + size[c["dst"]]) + 12 * n * c["Hkv"], "flops": 0}


def _new_lens(c):
    """New tokens of each sequence of a write."""
    return _lens(c["B"], c["T"], c["ragged"])


def _starts(c):
    if c["fresh"]:
        return [0] * c["B"]
    return [(b * 7919 + 37) % (c["Lmax"] - c["T"] + 1) for b in range(c["B"])]


# ---------------------------------------------------------------- 8-bit blocks, plain
def _pow2(e):
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _scale_of(amax, fmt):
    """The least power of two s, from 2^-64 on, with amax <= qmax * s (int32 arithmetic on the exponent: exact)."""
    frac, top = QFRAC[fmt]
    m, k = torch.frexp(amax)
    e = torch.where(amax > 0, k - top + (m > frac).int(), MIN_EXP)
    return _pow2(e.clamp(min=MIN_EXP))


def _round(x, fmt):
    return x.to(torch.float8_e4m3fn) if fmt == "e4m3" else x.round().to(torch.int8)


def _quantize(x, fmt, sblk):
    """x [..., L, H, D] float32 -> codes [..., L, H, D], scales [..., H, ceil(L / sblk)]."""
    if fmt == "bf16":
        return x.to(torch.bfloat16), None
    L, H = x.shape[-3], x.shape[-2]
    n = -(-L // sblk)
    p = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, n * sblk - L))
    p = p.view(*x.shape[:-3], n, sblk, H, D)
    s = _scale_of(p.abs().amax((-3, -1)), fmt)                                    # [..., n, H]
    codes = _round(p / s[..., None, :, None], fmt).view(*x.shape[:-3], n * sblk, H, D)[..., :L, :, :]
    return codes.contiguous(), s.transpose(-1, -2).contiguous()


def _values(codes, s, sblk):
    """The values that codes [..., L, H, D] with scales [..., H, n] stand for, in float32."""
    x = codes.float()
    if s is None:
        return x
    per_row = s.transpose(-1, -2).repeat_interleave(sblk, -2)[..., : codes.shape[-3], :]
    return x * per_row[..., None]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _tokens(shape, g):
    """Keys or values of a model: normal, the channels of different size, a few tokens much larger."""
    x = torch.randn(shape, generator=g, device="cuda")
    x *= 0.5 + torch.rand((shape[-2], shape[-1]), generator=g, device="cuda")
    big = torch.rand(shape[:-1], generator=g, device="cuda") < 0.01
    return (x * torch.where(big, 6.0, 1.0)[..., None]).to(torch.bfloat16)


def _filled(B, L, Hkv, fmt, sblk, g):
    """K and V of B sequences of L rows in one format: codes [B, L, Hkv, D], scales [B, Hkv, n], one sequence at a time."""
    n = -(-L // sblk)
    c = [torch.empty((B, L, Hkv, D), dtype=DTYPE[fmt], device="cuda") for _ in range(2)]
    s = [None if fmt == "bf16" else torch.empty((B, Hkv, n), device="cuda") for _ in range(2)]
    for b in range(B):
        for i in range(2):
            code, sc = _quantize(_tokens((L, Hkv, D), g).float(), fmt, sblk)
            c[i][b] = code
            if sc is not None:
                s[i][b] = sc
    return c[0], c[1], s[0], s[1]


def _paged(parts, page, sblk, g, spare=3):
    """The same cache in pages in a mixed order: (parts, block table)."""
    K = parts[0]
    B, L, Hkv = K.shape[:3]
    n = -(-L // page)
    table = torch.randperm(B * n + spare, generator=g, device="cuda")[: B * n].view(B, n)
    out = []
    for i, t in enumerate(parts):
        if t is None:
            out.append(None)
            continue
        if i < 2:
            t = t.view(torch.uint8) if t.dtype != torch.bfloat16 else t
            p = torch.zeros((B * n + spare, page, Hkv, D), dtype=t.dtype, device="cuda")
            p[table.view(-1)] = t.reshape(B * n, page, Hkv, D)
            p = p.view(parts[0].dtype)
        else:
            p = torch.full((B * n + spare, Hkv, page // sblk), 1.0, device="cuda")
            p[table.view(-1)] = t.view(B, Hkv, n, page // sblk).transpose(1, 2).reshape(B * n, Hkv, page // sblk)
        out.append(p)
    return out, table.to(torch.int32)


def _unpaged(t, table):
    """Pages [P, page, H, D] (or scales [P, H, k]) as contiguous sequences."""
    if t is None or table is None:
        return t
    B, n = table.shape
    x = (t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t)[table.view(-1).long()]
    if t.dim() == 4:
        return x.view(B, n * t.shape[1], t.shape[2], D).view(t.dtype)
    return x.view(B, n, t.shape[1], t.shape[2]).transpose(1, 2).reshape(B, t.shape[1], n * t.shape[2])


def _cache(B, L, Hkv, fmt, sblk, page, g):
    parts, table = _filled(B, L, Hkv, fmt, sblk, g), None
    if page:
        parts, table = _paged(parts, page, sblk, g)
    return dict(K=parts[0], V=parts[1], ks=parts[2], vs=parts[3], table=table, sblk=sblk, fmt=fmt)


def _empty(B, L, Hkv, fmt, sblk, page, g):
    """A cache with nothing in it."""
    n = -(-L // sblk)
    z = lambda *s, t=torch.float32: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    parts = [z(B, L, Hkv, D, t=DTYPE[fmt]), z(B, L, Hkv, D, t=DTYPE[fmt])] + ([None, None] if fmt == "bf16" else [z(B, Hkv, n), z(B, Hkv, n)])
    table = None
    if page:
        parts, table = _paged(parts, page, sblk, g)
    return dict(K=parts[0], V=parts[1], ks=parts[2], vs=parts[3], table=table, sblk=sblk, fmt=fmt)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _block_mask(c, g):
    """[B, Hkv, n, n]: key block 0, the diagonal and a fifth of the others; one row of the first head that reads it is empty."""
    n = -(-c["Lmax"] // 128)
    bm = (torch.rand((c["B"], c["Hkv"], n, n), generator=g, device="cuda") < 0.2)
    i = torch.arange(n, device="cuda")
    bm[:, :, i, i] = True
    bm[:, :, :, 0] = True
    if c["B"] > 3:
        bm[3] = False
    return (bm & (i[None, :] <= i[:, None])).to(torch.uint8)


def prepare(c, seed):
    g = _gen(seed)
    st = {"case": c}
    if c["op"] == "write":
        Lmax = c["Lmax"] if not c["page"] else _up(c["Lmax"], c["page"])
        make = _empty if c["fresh"] else _cache
        st["cache"] = make(c["B"], Lmax, c["Hkv"], c["fmt"], c["sblk"], c["page"], g)
        st["Kn"], st["Vn"] = (_tokens((c["B"], c["T"], c["Hkv"], D), g) for _ in range(2))
        st["start"], st["n"] = _i32(_starts(c)), _i32(_new_lens(c))
    elif c["op"] == "decode":
        st["cache"] = _cache(c["B"], c["Lmax"], c["Hkv"], c["fmt"], c["sblk"], c["page"], g)
        st["q"] = torch.randn((c["B"], c["Hq"], D), generator=g, device="cuda").to(torch.bfloat16)
        st["lens"] = _i32(_lens(c["B"], c["Lmax"], c["ragged"]))
        st["m"] = torch.tensor(_modes(c), dtype=torch.uint8, device="cuda")
        st["bm"] = _block_mask(c, g) if c["modes"] == "all" else None
        st["w"] = torch.zeros((c["B"], c["Hkv"], c["Lmax"]), device="cuda") if c["weights"] else None
    elif c["op"] == "weights":
        st["Q"] = torch.randn((c["B"], c["Tq"], c["Hq"], D), generator=g, device="cuda").to(torch.bfloat16)
        st["K"] = _tokens((c["B"], c["Lmax"], c["Hkv"], D), g)
        st["lens"] = _i32(_lens(c["B"], c["Lmax"], c["ragged"]))
        st["m"] = torch.tensor(_modes(c), dtype=torch.uint8, device="cuda")
        st["bm"] = _block_mask(c, g) if c["modes"] == "all" else None
        st["w"] = torch.zeros((c["B"], c["Hkv"], c["Lmax"]), device="cuda")
        st["LSE"] = _row_lse(st)
    elif c["op"] == "select":
        w = torch.rand((c["B"], c["Hkv"], c["Lmax"]), generator=g, device="cuda").pow(12)
        st["w"] = torch.where(w < 1e-6, 0.0, w)      # most keys were hardly looked at, a third of them never
        st["lens"] = _i32(_lens(c["B"], c["Lmax"], c["ragged"]))
    else:
        st["src"] = _cache(c["B"], c["Lsrc"], c["Hkv"], c["src"], c["sblk"], c["page"], g)
        st["dst"] = _empty(c["B"], c["Lmax"], c["Hkv"], c["dst"], c["sblk"], c["page"], g)
        st["n"] = _i32(_lens(c["B"], c["keep"], c["ragged"]))
        perm = torch.rand((c["B"], c["Hkv"], c["Lsrc"]), generator=g, device="cuda").argsort(-1)[..., : c["keep"]]
        st["index"] = perm.sort(-1).values.to(torch.int32).contiguous()
        st["w"] = torch.rand((c["B"], c["Hkv"], c["Lsrc"]), generator=g, device="cuda")
        st["w_out"] = torch.zeros((c["B"], c["Hkv"], c["Lmax"]), device="cuda")
    return st


# ---------------------------------------------------------------- plain forms
def _keep_mask(c, lens, m, bm, rows):
    """Which keys [B, Hkv, T, Lmax] the query rows at positions `rows` [B, T] keep (negative positions: none)."""
    j = torch.arange(c["Lmax"], device=rows.device)
    i = rows[:, None, :, None]
    causal = (j <= i) & (j < lens[:, None, None, None])
    mode = m[:, :, None, None]
    keep = causal & ((mode != SSA) | (j < c["sink"]) | (i - j < c["window"]))
    if bm is not None:
        qb = (rows.clamp(min=0) // 128).long()
        picked = torch.gather(bm, 2, qb[:, None, :, None].expand(-1, bm.shape[1], -1, bm.shape[3]))
        keep &= (mode != BLOCK) | (picked.repeat_interleave(128, -1)[..., : c["Lmax"]] != 0)
    return keep


def _rows(c, lens, T):
    return lens.long()[:, None] - T + torch.arange(T, device=lens.device)


def _scores(Q, K):
    """[B, Hkv, g, T, L] products of queries [B, T, Hq, D] and keys [B, L, Hkv, D]."""
    B, T, Hq = Q.shape[:3]
    Hkv = K.shape[2]
    q = Q.view(B, T, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    return torch.matmul(q, K.permute(0, 2, 3, 1)).view(B, Hkv, Hq // Hkv, T, K.shape[1])


def _row_lse(st):
    """The prefill's log-sum-exp of each query row, [B, Hq, Tq]: -inf where a row keeps nothing."""
    c = st["case"]
    keep = _keep_mask(c, st["lens"], st["m"], st["bm"], _rows(c, st["lens"], c["Tq"]))
    out = torch.empty((c["B"], c["Hkv"], c["Hq"] // c["Hkv"], c["Tq"]), device="cuda")
    for h in range(c["Hkv"]):
        g = c["Hq"] // c["Hkv"]
        s = _scores(st["Q"][:, :, h * g : (h + 1) * g].float(), st["K"][:, :, h : h + 1].float()).mul_(D**-0.5)
        s.masked_fill_(~keep[:, h : h + 1, None], -math.inf)
        out[:, h] = torch.logsumexp(s, -1)[:, 0]
    return out.view(c["B"], c["Hq"], c["Tq"])


def _plain_write(st):
    c, cache = st["case"], st["cache"]
    sblk, fmt, table, B, T = c["sblk"], c["fmt"], cache["table"], c["B"], c["T"]
    Lmax = cache["K"].shape[1] if table is None else table.shape[1] * c["page"]
    start, n = st["start"].long()[:, None], st["n"].long()[:, None]
    R = min(-(-(T + sblk - 1) // sblk) * sblk, Lmax)                  # rows of whole blocks that hold the new tokens
    r0 = torch.clamp(start // sblk * sblk, max=Lmax - R)
    pos = r0 + torch.arange(R, device="cuda")                         # [B, R]
    b = torch.arange(B, device="cuda")[:, None]
    outer, row = (b.expand(-1, R), pos) if table is None else (table.long().gather(1, pos // c["page"]), pos % c["page"])
    fresh = (pos >= start) & (pos < start + n)
    touched = fresh.view(B, -1, sblk).any(-1)                         # [B, R / sblk]
    before = ((pos < start).view(B, -1, sblk).any(-1) & touched)[..., None]
    for codes, scales, x in ((cache["K"], cache["ks"], st["Kn"]), (cache["V"], cache["vs"], st["Vn"])):
        raw = codes.view(torch.uint8) if fmt == "e4m3" else codes
        old = raw[outer, row].view(codes.dtype)                       # [B, R, Hkv, D]
        new = torch.where(fresh[..., None, None], x.gather(1, (pos - start).clamp(0, T - 1)[..., None, None].expand(-1, -1, c["Hkv"], D)).float(), 0.0)
        so = outer.view(B, -1, sblk)[..., 0], row.view(B, -1, sblk)[..., 0] // sblk
        s_old = scales[so[0], :, so[1]]                               # [B, nb, Hkv]
        s = _scale_of(new.view(B, -1, sblk, c["Hkv"], D).abs().amax((2, 4)), fmt)
        s = torch.where(before, torch.maximum(s, s_old), s)
        s = torch.where(touched[..., None], s, s_old)
        wide = lambda v: v.repeat_interleave(sblk, 1)[..., None]  # noqa: E731
        grown = wide((s != s_old) & before)
        value = torch.where(fresh[..., None, None], new / wide(s), old.float() * torch.where(grown, wide(s_old) / wide(s), 1.0))
        code = _round(value, fmt)
        stay = (~fresh)[..., None, None] & ((pos >= start)[..., None, None] | ~grown)
        code = torch.where(stay, raw[outer, row], code.view(raw.dtype))
        raw[outer, row] = code
        scales[so[0], :, so[1]] = s
    return _cache_out(cache)


def _cache_out(cache):
    return [x for x in (cache["K"], cache["V"], cache["ks"], cache["vs"]) if x is not None]


def _plain_decode(st):
    c, cache = st["case"], st["cache"]
    K, V = (_values(_unpaged(cache[t], cache["table"]), _unpaged(cache[s], cache["table"]), c["sblk"]) for t, s in (("K", "ks"), ("V", "vs")))
    lens = st["lens"].long()
    keep = _keep_mask(c, lens, st["m"], st["bm"], _rows(c, lens, 1))             # [B, Hkv, 1, L]
    s = _scores(st["q"].float()[:, None], K)[..., 0, :] * D**-0.5                 # [B, Hkv, g, L]
    s = s.masked_fill(~keep, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - top.masked_fill(top == -math.inf, 0.0))
    total = p.sum(-1, keepdim=True)
    O = torch.matmul(p, V.permute(0, 2, 1, 3)) / total.masked_fill(total == 0, 1.0)
    LSE = (top + torch.log(total))[..., 0].view(c["B"], c["Hq"])
    out = [O.reshape(c["B"], c["Hq"], D).to(torch.bfloat16), LSE]
    if c["weights"]:
        w = (p / total.masked_fill(total == 0, 1.0)).sum(2)
        j = torch.arange(c["Lmax"], device="cuda")
        out.append(torch.where(j < lens[:, None, None], w, st["w"]))
    return out


def _plain_weights(st):
    c, lens = st["case"], st["lens"].long()
    keep = _keep_mask(c, lens, st["m"], st["bm"], _rows(c, lens, c["Tq"]))
    s = _scores(st["Q"].float(), st["K"].float()).mul_(D**-0.5)
    lse = st["LSE"].view(c["B"], c["Hkv"], -1, c["Tq"], 1)
    s = s.sub_(lse.masked_fill(lse == -math.inf, 0.0)).exp_()
    w = s.mul_(keep[:, :, None]).sum((2, 3))
    j = torch.arange(c["Lmax"], device="cuda")
    return torch.where(j < lens[:, None, None], w, st["w"])


def _plain_select(st):
    c = st["case"]
    L = st["lens"].long()[:, None, None]
    j = torch.arange(c["Lmax"], device="cuda")
    w = torch.where((j < c["sink"]) | (j >= L - c["recent"]), math.inf, st["w"])
    w = torch.where(j < L, w, -math.inf)
    first = w.sort(dim=-1, descending=True, stable=True).indices[..., : c["keep"]]
    n = torch.clamp(L, max=c["keep"])
    k = torch.arange(first.shape[-1], device="cuda")
    at = torch.where(k < n, first, c["Lmax"]).sort(-1).values
    return torch.where(k < n, at, -1).to(torch.int32), n[:, 0, 0].to(torch.int32)


def _plain_compact(st):
    c, src, dst = st["case"], st["src"], st["dst"]
    live = torch.arange(c["keep"], device="cuda") < st["n"][:, None]              # [B, keep]
    at = st["index"].long()                                                       # [B, Hkv, keep]
    B, Hkv = c["B"], c["Hkv"]
    pos = torch.arange(c["keep"], device="cuda").expand(B, -1)
    if dst["table"] is None:
        outer, row = torch.arange(B, device="cuda")[:, None].expand(-1, c["keep"]), pos
    else:
        outer, row = dst["table"].long().gather(1, pos // c["page"]), pos % c["page"]
    for t, s in (("K", "ks"), ("V", "vs")):
        x = _values(_unpaged(src[t], src["table"]), _unpaged(src[s], src["table"]), c["sblk"])
        x = x.gather(1, at.transpose(1, 2)[..., None].expand(-1, -1, -1, D))
        x = torch.where(live[..., None, None], x, 0.0)
        codes, scales = _quantize(x, c["dst"], c["sblk"])
        raw = dst[t].view(torch.uint8) if c["dst"] == "e4m3" else dst[t]
        raw[outer, row] = torch.where(live[..., None, None], codes.view(raw.dtype), raw[outer, row])
        if scales is not None:
            first = slice(None, None, c["sblk"])
            so = outer[:, first], row[:, first] // c["sblk"]
            dst[s][so[0], :, so[1]] = torch.where(live[:, first, None], scales.transpose(1, 2), dst[s][so[0], :, so[1]])
    k = c["keep"]
    st["w_out"][..., :k] = torch.where(live[:, None], st["w"].gather(2, at), st["w_out"][..., :k])
    return _cache_out(dst) + [st["w_out"]]


# ---------------------------------------------------------------- the framework's calls
def _handles(st):
    """What a program sets up once for its buffers: the cache handles and the workspace."""
    import sparse_head_attention_gb300 as ea

    c, h = st["case"], {"ea": ea}
    for name in ("cache", "src", "dst"):
        if name in st:
            x = st[name]
            h[name] = ea.KVCache(x["K"], x["V"], x["ks"], x["vs"], scale_block=x["sblk"], block_table=x["table"])
    if c["op"] == "decode":
        h["ws"] = ea.decode_q8_workspace(c["B"], c["Hq"], c["Hkv"], c["Lmax"], weights=c["weights"])
    elif c["op"] == "weights":
        h["ws"] = ea.key_weights_workspace(c["B"], c["Tq"], c["Lmax"], c["Hq"], c["Hkv"])
    else:
        h["ws"] = ea.cache_workspace()
    st["handles"] = h
    return h


def _own(st):
    c, h = st["case"], st.get("handles") or _handles(st)
    ea, ws = h["ea"], h["ws"]
    if c["op"] == "write":
        ea.ea_cache_write(h["cache"], st["Kn"], st["Vn"], st["start"], st["n"], workspace=ws)
        return _cache_out(st["cache"])
    if c["op"] == "decode":
        O, LSE = ea.ea_hybrid_attn_decode_q8(st["q"], h["cache"], st["lens"], st["m"], sink=c["sink"], window=c["window"], block_mask=st["bm"],
                                             key_weights=st["w"], accumulate=False, workspace=ws)
        return [O, LSE] if st["w"] is None else [O, LSE, st["w"]]
    if c["op"] == "weights":
        return ea.ea_key_weights(st["Q"], st["K"], st["LSE"], st["m"], seqlens=st["lens"], sink=c["sink"], window=c["window"], block_mask=st["bm"],
                                 weights=st["w"], accumulate=False, workspace=ws)
    if c["op"] == "select":
        return ea.ea_evict_select(st["w"], st["lens"], keep=c["keep"], sink=c["sink"], recent=c["recent"], workspace=ws)
    ea.ea_cache_compact(h["src"], h["dst"], st["index"], st["n"], weights=st["w"], weights_out=st["w_out"], workspace=ws)
    return _cache_out(st["dst"]) + [st["w_out"]]


def run(st):
    if own:
        return _own(st)
    op = st["case"]["op"]
    return {"write": _plain_write, "decode": _plain_decode, "weights": _plain_weights, "select": _plain_select, "compact": _plain_compact}[op](st)


# ---------------------------------------------------------------- in 64 bits, from the definitions
def _np(t):
    """A tensor as a 64-bit array (whole numbers stay whole)."""
    return (t.double() if t.dtype.is_floating_point else t).cpu().numpy()


def _nearest(x, fmt):
    """The format's value nearest to x, ties to the even code."""
    if fmt == "int8":
        return np.rint(x)
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0**-6)))
    step = np.exp2(e - 3)
    return np.rint(x / step) * step


def _least_scale(a, fmt):
    if a == 0:
        return 2.0**MIN_EXP
    e = MIN_EXP
    guess = int(math.floor(math.log2(a / QMAX[fmt]))) - 1
    e = max(e, guess)
    while a > QMAX[fmt] * 2.0**e:
        e += 1
    return 2.0**e


def _place(cache, page, b, pos):
    if cache["table_np"] is None:
        return b, pos
    return cache["table_np"][b, pos // page], pos % page


def _exact_blocks(c, cache, out, b, first, count, value, fmt):
    """Writes rows first .. first + count of sequence b: value(i, h) [count, Hkv, D] as float64 for each of K and V."""
    sblk, page = c["sblk"], c["page"]
    for i in range(2):
        x = value(i)
        codes, scales = out[i], out[2 + i] if fmt != "bf16" else None
        p = first
        while p < first + count:
            stop = min((p // sblk + 1) * sblk, first + count)
            o, r = _place(cache, page, b, p)
            part = x[p - first : stop - first]
            if fmt == "bf16":
                codes[o, r : r + stop - p] = part
                p = stop
                continue
            amax = np.abs(part).max((0, 2))
            for h in range(c["Hkv"]):
                s = _least_scale(amax[h], fmt)
                k = p % sblk                                # rows of the block that were there
                if k:
                    was = scales[o, h, r // sblk]
                    s = max(s, was)
                    if s != was:
                        codes[o, r - k : r, h] = _nearest(codes[o, r - k : r, h] * (was / s), fmt)
                codes[o, r : r + stop - p, h] = _nearest(part[:, h] / s, fmt)
                scales[o, h, r // sblk] = s
            p = stop


def _whole_if(fmt, arrays):
    return [a.astype(np.int64) if fmt == "int8" and i < 2 else a for i, a in enumerate(arrays)]


def _as_np(cache):
    cache["table_np"] = None if cache["table"] is None else cache["table"].cpu().numpy()
    return [None if cache[k] is None else _np(cache[k]).astype(np.float64) for k in ("K", "V", "ks", "vs")]


def exact(c, seed):
    st = prepare(c, seed)
    if c["op"] == "write":
        out = _as_np(st["cache"])
        new = [_np(st["Kn"]), _np(st["Vn"])]
        for b, (p, n) in enumerate(zip(_starts(c), _new_lens(c))):
            if n:
                _exact_blocks(c, st["cache"], out, b, p, n, lambda i: new[i][b, :n], c["fmt"])
        return _whole_if(c["fmt"], out)
    if c["op"] == "compact":
        src, out = _as_np(st["src"]), _as_np(st["dst"])
        index, w, w_out = st["index"].cpu().numpy(), _np(st["w"]), _np(st["w_out"])
        for b, n in enumerate(_lens(c["B"], c["keep"], c["ragged"])):
            if not n:
                continue
            at = index[b, :, :n]                                                    # [Hkv, n]
            o, r = _place(st["src"], c["page"], b, at) if c["page"] else (np.full_like(at, b), at)
            heads = np.arange(c["Hkv"])[:, None]

            def value(i):
                x = src[i][o, r, heads]                                             # [Hkv, n, D]
                if src[2 + i] is not None:
                    x = x * src[2 + i][o, heads, r // c["sblk"]][..., None]
                return x.transpose(1, 0, 2)

            if c["dst"] == "bf16":
                _exact_blocks(c, st["dst"], out, b, 0, n, value, "bf16")
            else:
                _exact_blocks(c, st["dst"], out, b, 0, n, value, c["dst"])
            w_out[b, :, :n] = np.take_along_axis(w[b], at.astype(np.int64), 1)
        return [x for x in _whole_if(c["dst"], out) if x is not None] + [w_out]
    if c["op"] == "select":
        w, lens = _np(st["w"]), _lens(c["B"], c["Lmax"], c["ragged"])
        index = np.full((c["B"], c["Hkv"], min(c["keep"], c["Lmax"])), -1, np.int64)
        for b, L in enumerate(lens):
            n = min(L, c["keep"])
            for h in range(c["Hkv"]):
                if L <= c["keep"]:
                    index[b, h, :n] = np.arange(n)
                    continue
                middle = np.arange(c["sink"], L - c["recent"])
                best = middle[np.argsort(-w[b, h, middle], kind="stable")[: c["keep"] - c["sink"] - c["recent"]]]
                index[b, h, :n] = np.sort(np.concatenate([np.arange(c["sink"]), best, np.arange(L - c["recent"], L)]))
        return index, np.array([min(L, c["keep"]) for L in lens], np.int64)
    return _exact_attention(c, st)


def _exact_attention(c, st):
    """Decode steps and key weights, one KV head at a time, in float64 on the GPU."""
    g, lens, modes = c["Hq"] // c["Hkv"], _lens(c["B"], c["Lmax"], c["ragged"]), _modes(c)
    decode = c["op"] == "decode"
    T = 1 if decode else c["Tq"]
    O = torch.zeros((c["B"], c["Hq"], D), dtype=torch.float64, device="cuda")
    LSE = torch.full((c["B"], c["Hq"]), -math.inf, dtype=torch.float64, device="cuda")
    W = st["w"].double() if st["w"] is not None else None
    if decode:
        cache = st["cache"]
        K, V, ks, vs = (_unpaged(cache[k], cache["table"]) for k in ("K", "V", "ks", "vs"))
    for b, L in enumerate(lens):
        j = torch.arange(L, device="cuda")
        for h in range(c["Hkv"]):
            if W is not None:
                W[b, h, :L] = 0
            if L == 0:
                continue
            if decode:
                k = K[b, :L, h].double() * ks[b, h, j // c["sblk"], None].double()
                v = V[b, :L, h].double() * vs[b, h, j // c["sblk"], None].double()
            else:
                k = st["K"][b, :L, h].double()
            for t0 in range(max(0, T - L), T, 2048):
                t = torch.arange(t0, min(t0 + 2048, T), device="cuda")
                i = (L - T + t)[:, None]
                keep = j <= i
                if modes[b][h] == SSA:
                    keep = keep & ((j < c["sink"]) | (i - j < c["window"]))
                elif modes[b][h] == BLOCK:
                    keep = keep & (st["bm"][b, h][i // 128, j // 128] != 0)
                for q in range(h * g, (h + 1) * g):
                    x = (st["q"][b, q][None] if decode else st["Q"][b, t, q]).double() @ k.T * D**-0.5
                    x = torch.where(keep, x, -math.inf)
                    if decode:
                        if not bool(keep.any()):
                            continue
                        LSE[b, q] = torch.logsumexp(x[0], 0)
                        p = torch.exp(x[0] - LSE[b, q])
                        O[b, q] = p @ v
                    else:
                        lse = st["LSE"][b, q, t].double()[:, None]
                        p = torch.where(keep, torch.exp(x - torch.where(lse == -math.inf, 0.0, lse)), 0.0).sum(0)
                    if W is not None:
                        W[b, h, :L] += p
    if not decode:
        return W
    return [O, LSE] + ([W] if W is not None else [])
