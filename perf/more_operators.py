"""What is measured of the operators around drafted tokens: rotating queries and keys by their positions, appending rotated
keys to a cache, the ancestors of a token tree, attention of the tree over a cache, and the walk that accepts a path.

Every case has a plain form in torch, and a call of the framework's operator.  Head dim 128 throughout."""
import math

import torch

own = False

D = 128
FULL, SSA, BLOCK = 0, 1, 2
DTYPE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8, "bf16": torch.bfloat16}
# qmax = fraction * 2^exponent, fraction in [0.5, 1)
QFRAC = {"e4m3": (0.875, 9), "int8": (0.9921875, 7)}
MIN_EXP = -64


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one layer's queries and keys of a few drafted tokens, which are in no cache yet
        dict(name="rope_drafts_b4_t16", op="rope", B=4, T=16, Hq=32, Hkv=8, rot=128, pairs="half", base=500000, ahead=30000, ragged=True),
        # a long chunk of two prompts, half of the dims rotated, neighbouring dims paired
        dict(name="rope_chunk_8k_partial", op="rope", B=2, T=8192, Hq=32, Hkv=8, rot=64, pairs="next", base=10000, ahead=1000000, ragged=False),
        # a 32K prompt goes into an empty paged cache, its queries rotated beside it
        dict(name="append_prefill_32k_paged", op="append", B=1, T=32768, Hq=32, Hkv=8, rot=128, pairs="half", base=500000, ahead=0, fmt="bf16", sblk=64, page=256, cap=32768, rows=False, fresh=True, ragged=False),
        # the accepted ones of 24 drafted tokens of each sequence go into an 8-bit cache
        dict(name="append_accepted_b32_e4m3", op="append", B=32, T=24, Hq=0, Hkv=8, rot=128, pairs="half", base=500000, ahead=0, fmt="e4m3", sblk=64, page=0, cap=256, rows=True, fresh=False, ragged=True),
        # the ancestors of one small tree
        dict(name="plan_b1_t16", op="plan", B=1, T=16, shape="tree", ragged=False),
        # of a large batch's trees of the largest size
        dict(name="plan_b64_t128", op="plan", B=64, T=128, shape="tree", ragged=True),
        # the smallest step: one token of one short sequence
        dict(name="attend_b1_t1_l2k", op="attend", B=1, T=1, Hq=32, Hkv=8, Lmax=2000, fmt="bf16", sblk=64, page=0, modes="full", sink=128, window=2048, shape="chain", ragged=False),
        # trees of 24 over 8-bit pages of different lengths, most heads streaming
        dict(name="attend_b8_t24_int8_paged", op="attend", B=8, T=24, Hq=32, Hkv=8, Lmax=30000, fmt="int8", sblk=64, page=64, modes="mix", sink=128, window=2048, shape="tree", ragged=True),
        # odd sizes, every kind of head, five query heads to a KV head
        dict(name="attend_b3_t61_e4m3_all", op="attend", B=3, T=61, Hq=20, Hkv=4, Lmax=20001, fmt="e4m3", sblk=32, page=0, modes="all", sink=100, window=1500, shape="tree", ragged=True),
        # the largest: trees of 32 over sixteen sequences of 64K, every head attending to all of its cache
        dict(name="attend_b16_t32_l64k_full", op="attend", B=16, T=32, Hq=32, Hkv=8, Lmax=65536, fmt="bf16", sblk=64, page=0, modes="full", sink=128, window=4096, shape="tree", ragged=False),
        # which path of one small tree stays
        dict(name="accept_b1_t16", op="accept", B=1, T=16, shape="tree", ragged=False),
        # of a large batch
        dict(name="accept_b64_t128", op="accept", B=64, T=128, shape="tree", ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _up(x, m):
    return -(-x // m) * m


def draw(rng):
    op = rng.choice(["rope", "append", "plan", "attend", "attend", "accept"])
    shape = rng.choice(["tree", "chain", "star"])
    ragged = rng.random() < 0.6
    if op in ("plan", "accept"):
        # (the ancestors of a token or two are always the same)
        return dict(op=op, B=_log(rng, 1, 64), T=_log(rng, 16 if op == "plan" else 1, 128), shape=shape, ragged=ragged)
    fmt = rng.choice(["bf16", "e4m3", "int8"])
    Hkv = rng.choice([1, 2, 4, 8])
    g = rng.randrange(1, 9)
    sblk = rng.choice([16, 32, 64, 128])
    page = rng.choice([0, 0, 64, 128, 256])
    if fmt != "bf16" and page:
        page = max(page, sblk)
    if op == "attend":
        B = _log(rng, 1, 32)
        T = _log(rng, 1, 128)
        Lmax = _log(rng, 1, 131072)
        Lmax = max(1, min(Lmax, 16 * 65536 * 8 // (B * Hkv), 16 * 65536 * 32 * 32 // (B * Hkv * g * T)))
        return dict(op=op, B=B, T=T, Hq=Hkv * g, Hkv=Hkv, Lmax=Lmax, fmt=fmt, sblk=sblk, page=page, modes=rng.choice(["full", "mix", "all"]),
                    sink=rng.randrange(0, 200), window=_log(rng, 1, 4096), shape=shape, ragged=ragged)
    B = _log(rng, 1, 64)
    T = max(1, min(_log(rng, 1, 32768), 32768 * 8 // (B * Hkv)))
    g = min(g, 4)
    rot = rng.choice([32, 64, 96, 128, 128])
    c = dict(op=op, B=B, T=T, Hq=Hkv * g, Hkv=Hkv, rot=rot, pairs=rng.choice(["half", "next"]), base=rng.choice([10000, 500000]), ahead=rng.choice([0, _log(rng, 1, 1000000)]), ragged=ragged)
    if op == "append":
        rows = T <= 128 and rng.random() < 0.5
        c.update(fmt=fmt, sblk=sblk, page=page, cap=_up(T + rng.randrange(0, 300), 256), rows=rows, fresh=rng.random() < 0.3)
        if rows or rng.random() < 0.2:
            c["Hq"] = 0
    return c


def _lens(B, most, ragged):
    """Lengths of a batch's sequences: all `most`, or spread over 0 .. most with an empty one and one of a single token among them."""
    if not ragged:
        return [most] * B
    v = [int(round(most * ((b * 0.6180339887 + 0.37) % 1.0))) for b in range(B)]
    v[0] = most
    if B > 1:
        v[1] = 0
    if B > 2:
        v[2] = min(1, most)
    return v


def _nodes(c):
    """Drafted tokens of each sequence: all T, or fewer (none in one of them)."""
    if not c["ragged"]:
        return [c["T"]] * c["B"]
    v = [1 + (b * 7919 + c["T"] - 1) % c["T"] for b in range(c["B"])]
    if c["B"] > 3:
        v[3] = 0
    return v


def _modes(c):
    if c["modes"] == "full":
        pick = lambda i: FULL  # noqa: E731
    elif c["modes"] == "mix":  # a quarter of the heads attends to everything
        pick = lambda i: FULL if i % 4 == 1 else SSA  # noqa: E731
    else:
        pick = lambda i: (BLOCK, FULL, SSA)[i % 3]  # noqa: E731
    return [[pick(b + h) for h in range(c["Hkv"])] for b in range(c["B"])]


def _new(c):
    """New tokens of each sequence of a rotation or an append."""
    if c["op"] == "append" and c["rows"]:
        return [0 if c["ragged"] and b == 3 else 1 + (b * 5) % c["T"] if c["ragged"] else c["T"] for b in range(c["B"])]
    return _lens(c["B"], c["T"], c["ragged"])


def _starts(c):
    if c["fresh"]:
        return [0] * c["B"]
    return [(b * 7919 + 37) % (c["cap"] - c["T"] + 1) for b in range(c["B"])]


def work(c):
    if c["op"] in ("plan", "accept"):
        n = sum(_nodes(c))
        return {"bytes": n * (24 if c["op"] == "plan" else 16) + 8 * c["B"], "flops": 0}
    if c["op"] == "attend":
        size = 512 if c["fmt"] == "bf16" else 256 + 8 / c["sblk"]
        total = flops = 0.0
        for ms, L, n in zip(_modes(c), _lens(c["B"], c["Lmax"], c["ragged"]), _nodes(c)):
            if n:
                for m in ms:
                    kept = min(L, c["sink"] + c["window"]) if m == SSA else L if m == FULL else L / 5
                    total += kept * size + n * 512
                    flops += 4 * D * (c["Hq"] // c["Hkv"]) * n * (kept + (n + 1) / 2)
                total += n * c["Hq"] * (4 * D + 4)
        return {"bytes": total, "flops": flops}
    n = sum(_new(c)) if c["op"] == "append" else c["B"] * c["T"]
    kv = 4 * c["Hkv"] if c["op"] == "rope" else 2 * c["Hkv"] * (4 if c["fmt"] == "bf16" else 3)
    return {"bytes": n * D * (4 * c["Hq"] + kv), "flops": 3 * n * c["rot"] * (c["Hq"] + c["Hkv"])}


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _tokens(shape, g):
    """Keys or values of a model: normal, the channels of different size, a few tokens much larger."""
    x = torch.randn(shape, generator=g, device="cuda")
    x *= 0.5 + torch.rand((shape[-2], shape[-1]), generator=g, device="cuda")
    big = torch.rand(shape[:-1], generator=g, device="cuda") < 0.01
    return (x * torch.where(big, 3.0, 1.0)[..., None]).to(torch.bfloat16)


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
    """x [L, H, D] float32 -> codes [L, H, D], scales [H, ceil(L / sblk)]."""
    L, H = x.shape[0], x.shape[1]
    n = -(-L // sblk)
    p = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, n * sblk - L)).view(n, sblk, H, D)
    s = _scale_of(p.abs().amax((1, 3)), fmt)
    codes = _round(p / s[:, None, :, None], fmt).view(n * sblk, H, D)[:L]
    return codes.contiguous(), s.transpose(0, 1).contiguous()


def _cache(B, L, Hkv, fmt, sblk, page, g, empty=False):
    """K and V of B sequences of L rows: codes [B, L, Hkv, D], scales [B, Hkv, n]; with `page`, in pages in a mixed order."""
    n = -(-L // sblk)
    parts = [torch.zeros((B, L, Hkv, D), dtype=DTYPE[fmt], device="cuda") for _ in range(2)]
    parts += [None if fmt == "bf16" else torch.zeros((B, Hkv, n), device="cuda") for _ in range(2)]
    for b in range(0 if empty else B):
        for i in range(2):
            x = _tokens((L, Hkv, D), g)
            if fmt == "bf16":
                parts[i][b] = x
            else:
                parts[i][b], parts[2 + i][b] = _quantize(x.float(), fmt, sblk)
    table = None
    if page:
        P = L // page
        table = torch.randperm(B * P + 3, generator=g, device="cuda")[: B * P].view(B, P)
        for i, t in enumerate(parts):
            if t is None:
                continue
            if i < 2:
                p = torch.zeros((B * P + 3, page, Hkv, D), dtype=t.dtype, device="cuda")
                _bits(p)[table.view(-1)] = _bits(t).view(B * P, page, Hkv, D)
            else:
                p = torch.full((B * P + 3, Hkv, page // sblk), 1.0, device="cuda")
                p[table.view(-1)] = t.view(B, Hkv, P, page // sblk).transpose(1, 2).reshape(B * P, Hkv, page // sblk)
            parts[i] = p
        table = table.to(torch.int32)
    return dict(K=parts[0], V=parts[1], ks=parts[2], vs=parts[3], table=table, sblk=sblk, fmt=fmt)


def _bits(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def _tree(c, g):
    """Parents [B, T] (-1: a root) of each sequence's drafted tokens, behind the last one -1."""
    B, T = c["B"], c["T"]
    t = torch.arange(T, device="cuda").expand(B, T)
    u = torch.rand((B, T), generator=g, device="cuda")
    if c["shape"] == "chain":  # one after the other, now and then from the root again
        p = torch.where(u < 0.05, 0, t - 1)
    elif c["shape"] == "star":  # most of them alternatives to one another
        p = torch.where(u < 0.9, 0, t - 1)
    else:  # any token before, the earlier ones likelier
        p = (t * u * u).long()
    p = torch.minimum(p, t - 1)
    n = _i32(_nodes(c))
    return torch.where(t < n[:, None], p, -1).to(torch.int32), n


def _inv_freq(c):
    i = torch.arange(c["rot"] // 2, dtype=torch.float64, device="cuda")
    return (float(c["base"]) ** (-2 * i / c["rot"])).float()


def _block_mask(c, cap, g):
    """[B, Hkv, n, n]: key block 0, the diagonal and a fifth of the others; one sequence's rows are empty."""
    n = -(-cap // 128)
    bm = torch.rand((c["B"], c["Hkv"], n, n), generator=g, device="cuda") < 0.2
    i = torch.arange(n, device="cuda")
    bm[:, :, i, i] = True
    bm[:, :, :, 0] = True
    if c["B"] > 4:
        bm[4] = False
    return (bm & (i[None, :] <= i[:, None])).to(torch.uint8)


def prepare(c, seed):
    g = _gen(seed)
    st = {"case": c}
    B, T = c["B"], c["T"]
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    if c["op"] == "plan":
        st["parents"], st["n"] = _tree(c, g)
        st["depth"], st["mask"] = z(B, T, t=torch.int32), z(B, T, 4, t=torch.int32)
    elif c["op"] == "accept":
        st["parents"], st["n"] = _tree(c, g)
        # few different tokens: siblings hold the same one now and then, and paths of all lengths are accepted
        st["tokens"] = torch.randint(0, 3, (B, T), generator=g, device="cuda").to(torch.int32)
        p = st["parents"].clamp(min=0).long()
        st["targets"] = torch.randint(0, 128000, (B, T), generator=g, device="cuda").to(torch.int32)
        some = torch.rand((B, T), generator=g, device="cuda") < 0.8
        # what the model says after a token is, mostly, what its first child holds
        kid = torch.full((B, T), T, device="cuda").scatter_reduce(1, p, torch.arange(T, device="cuda").expand(B, T).where(st["parents"] >= 0, T), "amin")
        st["targets"] = torch.where(some & (kid < T), st["tokens"].gather(1, kid.clamp(max=T - 1)), st["targets"])
    elif c["op"] == "attend":
        cap = _up(c["Lmax"] + T, c["page"] or 1)
        st["cache"] = _cache(B, cap, c["Hkv"], c["fmt"], c["sblk"], c["page"], g)
        st["Q"] = torch.randn((B, T, c["Hq"], D), generator=g, device="cuda").to(torch.bfloat16)
        st["K"], st["V"] = (_tokens((B, T, c["Hkv"], D), g) for _ in range(2))
        parents, st["n"] = _tree(c, g)
        st["depth"], st["mask"] = _plain_plan(parents, st["n"])
        st["lens"] = _i32(_lens(B, c["Lmax"], c["ragged"]))
        st["m"] = torch.tensor(_modes(c), dtype=torch.uint8, device="cuda")
        st["bm"] = _block_mask(c, cap, g) if c["modes"] == "all" else None
        st["O"], st["LSE"] = z(B, T, c["Hq"], D), z(B, c["Hq"], T, t=torch.float32)
    else:
        Hq, Hkv = c["Hq"], c["Hkv"]
        st["inv"] = _inv_freq(c)
        st["Q"] = torch.randn((B, T, Hq, D), generator=g, device="cuda").to(torch.bfloat16) if Hq else None
        st["K"] = _tokens((B, T, Hkv, D), g)
        st["n"] = _i32(_new(c))
        t = torch.arange(T, dtype=torch.int32, device="cuda")
        first = torch.randint(0, c["ahead"] + 1, (B, 1), generator=g, device="cuda").to(torch.int32)
        st["Qo"] = z(B, T, Hq, D) if Hq else None
        st["pos"] = first + t if c["op"] == "rope" or c["ahead"] else None
        if c["op"] == "rope":
            st["Ko"] = z(B, T, Hkv, D)
        else:
            st["V"] = _tokens((B, T, Hkv, D), g)
            st["cache"] = _cache(B, c["cap"], Hkv, c["fmt"], c["sblk"], c["page"], g, empty=c["fresh"])
            st["start"] = _i32(_starts(c))
            st["rows"] = None
            if c["rows"]:
                some = torch.rand((B, T), generator=g, device="cuda").argsort(1)
                st["rows"] = some.to(torch.int32).contiguous()
    return st


# ---------------------------------------------------------------- plain forms
def _rotate(x, pos, c, inv):
    """x [B, T, H, D] float32 rotated by positions [B, T]: the angles in 64 bits (positions reach far), the products in 32."""
    a = pos.double()[..., None] * inv.double()
    cos, sin = a.cos().float()[:, :, None], a.sin().float()[:, :, None]
    r = c["rot"]
    y = x.clone()
    if c["pairs"] == "half":
        u, v = x[..., : r // 2], x[..., r // 2 : r]
        y[..., : r // 2], y[..., r // 2 : r] = u * cos - v * sin, v * cos + u * sin
    else:
        u, v = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = u * cos - v * sin, v * cos + u * sin
    return y


def _plain_rope(st):
    c = st["case"]
    live = (torch.arange(c["T"], device="cuda") < st["n"][:, None])[..., None, None]
    return [torch.where(live, _rotate(x.float(), st["pos"], c, st["inv"]).to(torch.bfloat16), o) for x, o in ((st["Q"], st["Qo"]), (st["K"], st["Ko"]))]


def _take(x, rows):
    return x if rows is None else x.gather(1, rows.long()[..., None, None].expand(-1, -1, *x.shape[2:]))


def _plain_append(st):
    c, cache = st["case"], st["cache"]
    fmt, table, B, T, cap = c["fmt"], cache["table"], c["B"], c["T"], c["cap"]
    sblk = c["sblk"] if fmt != "bf16" else 1
    start, n = st["start"].long()[:, None], st["n"].long()[:, None]
    t = torch.arange(T, device="cuda")
    pos = start + t if st["pos"] is None else _take(st["pos"][..., None, None], st["rows"])[..., 0, 0].long()
    new = _rotate(_take(st["K"], st["rows"]).float(), pos, c, st["inv"]), _take(st["V"], st["rows"]).float()
    R = min(-(-(T + sblk - 1) // sblk) * sblk, cap)                   # rows of whole blocks that hold the new tokens
    r0 = torch.clamp(start // sblk * sblk, max=cap - R)
    at = r0 + torch.arange(R, device="cuda")                          # [B, R]
    outer, row = (torch.arange(B, device="cuda")[:, None].expand(-1, R), at) if table is None else (table.long().gather(1, at // c["page"]), at % c["page"])
    fresh = (at >= start) & (at < start + n)
    touched = fresh.view(B, -1, sblk).any(-1)                         # [B, R / sblk]
    before = ((at < start).view(B, -1, sblk).any(-1) & touched)[..., None]
    for codes, scales, x in ((cache["K"], cache["ks"], new[0]), (cache["V"], cache["vs"], new[1])):
        raw = _bits(codes)
        old = raw[outer, row]                                         # [B, R, Hkv, D]
        x = torch.where(fresh[..., None, None], x.gather(1, (at - start).clamp(0, T - 1)[..., None, None].expand(-1, -1, c["Hkv"], D)), 0.0)
        if fmt == "bf16":
            raw[outer, row] = torch.where(fresh[..., None, None], x.to(torch.bfloat16), old)
            continue
        so = outer.view(B, -1, sblk)[..., 0], row.view(B, -1, sblk)[..., 0] // sblk
        s_old = scales[so[0], :, so[1]]                               # [B, nb, Hkv]
        s = _scale_of(x.abs().view(B, -1, sblk, c["Hkv"], D).amax((2, 4)), fmt)
        s = torch.where(before, torch.maximum(s, s_old), s)
        s = torch.where(touched[..., None], s, s_old)
        wide = lambda v: v.repeat_interleave(sblk, 1)[..., None]  # noqa: E731
        grown = wide((s != s_old) & before)
        value = torch.where(fresh[..., None, None], x / wide(s), old.view(codes.dtype).float() * torch.where(grown, wide(s_old) / wide(s), 1.0))
        stay = (~fresh)[..., None, None] & ((at >= start)[..., None, None] | ~grown)
        raw[outer, row] = torch.where(stay, old, _bits(_round(value, fmt)))
        scales[so[0], :, so[1]] = s
    if not c["Hq"]:
        return _cache_out(cache)
    q = _rotate(st["Q"].float(), start + t if st["pos"] is None else st["pos"], c, st["inv"]).to(torch.bfloat16)
    return [torch.where((t < n)[..., None, None], q, st["Qo"])] + _cache_out(cache)


def _per_row(s, sblk, rows):
    return s.transpose(-1, -2).repeat_interleave(sblk, -2)[..., :rows, :]


def _cache_out(cache):
    """The cache, an 8-bit one as the values that its codes stand for (exact in bfloat16)."""
    if cache["fmt"] == "bf16":
        return [cache["K"], cache["V"]]
    return [cache[t].to(torch.bfloat16) * _per_row(cache[s], cache["sblk"], cache[t].shape[1])[..., None].to(torch.bfloat16) for t, s in (("K", "ks"), ("V", "vs"))]


def _adjacent(parents, n):
    """[B, T, T] float32: 1 where the second node is the first one's parent, or itself."""
    T = parents.shape[1]
    t = torch.arange(T, device=parents.device)
    a = (parents[..., None] == t) | (t[:, None] == t)
    return (a & (t < n[:, None])[..., None]).float()


def _closure(parents, n):
    """[B, T, T] bool: the second node is the first one's ancestor, or itself (squared until every path is in it)."""
    a = _adjacent(parents, n)
    for _ in range(max(1, (parents.shape[1] - 1).bit_length())):
        a = (torch.matmul(a, a) > 0).float()
    return a > 0


def _plain_plan(parents, n):
    """Depth [B, T] and ancestors (and itself) as bits [B, T, 4]; zeros behind a sequence's last node."""
    B, T = parents.shape
    up = _closure(parents, n)
    depth = (up.sum(-1) - 1).clamp(min=0).to(torch.int32)
    bits = torch.nn.functional.pad(up, (0, 128 - T)).view(B, T, 4, 32).long() << torch.arange(32, device=parents.device)
    bits = bits.sum(-1)
    return depth, torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32)


def _plain_accept(st):
    parents, tokens, targets, n = st["parents"].long(), st["tokens"], st["targets"], st["n"].long()
    B, T = parents.shape
    t = torch.arange(T, device="cuda")
    live = t < n[:, None]
    hit = live & (parents >= 0) & (tokens == targets.gather(1, parents.clamp(min=0)))
    # of siblings that hit, the first
    same = (parents[:, :, None] == parents[:, None, :]) & hit[:, None, :] & (t < t[:, None])
    good = (hit & ~same.any(-1)) | ((t == 0) & live)
    up = _closure(parents, n)
    ok = live & ~(up & ~good[:, None, :]).any(-1)
    depth = (up.sum(-1) - 1).clamp(min=0)
    count = ok.sum(-1)
    path = torch.full((B, T + 1), -1, dtype=torch.long, device="cuda").scatter(1, torch.where(ok, depth, T), t.expand(B, T))[:, :T]
    path = torch.where(t < count[:, None], path, -1)
    last = path.gather(1, (count - 1).clamp(min=0)[:, None])
    token = torch.where(count > 0, targets.gather(1, last.clamp(min=0))[:, 0], -1)
    return [path.to(torch.int32), count.to(torch.int32), token.to(torch.int32)]


def _unpaged(t, table):
    """Pages [P, page, H, D] (or scales [P, H, k]) as contiguous sequences."""
    if t is None or table is None:
        return t
    B, n = table.shape
    x = _bits(t)[table.view(-1).long()]
    if t.dim() == 4:
        return x.view(B, n * t.shape[1], t.shape[2], D).view(t.dtype)
    return x.view(B, n, t.shape[1], t.shape[2]).transpose(1, 2).reshape(B, t.shape[1], n * t.shape[2])


def _values(cache, key, dtype):
    """K or V of a cache as numbers [B, L, Hkv, D]."""
    x = _unpaged(cache[key], cache["table"]).to(dtype)
    s = _unpaged(cache["ks" if key == "K" else "vs"], cache["table"])
    return x if s is None else x.mul_(_per_row(s, cache["sblk"], x.shape[1])[..., None])


def _keep(st, b0, b1, L):
    """[b, Hkv, T, L + T] bool: the cache's keys and the drafted ones that each drafted token of sequences b0 .. b1 - 1 keeps."""
    c = st["case"]
    T = c["T"]
    lens, depth, m, n = (st[k][b0:b1] for k in ("lens", "depth", "m", "n"))
    pos = (lens[:, None] + depth).long()                                     # [b, T]
    j = torch.arange(L, device="cuda").expand(len(lens), L)
    at = torch.cat([j, pos], 1)                                              # positions of the keys [b, L + T]
    bits = (st["mask"][b0:b1, :, :, None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
    t = torch.arange(T, device="cuda")
    up = bits.reshape(len(lens), T, 128)[..., :T].bool() & (t < n[:, None])[:, None, :]
    there = torch.cat([(j < lens[:, None])[:, None, :].expand(-1, T, -1), up], 2)[:, None]
    i, k = pos[:, None, :, None], at[:, None, None, :]
    mode = m[:, :, None, None]
    keep = there & ((mode != SSA) | (k < c["sink"]) | (i - k < c["window"]))
    if st["bm"] is not None:
        bm = st["bm"][b0:b1]
        top = bm.shape[2] - 1
        rows = torch.gather(bm, 2, (pos // 128).clamp(max=top)[:, None, :, None].expand(-1, bm.shape[1], -1, bm.shape[3]))
        picked = torch.gather(rows, 3, (at // 128).clamp(max=top)[:, None, None, :].expand(-1, bm.shape[1], T, -1))
        keep &= (mode != BLOCK) | (picked != 0)
    return keep


def _plain_attend(st):
    c = st["case"]
    B, T, Hkv, g = c["B"], c["T"], c["Hkv"], c["Hq"] // c["Hkv"]
    K, V = (torch.cat([_values(st["cache"], x, torch.float32), st[x].float()], 1) for x in ("K", "V"))
    L = K.shape[1] - T
    # what lies behind a sequence's tokens counts as nothing, whatever it holds
    j = torch.arange(L, device="cuda")
    t = torch.arange(T, device="cuda")
    real = torch.cat([j < st["lens"][:, None], t < st["n"][:, None]], 1)[..., None, None]
    V = torch.where(real, V, 0.0)
    q = st["Q"].float().view(B, T, Hkv, g, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, g * T, D)
    s = torch.matmul(q, K.permute(0, 2, 3, 1)).mul_(D**-0.5).view(B, Hkv, g, T, L + T)
    s.masked_fill_(~_keep(st, 0, B, L)[:, :, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = s.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    O = torch.matmul(p.view(B, Hkv, g * T, L + T), V.permute(0, 2, 1, 3)).view(B, Hkv, g, T, D) / total.masked_fill(total == 0, 1.0)
    LSE = (top + torch.log(total))[..., 0].view(B, c["Hq"], T)
    O = O.permute(0, 3, 1, 2, 4).reshape(B, T, c["Hq"], D).to(torch.bfloat16)
    live = t < st["n"][:, None]
    return [torch.where(live[..., None, None], O, st["O"]), torch.where(live[:, None], LSE, st["LSE"])]


# ---------------------------------------------------------------- the framework's calls
def _handle(st, ea):
    """The cache's handle, which a user's program makes once."""
    if "handle" not in st:
        k = st["cache"]
        st["handle"] = ea.KVCache(k["K"], k["V"], k["ks"], k["vs"], scale_block=k["sblk"], block_table=k["table"])
    return st["handle"]


def _workspace(st, make):
    """The call's workspace, which a user's program keeps."""
    if "workspace" not in st:
        st["workspace"] = make()
    return st["workspace"]


def run(st):
    c = st["case"]
    if not own:
        if c["op"] == "rope":
            return _plain_rope(st)
        if c["op"] == "append":
            return _plain_append(st)
        if c["op"] == "plan":
            return list(_plain_plan(st["parents"], st["n"]))
        return _plain_attend(st) if c["op"] == "attend" else _plain_accept(st)
    import sparse_head_attention_gb300 as ea

    if c["op"] == "rope":
        return ea.ea_rope(st["Q"], st["K"], st["pos"], st["inv"], n_new=st["n"], interleaved=c["pairs"] == "next", Q_out=st["Qo"], K_out=st["Ko"],
                          workspace=_workspace(st, ea.cache_workspace))
    if c["op"] == "append":
        q = ea.ea_cache_write_rope(_handle(st, ea), st["K"], st["V"], st["inv"], Q=st["Q"], Q_out=st["Qo"], start=st["start"], n_new=st["n"], rows=st["rows"],
                                   positions=st["pos"], interleaved=c["pairs"] == "next", workspace=_workspace(st, ea.cache_workspace))
        return ([q] if c["Hq"] else []) + _cache_out(st["cache"])
    if c["op"] == "plan":
        return list(ea.ea_tree_plan(st["parents"], st["n"], depth=st["depth"], mask=st["mask"], workspace=_workspace(st, ea.cache_workspace)))
    if c["op"] == "accept":
        return list(ea.ea_tree_accept(st["tokens"], st["parents"], st["targets"], st["n"], workspace=_workspace(st, ea.cache_workspace)))
    cache = _handle(st, ea)
    return list(ea.ea_hybrid_attn_tree(st["Q"], st["K"], st["V"], cache, st["lens"], st["depth"], st["mask"], st["m"], sink=c["sink"], window=c["window"], n_nodes=st["n"],
                                       block_mask=st["bm"], O=st["O"], LSE=st["LSE"],
                                       workspace=_workspace(st, lambda: ea.tree_workspace(c["B"], c["T"], c["Hq"], c["Hkv"], cache.capacity))))


# ---------------------------------------------------------------- in 64 bits
def _turn(x, angle, c):
    """x [..., D] float64 rotated by angles [..., rot / 2], as complex numbers."""
    r = c["rot"]
    part = x[..., :r]
    pairs = part.unflatten(-1, (2, r // 2)).transpose(-1, -2) if c["pairs"] == "half" else part.unflatten(-1, (r // 2, 2))
    z = torch.complex(pairs[..., 0].contiguous(), pairs[..., 1].contiguous()) * torch.polar(torch.ones_like(angle), angle)
    back = torch.view_as_real(z)
    back = back.transpose(-1, -2).flatten(-2) if c["pairs"] == "half" else back.flatten(-2)
    return torch.cat([back, x[..., r:]], -1)


def _exact_append(st):
    c, cache = st["case"], st["cache"]
    inv = st["inv"].double()
    out = []
    starts, counts = _starts(c), _new(c)
    if c["Hq"]:
        q = st["Qo"].double()
        for b in range(c["B"]):
            n = counts[b]
            pos = st["pos"][b, :n].double() if st["pos"] is not None else starts[b] + torch.arange(n, device="cuda").double()
            q[b, :n] = _turn(st["Q"][b, :n].double(), (pos[:, None] * inv)[:, None, :], c)
        out.append(q)
    for key in ("K", "V"):
        sk = "ks" if key == "K" else "vs"
        full = cache[key].double()
        if cache[sk] is not None:
            full *= _per_row(cache[sk], c["sblk"], full.shape[1])[..., None].double()
        for b in range(c["B"]):
            n = counts[b]
            idx = st["rows"][b, :n].long() if st["rows"] is not None else torch.arange(n, device="cuda")
            x = st[key][b].double()[idx]
            if key == "K":
                pos = st["pos"][b][idx].double() if st["pos"] is not None else starts[b] + torch.arange(n, device="cuda").double()
                x = _turn(x, (pos[:, None] * inv)[:, None, :], c)
            page = c["page"] or c["cap"]
            step = page if c["fmt"] == "bf16" else c["sblk"]
            lo = starts[b]
            while lo < starts[b] + n:
                first = lo // step * step
                hi = min(first + step, starts[b] + n)
                o = b if cache["table"] is None else int(cache["table"][b, first // page])
                r = first % page
                new = x[lo - starts[b] : hi - starts[b]]
                if c["fmt"] == "bf16":
                    full[o, r + lo - first : r + hi - first] = new
                else:
                    s = _scale_of(new.abs().amax((0, 2)).float(), c["fmt"]).double()
                    was = cache[sk][o, :, r // step].double()
                    if lo > first:
                        s = torch.maximum(s, was)
                    grown = s > was
                    held = full[o, r : r + lo - first]
                    full[o, r : r + lo - first] = torch.where(grown[:, None], _round((held / s[:, None]).float(), c["fmt"]).double() * s[:, None], held)
                    full[o, r + lo - first : r + hi - first] = _round((new / s[:, None]).float(), c["fmt"]).double() * s[:, None]
                    # the rows behind keep their codes, under the block's scale
                    codes = cache[key][o, r + hi - first : r + step].double()
                    full[o, r + hi - first : r + step] = codes * s[:, None]
                lo = hi
        out.append(full)
    return out


def _exact_attend(st):
    c = st["case"]
    g, T = c["Hq"] // c["Hkv"], c["T"]
    O, LSE = st["O"].double(), st["LSE"].double()
    k = st["cache"]
    for b, (L, n) in enumerate(zip(_lens(c["B"], c["Lmax"], c["ragged"]), _nodes(c))):
        if not n:
            continue
        one = dict(k, K=k["K"][b : b + 1], V=k["V"][b : b + 1], ks=None if k["ks"] is None else k["ks"][b : b + 1], vs=None if k["vs"] is None else k["vs"][b : b + 1])
        if k["table"] is not None:
            one = dict(k, table=k["table"][b : b + 1])
        keep = _keep(st, b, b + 1, L)[0]
        K, V = (torch.cat([_values(one, x, torch.float64)[0, :L], st[x][b].double()]) for x in ("K", "V"))
        for h in range(c["Hkv"]):
            q = st["Q"][b, :n, h * g : (h + 1) * g].double()
            x = torch.einsum("tgd,kd->gtk", q, K[:, h]) / math.sqrt(D)
            x = x.masked_fill(~keep[h, :n], -math.inf)
            lse = torch.logsumexp(x, -1)
            p = torch.exp(x - lse[..., None]).nan_to_num(nan=0.0)
            v = V[:, h].clone()
            v[L + n :] = 0.0
            O[b, :n, h * g : (h + 1) * g] = torch.einsum("gtk,kd->tgd", p, v)
            LSE[b, h * g : (h + 1) * g, :n] = lse
    return [O, LSE]


def exact(c, seed):
    st = prepare(c, seed)
    if c["op"] == "rope":
        out = []
        for x, o in ((st["Q"], st["Qo"]), (st["K"], st["Ko"])):
            y = _turn(x.double(), (st["pos"].double()[..., None] * st["inv"].double())[:, :, None, :], c)
            live = torch.arange(c["T"], device="cuda") < st["n"][:, None]
            out.append(torch.where(live[..., None, None], y, o.double()))
        return out
    if c["op"] == "append":
        return _exact_append(st)
    return _exact_attend(st) if c["op"] == "attend" else None
