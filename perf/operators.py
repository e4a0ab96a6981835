"""Cases that measure the token-by-token (decode) operators of the library.

Five operators on a paged K/V cache whose pages are one selection block each:

  append  K and V rows of new tokens quantised into the cache, with the summaries of the blocks
          they complete, and the written tokens read back as the values they stand for
  read    the values a range of cached tokens stands for
  select  the kept blocks of single query tokens, from the block summaries
  attn    attention of single query tokens over given kept blocks, from the quantised pages
  decode  select and attn as one call

`run` computes them in plain torch operations on the same buffers, or with `own` set calls the
library. The record of one (page, kv head) is block/16 tiles of 16 tokens; a tile is the K codes,
the V codes and, at 4 and 8 bits, 16 rows of bfloat16 scales (K groups, then V groups, of 32
channels each). The order of the codes inside a tile is `_order` below.
"""

import functools
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
BITS = {"bf16": 16, "q8": 8, "q4": 4}
GROUP = 32  # channels that share a scale
TILE = 16  # tokens of a tile

# Head layouts, block sizes and budgets are those of the library's own workloads: 32 query and 8
# kv heads of 128 (block 128), 28 and 4, and 2 and 2 of 64 (block 64).


def _case(name, op, fmt, nseq, Hq, Hkv, D, block, length, ragged=False, T=1, share="group",
          metric="product", vsum="mean", rho=0.05, tau=64.0, kmin=8, draft=1):
    c = dict(op=op, fmt=fmt, nseq=nseq, Hq=Hq, Hkv=Hkv, D=D, block=block, length=length,
             ragged=ragged, T=T, share=share, metric=metric, vsum=vsum, rho=rho, tau=tau,
             kmin=kmin, draft=draft)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one new token of each of 16 conversations: what every generated token pays in a layer
        _case("append-step-q4", "append", "q4", 16, 32, 8, 128, 128, 16384, ragged=True, T=1),
        # chunks of several prompts prefilled together, ragged, small heads
        _case("append-chunks-q8", "append", "q8", 8, 16, 8, 64, 64, 8192, ragged=True, T=1999,
              vsum="max"),
        # the K and V of a whole long prompt go to the cache after its prefill
        _case("append-prompt-bf16", "append", "bf16", 1, 32, 8, 128, 128, 131072, T=131072),
        # a 4-bit sequence read back for a dense step or a copy to another cache
        _case("read-32k-q4", "read", "q4", 1, 32, 8, 128, 128, 32768, T=32768),
        # parts of several 8-bit sequences read back
        _case("read-ragged-q8", "read", "q8", 6, 28, 4, 128, 128, 9000, ragged=True, T=3001),
        # the block choice of one token at the end of a 128K context
        _case("select-128k-b1", "select", "q4", 1, 32, 8, 128, 128, 131072),
        # a batch of ragged contexts, a list for each head, the additive metric
        _case("select-ragged-b32", "select", "q8", 32, 28, 4, 128, 64, 65536, ragged=True,
              share="head", metric="additive", vsum="max", rho=0.1, tau=48.0, kmin=4),
        # one token at 128K over its kept blocks of a 4-bit cache
        _case("attn-128k-b1-q4", "attn", "q4", 1, 32, 8, 128, 128, 131072),
        # a batch with a list for each head, 16-bit pages
        _case("attn-ragged-b32-bf16", "attn", "bf16", 32, 32, 8, 128, 128, 16384, ragged=True,
              share="head", rho=0.1, tau=32.0, kmin=4),
        # every block kept (rho 1): dense attention over an 8-bit cache
        _case("attn-dense-64k-q8", "attn", "q8", 4, 28, 4, 128, 128, 65536, ragged=True, rho=1.0),
        # a short context of small heads: the smallest call of the whole step
        _case("decode-1k-b1-bf16", "decode", "bf16", 1, 2, 2, 64, 64, 1000, share="head",
              rho=0.25, tau=4.0, kmin=2),
        # a serving batch with two draft tokens a sequence, 4-bit pages
        _case("decode-32k-b32-q4", "decode", "q4", 32, 32, 8, 128, 128, 32768, ragged=True,
              rho=0.1, tau=32.0, kmin=4, draft=2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "select", "attn", "attn", "decode", "decode"])
    fmt = rng.choice(["bf16", "q8", "q4"])
    D, block = rng.choice([64, 128]), rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 5, 7, 8])
    nseq = _log(rng, 1, 32)
    # the cached tokens of all sequences stay below those of the largest listed cases
    length = _log(rng, 100, min(131072, 4194304 // (nseq * Hkv)))
    T = 1
    if op in ("append", "read"):
        T = 1 if rng.random() < 0.25 else _log(rng, 1, length)
    dense = op == "attn" and nseq * length * Hkv <= 1048576 and rng.random() < 0.3
    return _case(None, op, fmt, nseq, Hq, Hkv, D, block, length, ragged=rng.random() < 0.7, T=T,
                 share=rng.choice(["head", "group"]), metric=rng.choice(["product", "additive"]),
                 vsum=rng.choice(["mean", "max"]), rho=1.0 if dense else rng.choice([0.05, 0.1, 0.2]),
                 tau=rng.choice([4.0, 16.0, 32.0]), kmin=rng.choice([2, 4, 8]),
                 draft=rng.choice([1, 1, 2, 4]))


# ------------------------------------------------------------------ sizes that a case fixes

BETA = 0.2  # weight of the V magnitude in the additive metric


def _lengths(c):
    """Cached tokens of each sequence (new ones included): ragged ones spread from 1 to length."""
    if not c["ragged"]:
        return [c["length"]] * c["nseq"]
    r = random.Random(c["length"] * 131 + c["nseq"])
    return [c["length"] if s == 0 else r.randint(1, c["length"]) for s in range(c["nseq"])]


def _counts(c):
    """New (or read) tokens of each sequence: at most T, at most the length; one may be 0."""
    r = random.Random(c["length"] * 17 + c["nseq"])
    out = []
    for s, n in enumerate(_lengths(c)):
        top = min(c["T"], n)
        out.append(r.randint(0, top) if c["ragged"] and c["T"] > 1 and s else top)
    return out


def _budget(c):
    """k(i) for every block index of the longest sequence: the exponential schedule."""
    nb = -(-c["length"] // c["block"])
    ks = []
    for i in range(nb):
        rho = c["rho"] + (1.0 - c["rho"]) * math.exp(-i / c["tau"])
        k = min(max(math.ceil(rho * (i + 1)), c["kmin"]), i + 1)
        ks.append(1 if i == 0 else max(2, k))
    return ks


def _rows(c):
    """(sequence, visible tokens) of each query row: a sequence's draft tokens see one more each."""
    rows = []
    for s, n in enumerate(_lengths(c)):
        rows += [(s, max(n - c["draft"] + 1 + t, 0)) for t in range(c["draft"])]
    return rows


def _record(c):
    per = TILE * c["D"] * 2 * BITS[c["fmt"]] // 8
    if c["fmt"] != "bf16":
        per += TILE * 2 * (c["D"] // GROUP) * 2
    return per * (c["block"] // TILE)


def work(case):
    c = case
    D, Hq, Hkv, block, G = c["D"], c["Hq"], c["Hkv"], c["block"], c["Hq"] // c["Hkv"]
    row = 2 * D * Hkv  # elements of one token's K and V
    cached = _record(c) * Hkv / block  # bytes of one token in the cache
    if c["op"] in ("append", "read"):
        n = sum(_counts(c))
        blocks = 0
        for t, k in zip(_lengths(c), _counts(c)):
            blocks += t // block - (t - k) // block
        if c["op"] == "read":
            return {"bytes": n * (cached + 2 * row), "flops": n * row}
        # rows in, codes out, and values out
        return {"bytes": n * (2 * row + cached + 2 * row) + blocks * Hkv * (4 * D + 4),
                "flops": 6.0 * n * row}
    ks, nbytes, flops, seen = _budget(c), 0.0, 0.0, {}
    for s, n in _rows(c):
        if n == 0:
            continue
        i = -(-n // block) - 1
        k = ks[i]
        if c["op"] != "attn":
            flops += 2.0 * Hq * i * D
            if s not in seen:  # the draft tokens of a sequence read the same summaries
                nbytes += i * Hkv * (4 * D + 4)
            nbytes += 4 * Hq * k
        if c["op"] != "select":
            flops += 4.0 * Hq * k * block * D
            # distinct blocks a kv head reads, its heads and draft tokens choosing apart by chance
            kinds = c["draft"] * (G if c["share"] == "head" else 1)
            if s not in seen:
                free = max(i - 1, 0)
                some = free * (1.0 - (1.0 - (max(k - 2, 0) / free)) ** kinds) if free else 0.0
                full = some + min(i, 1)
                nbytes += (full * block + n - i * block) * cached
            nbytes += 2 * 2 * Hq * D + 4 * Hq
        seen[s] = True
    return {"bytes": nbytes, "flops": flops}


# ------------------------------------------------------------------ the cache's layout


@functools.lru_cache(maxsize=None)
def _order(fmt, D, what):
    """For each element position of a tile's K or V codes: token * D + channel."""
    ng, words = D // GROUP, {"q4": 1, "q8": 2, "bf16": 4}[fmt]  # words of a lane's row and group
    per = 32 // BITS[fmt]  # elements of a 32-bit word
    out = np.full(TILE * D, -1, dtype=np.int64)
    for r in range(TILE):
        for d in range(D):
            g, x = d // GROUP, d % GROUP
            if what == "k":  # lane: token r % 8, channels 8 lane..8 lane + 7 of the group
                i, lane, e = r // 8, (r % 8) * 4 + x // 8, x % 8
                w, p = {"q4": (0, e // 2 + 4 * (e % 2)), "q8": (e // 4, (0, 2, 1, 3)[e % 4]),
                        "bf16": (e // 2, e % 2)}[fmt]
            else:  # lane: token pair, channels 4 lane..4 lane + 3 of the group
                i, lane, e, y = r // 8, (x // 4) * 4 + (r % 8) // 2, x % 4, r % 2
                w, p = {"q4": (0, 4 * y + e), "q8": (e // 2, 2 * y + e % 2), "bf16": (e, y)}[fmt]
            n = (i * ng + g) * words + w
            out[(((n // 4) * 32 + lane) * 4 + n % 4) * per + p] = r * D + d
    assert (out >= 0).all()
    return out


@functools.lru_cache(maxsize=None)
def _index(fmt, D, what, back):
    o = _order(fmt, D, what)
    return torch.from_numpy(np.argsort(o) if back else o).to(DEV)


def _quantise(x, fmt):
    """Codes (int) and scales of x [..., D], groups of 32 channels."""
    top = 7 if fmt == "q4" else 127
    g = x.float().unflatten(-1, (-1, GROUP))
    amax = g.abs().amax(-1)
    s = (amax / top).to(torch.bfloat16)
    s = torch.where(torch.isfinite(amax), s, torch.full_like(s, float("nan")))
    f = s.float()[..., None]
    c = torch.where(f > 0, torch.round(g / f).clamp(-top, top), torch.zeros_like(g))
    return c.flatten(-2).to(torch.int32), s


def _dequantise(c, s):
    return (c.float().unflatten(-1, (-1, GROUP)) * s.float()[..., None]).flatten(-2)


def _pack(k, v, fmt):
    """Records [..., bytes] of k and v [..., block, D] bfloat16."""
    D = k.shape[-1]
    parts, scales = [], []
    for what, x in (("k", k), ("v", v)):
        idx = _index(fmt, D, what, False)
        if fmt == "bf16":
            e = x.unflatten(-2, (-1, TILE)).flatten(-2)[..., idx]
            parts.append(e.contiguous().view(torch.uint8))
            continue
        c, s = _quantise(x, fmt)
        scales.append(s.unflatten(-2, (-1, TILE)))
        e = c.unflatten(-2, (-1, TILE)).flatten(-2)[..., idx] + (8 if fmt == "q4" else 128)
        if fmt == "q4":
            e = e[..., 0::2] | (e[..., 1::2] << 4)
        parts.append(e.to(torch.uint8))
    if scales:
        parts.append(torch.cat(scales, -1).contiguous().flatten(-2).view(torch.uint8))
    return torch.cat(parts, -1).flatten(-2)


def _unpack(rec, fmt, D):
    """K and V [..., block, D] float32 of records [..., bytes]."""
    size = TILE * D * BITS[fmt] // 8
    ng = D // GROUP
    t = rec.unflatten(-1, (-1, rec.shape[-1] // _tiles(rec, fmt, D)))
    out = []
    if fmt != "bf16":
        sc = t[..., 2 * size:].contiguous().view(torch.bfloat16).unflatten(-1, (TILE, 2 * ng))
    for n, what in enumerate("kv"):
        e = t[..., n * size:(n + 1) * size].contiguous()
        if fmt == "bf16":
            x = e.view(torch.bfloat16).float()
        elif fmt == "q4":
            x = torch.stack((e & 15, e >> 4), -1).flatten(-2).float() - 8.0
        else:
            x = e.float() - 128.0
        x = x[..., _index(fmt, D, what, True)].unflatten(-1, (TILE, D))
        if fmt != "bf16":
            x = _dequantise(x, sc[..., n * ng:(n + 1) * ng])
        out.append(x.flatten(-3, -2))
    return out


def _tiles(rec, fmt, D):
    per = TILE * D * 2 * BITS[fmt] // 8 + (0 if fmt == "bf16" else TILE * 4 * (D // GROUP))
    return rec.shape[-1] // per


def _summaries(k, v, vsum):
    n = v.square().sum(-1).sqrt()
    return k.mean(-2), n.amax(-1) if vsum == "max" else n.mean(-1)


# ------------------------------------------------------------------ inputs


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV).manual_seed(seed * 7919 + 11)
    D, Hq, Hkv, block, fmt = c["D"], c["Hq"], c["Hkv"], c["block"], c["fmt"]
    lens = _lengths(c)
    nb = -(-c["length"] // block)
    need = [-(-n // block) for n in lens]
    pages = sum(need) + 3

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((c["nseq"], nb), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = torch.arange(at, at + n, dtype=torch.int32)
        at += n
    table = torch.where(table.to(DEV) < 0, -1, order[table.to(DEV).long().clamp(min=0)])

    # keys: some channels with an offset and a larger spread, every block with a drift of its
    # own (so that blocks score apart); values: a few rows of large norm
    spread = torch.exp(0.4 * normal(Hkv, 1, D))
    offset = 0.5 * normal(Hkv, 1, D)
    store = torch.empty(pages, Hkv, _record(c), dtype=torch.uint8, device=DEV)
    kbar = torch.empty(pages, Hkv, D, device=DEV)
    vnorm = torch.empty(pages, Hkv, device=DEV)

    def rows(n, tokens):
        k = normal(n, Hkv, tokens, D) * spread + offset + 0.4 * normal(n, Hkv, 1, D)
        v = normal(n, Hkv, tokens, D)
        v = v * torch.where(torch.rand(n, Hkv, tokens, 1, generator=gen, device=DEV) < 0.01,
                            5.0, 1.0) * torch.exp(0.3 * normal(n, Hkv, 1, 1))
        return k.to(torch.bfloat16), v.to(torch.bfloat16)

    step = max(1, (1 << 25) // (Hkv * block * D))
    for a in range(0, pages, step):
        b = min(a + step, pages)
        k, v = rows(b - a, block)
        store[a:b] = _pack(k, v, fmt)
        kbar[a:b], vnorm[a:b] = _summaries(*_unpack(store[a:b], fmt, D), c["vsum"])

    st = dict(case=c, pages=store, kbar=kbar, vnorm=vnorm, table=table)
    if c["op"] in ("append", "read"):
        n = _counts(c)
        T = max(max(n), 1)
        st["pos"] = torch.tensor([a - b for a, b in zip(lens, n)], dtype=torch.int32, device=DEV)
        st["count"] = torch.tensor(n, dtype=torch.int32, device=DEV)
        st["k"] = torch.zeros(c["nseq"], Hkv, T, D, dtype=torch.bfloat16, device=DEV)
        st["v"] = torch.zeros_like(st["k"])
        if c["op"] == "append":
            # a projection's output, token-major, seen as [sequence, head, token, channel]
            k, v = rows(c["nseq"], T)
            st["k_new"] = k.transpose(1, 2).contiguous().transpose(1, 2)
            st["v_new"] = v.transpose(1, 2).contiguous().transpose(1, 2)
        return st
    r = _rows(c)
    R = len(r)
    st["q"] = (normal(R, Hq, D) * 1.2).to(torch.bfloat16)
    st["rows"] = torch.tensor([s for s, _ in r], dtype=torch.int32, device=DEV)
    st["lens"] = torch.tensor([n for _, n in r], dtype=torch.int32, device=DEV)
    ks = _budget(c)
    st["budget"] = torch.tensor(ks, dtype=torch.int32, device=DEV)
    st["kcap"] = max(ks)
    if c["op"] == "attn":  # lists as a selection leaves them
        st["sel_idx"], st["sel_cnt"] = _lists(st, torch.rand(
            R, Hkv if c["share"] == "group" else Hq, nb, generator=gen, device=DEV,
            dtype=torch.float64))
    return st


# ------------------------------------------------------------------ the plain forms


def _lists(st, key):
    """Kept blocks by descending key [R, lists, nb]: (sel_idx [R, Hq, kcap], sel_cnt [R, Hq])."""
    c, lens = st["case"], st["lens"].long()
    nb, kcap = key.shape[-1], st["kcap"]
    last = (lens + c["block"] - 1) // c["block"] - 1  # the diagonal block; -1: no token
    j = torch.arange(nb, device=DEV)
    last3 = last[:, None, None]
    key = torch.nan_to_num(key, nan=-1e300, neginf=-1e300, posinf=1e300)
    key = torch.where((j == 0) | (j == last3), torch.full_like(key, float("inf")), key)
    key = torch.where(j <= last3, key, torch.full_like(key, -float("inf")))
    pick = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :kcap]
    cnt = torch.where(last >= 0, st["budget"].long()[last.clamp(min=0)], torch.zeros_like(last))
    live = torch.arange(pick.shape[-1], device=DEV) < cnt[:, None, None]
    pick = torch.sort(torch.where(live, pick, torch.full_like(pick, nb)), dim=-1).values
    pick = torch.where(live, pick, torch.full_like(pick, -1)).to(torch.int32)
    per = c["Hq"] // key.shape[1]
    cnt = cnt.to(torch.int32)[:, None].expand(-1, c["Hq"])
    return pick.repeat_interleave(per, 1), cnt.contiguous()


def _plain_select(st):
    c = st["case"]
    R, Hq, D = st["q"].shape
    Hkv, G = c["Hkv"], c["Hq"] // c["Hkv"]
    t = st["table"].long()[st["rows"].long()]  # [R, nb]
    nb = t.shape[1]
    last = (st["lens"].long() + c["block"] - 1) // c["block"] - 1
    full = (torch.arange(nb, device=DEV) < last[:, None])[:, None, None, :]
    # in 64 bits: the choice between two close blocks hangs on the last digits
    kb = st["kbar"][t.clamp(min=0)].double().permute(0, 2, 3, 1)  # [R, Hkv, D, nb]
    n = st["vnorm"][t.clamp(min=0)].double().transpose(1, 2)  # [R, Hkv, nb]
    s = torch.matmul(st["q"].double().view(R, Hkv, G, D), kb) / math.sqrt(D)
    if c["metric"] == "additive":
        key = s + BETA * (2.0 * torch.log(n)).clamp(min=0.0)[:, :, None]
        if c["share"] == "group":
            key = key.sum(2)
    elif c["share"] == "group":
        # the softmax of each head over the full blocks, summed over the group's heads
        masked = torch.where(full, s, torch.full_like(s, -float("inf")))
        top = masked.amax(-1, keepdim=True).nan_to_num(neginf=0.0)
        lse = top + torch.log(torch.exp(masked - top).sum(-1, keepdim=True))
        z = s - lse
        zt = z.amax(2, keepdim=True)
        key = (zt + torch.log(torch.exp(z - zt).sum(2, keepdim=True))).squeeze(2) + torch.log(n)
    else:
        key = s + torch.log(n)[:, :, None]
    return _lists(st, key if c["share"] == "group" else key.flatten(1, 2))


def _plain_attn(st, sel_idx, sel_cnt):
    c = st["case"]
    R, Hq, D = st["q"].shape
    Hkv, block = c["Hkv"], c["block"]
    G = Hq // Hkv
    per = G if c["share"] == "group" else 1  # heads that share a list
    L = Hq // per
    idx, cnt = sel_idx[:, ::per].long(), sel_cnt[:, ::per].long()
    live = torch.arange(idx.shape[-1], device=DEV) < cnt[..., None]
    page = st["table"].long()[st["rows"].long()[:, None, None], idx.clamp(min=0)]
    head = torch.arange(L, device=DEV) // (G // per)
    k, v = _unpack(st["pages"][page.clamp(min=0), head[None, :, None]], c["fmt"], D)
    pos = idx[..., None] * block + torch.arange(block, device=DEV)
    seen = (live[..., None] & (pos < st["lens"].long()[:, None, None, None])).flatten(2)
    k, v = k.flatten(2, 3), v.flatten(2, 3)  # [R, L, tokens, D]
    v = torch.where(seen[..., None], v, torch.zeros_like(v))
    q = st["q"].float().view(R, L, per, D)
    z = torch.matmul(q, k.transpose(2, 3)) / math.sqrt(D)
    z = torch.where(seen[:, :, None], z, torch.full_like(z, -float("inf")))
    top = z.amax(-1, keepdim=True).nan_to_num(neginf=0.0)
    p = torch.exp(z - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + torch.log(total)).view(R, Hq)
    return o.reshape(R, Hq, D).to(torch.bfloat16), lse


def _token_at(st, T):
    """Page, slot and liveness of tokens pos .. pos + T - 1 of each sequence: [nseq, T]."""
    c, t = st["case"], torch.arange(T, device=DEV)
    at = st["pos"].long()[:, None] + t
    live = t < st["count"].long()[:, None]
    blk = torch.where(live, at // c["block"], torch.zeros_like(at))
    page = torch.gather(st["table"].long(), 1, blk)
    return page, at % c["block"], live


def _plain_read(st):
    c = st["case"]
    T = st["k"].shape[2]
    page, slot, live = _token_at(st, T)
    seq, t = live.nonzero(as_tuple=True)
    uniq, where = torch.unique(page[seq, t], return_inverse=True)
    for x, dst in zip(_unpack(st["pages"][uniq], c["fmt"], c["D"]), (st["k"], st["v"])):
        dst[seq, :, t] = x[where, :, slot[seq, t]].to(torch.bfloat16)
    return {"k": st["k"], "v": st["v"]}


def _plain_append(st):
    c = st["case"]
    T = st["k"].shape[2]
    page, slot, live = _token_at(st, T)
    seq, t = live.nonzero(as_tuple=True)
    if seq.numel():
        uniq, where = torch.unique(page[seq, t], return_inverse=True)
        k, v = (x.to(torch.bfloat16) for x in _unpack(st["pages"][uniq], c["fmt"], c["D"]))
        # 4- and 8-bit rows that stay are kept by their bytes: only new rows are packed again
        new = torch.zeros(uniq.numel(), c["block"], dtype=torch.bool, device=DEV)
        new[where, slot[seq, t]] = True
        k[where, :, slot[seq, t]] = st["k_new"][seq, :, t]
        v[where, :, slot[seq, t]] = st["v_new"][seq, :, t]
        packed = _pack(k, v, c["fmt"])
        fresh = _pack_mask(new, c)[:, None]
        old = st["pages"][uniq]
        rec = (packed & fresh) | (old & ~fresh)
        st["pages"][uniq] = rec
        # a block is summarised when its last token arrives
        done = new[:, -1]
        kb, vn = _summaries(*_unpack(rec, c["fmt"], c["D"]), c["vsum"])
        st["kbar"][uniq[done]], st["vnorm"][uniq[done]] = kb[done], vn[done]
    return {**_plain_read(st), "kbar": st["kbar"], "vnorm": st["vnorm"]}


def _pack_mask(new, c):
    """Bytes [n, record] whose bits are those of the tokens in new [n, block]."""
    D, fmt = c["D"], c["fmt"]
    tok = new.unflatten(-1, (-1, TILE))
    parts = []
    for what in "kv":
        e = tok[..., _index(fmt, D, what, False) // D]
        if fmt == "bf16":
            parts.append(e.repeat_interleave(2, -1).to(torch.uint8) * 255)
        elif fmt == "q8":
            parts.append(e.to(torch.uint8) * 255)
        else:
            parts.append(e[..., 0::2].to(torch.uint8) * 15 | e[..., 1::2].to(torch.uint8) * 240)
    if fmt != "bf16":
        parts.append(tok.repeat_interleave(4 * (D // GROUP), -1).to(torch.uint8) * 255)
    return torch.cat(parts, -1).flatten(-2)


def run(state):
    st, c = state, state["case"]
    if own:
        from block_sparse_causal_pooling_b200 import decode as S

        cache = S.PagedCache(st["pages"], st["kbar"], st["vnorm"], st["table"], c["block"],
                             c["fmt"], vsum=c["vsum"])
        if c["op"] in ("append", "read"):
            if c["op"] == "append":
                S.stem_cache_append(cache, st["k_new"], st["v_new"], st["pos"], st["count"])
            S.stem_cache_read(cache, st["pos"], st["count"], st["k"], st["v"])
            out = {"k": st["k"], "v": st["v"]}
            return out if c["op"] == "read" else {**out, "kbar": st["kbar"],
                                                  "vnorm": st["vnorm"]}
        if c["op"] == "attn":
            o, lse = S.stem_decode_attn(cache, st["q"], st["lens"], st["sel_idx"], st["sel_cnt"],
                                        share=c["share"], rows=st["rows"])
            return {"out": o, "lse": lse}
        method = S.make_method("exp", rho_min=c["rho"], tau=c["tau"], k_min=c["kmin"],
                               metric=c["metric"], beta=BETA, clamp=True, vsum=c["vsum"],
                               share=c["share"])
        if c["op"] == "select":
            idx, cnt = S.stem_decode_select(cache, st["q"], st["lens"], st["budget"], st["kcap"],
                                            method, rows=st["rows"])
            return {"sel_idx": idx, "sel_cnt": cnt}
        o, lse, idx, cnt = S.stem_decode(cache, st["q"], st["lens"], st["budget"], st["kcap"],
                                         method, rows=st["rows"])
        return {"out": o, "lse": lse, "sel_idx": idx, "sel_cnt": cnt}
    if c["op"] == "read":
        return _plain_read(st)
    if c["op"] == "append":
        return _plain_append(st)
    if c["op"] == "attn":
        o, lse = _plain_attn(st, st["sel_idx"], st["sel_cnt"])
        return {"out": o, "lse": lse}
    idx, cnt = _plain_select(st)
    if c["op"] == "select":
        return {"sel_idx": idx, "sel_cnt": cnt}
    o, lse = _plain_attn(st, idx, cnt)
    return {"out": o, "lse": lse, "sel_idx": idx, "sel_cnt": cnt}


# ------------------------------------------------------------------ the definition in 64 bits


def _exact_values(rec, c):
    """K and V [n, block, D] float64 of records [n, bytes] of one head: each code by its address."""
    fmt, D = c["fmt"], c["D"]
    ng, bits = D // GROUP, BITS[fmt]
    size = TILE * D * bits // 8
    per = 2 * size + (0 if fmt == "bf16" else TILE * 4 * ng)
    token = torch.arange(c["block"], device=rec.device)[:, None]
    d = torch.arange(D, device=rec.device)[None, :]
    r, base = token % TILE, (token // TILE) * per
    g, x = d // GROUP, d % GROUP
    out = []
    for n in range(2):
        if n == 0:
            lane, e, pair = (r % 8) * 4 + x // 8, x % 8, 0
        else:
            lane, e, pair = (x // 4) * 4 + (r % 8) // 2, x % 4, r % 2
        w = (r // 8) * ng + g  # words before this one in the lane's row
        if fmt == "q4":
            bit = (4 * (e // 2) + 16 * (e % 2)) if n == 0 else 16 * pair + 4 * e
        elif fmt == "q8":
            w = w * 2 + (e // 4 if n == 0 else e // 2)
            bit = (16 * (e % 2) + 8 * (e % 4 // 2)) if n == 0 else 16 * pair + 8 * (e % 2)
        else:
            w = w * 4 + (e // 2 if n == 0 else e)
            bit = 16 * (e % 2) if n == 0 else 16 * pair
        byte = base + n * size + (w // 4 * 32 + lane) * 16 + w % 4 * 4 + bit // 8
        byte, shift = torch.broadcast_tensors(byte, torch.as_tensor(bit % 8))
        raw = rec[:, byte.reshape(-1)].view(-1, c["block"], D).long()
        if fmt == "bf16":
            raw = raw + 256 * rec[:, byte.reshape(-1) + 1].view(-1, c["block"], D).long()
            out.append(_bits16(raw))
            continue
        code = ((raw >> shift) & ((1 << bits) - 1)).double() - (1 << (bits - 1))
        sb = (base + 2 * size + r * 4 * ng + 2 * (n * ng + g)).expand(-1, D).reshape(-1)
        sc = _bits16(rec[:, sb].long() + 256 * rec[:, sb + 1].long()).view(-1, c["block"], D)
        out.append(code * sc)
    return out


def _bits16(raw):
    """The bfloat16 numbers of 16-bit patterns, in 64 bits."""
    wide = torch.where(raw >= 32768, raw - 65536, raw).to(torch.int16)
    return wide.view(torch.bfloat16).double()


def _exact_code(x, fmt):
    """The values that a row x [..., D] stands for once it is in the cache, in 64 bits."""
    x = x.double()
    if fmt == "bf16":
        return x
    top = 7.0 if fmt == "q4" else 127.0
    y = x.reshape(*x.shape[:-1], -1, GROUP)
    s = (y.abs().max(-1, keepdim=True).values / top).float().to(torch.bfloat16).double()
    q = torch.where(s > 0, torch.minimum(torch.maximum(torch.round(y / s.clamp(min=1e-300)),
                                                       torch.tensor(-top, device=x.device,
                                                                    dtype=torch.float64)),
                                         torch.tensor(top, device=x.device,
                                                      dtype=torch.float64)), 0.0 * y)
    return (q * s).reshape(x.shape)


def exact(case, seed):
    c = case
    st = prepare(case, seed)
    block, D, Hkv = c["block"], c["D"], c["Hkv"]
    lens, table = _lengths(c), st["table"].cpu().tolist()
    if c["op"] in ("append", "read"):
        k, v = torch.zeros(st["k"].shape, dtype=torch.float64, device=DEV), None
        v = torch.zeros_like(k)
        kbar, vnorm = st["kbar"].double(), st["vnorm"].double()
        for s, (n, m) in enumerate(zip(lens, _counts(c))):
            first = n - m
            for b in range(first // block, -(-n // block) if m else 0):
                lo, hi = max(first, b * block), min(n, (b + 1) * block)
                pg = table[s][b]
                old = [torch.stack(x) for x in zip(*[
                    [y[0] for y in _exact_values(st["pages"][pg, h][None], c)]
                    for h in range(Hkv)])]
                a, z = lo - b * block, hi - b * block
                if c["op"] == "append":
                    old[0][:, a:z] = _exact_code(st["k_new"][s, :, lo - first:hi - first],
                                                 c["fmt"])
                    old[1][:, a:z] = _exact_code(st["v_new"][s, :, lo - first:hi - first],
                                                 c["fmt"])
                    if z == block:
                        kbar[pg] = old[0].sum(1) / block
                        norm = torch.linalg.vector_norm(old[1], dim=-1)
                        vnorm[pg] = norm.max(1).values if c["vsum"] == "max" else norm.sum(1) / block
                k[s, :, lo - first:hi - first] = old[0][:, a:z]
                v[s, :, lo - first:hi - first] = old[1][:, a:z]
        out = {"k": k, "v": v}
        return out if c["op"] == "read" else {**out, "kbar": kbar, "vnorm": vnorm}
    if c["op"] == "select":
        return None  # whole numbers alone
    R, Hq = len(_rows(c)), c["Hq"]
    G = Hq // Hkv
    if R * Hq > 4096:
        return None
    idx, cnt = ((st["sel_idx"], st["sel_cnt"]) if c["op"] == "attn" else _plain_select(st))
    idx, cnt = idx.cpu().tolist(), cnt.cpu().tolist()
    out = torch.zeros(R, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.full((R, Hq), -float("inf"), dtype=torch.float64, device=DEV)
    for r, (s, n) in enumerate(_rows(c)):
        for h in range(Hq):
            kept = idx[r][h][:cnt[r][h]]
            if not kept:
                continue
            if c["share"] == "head" or h % G == 0:
                pg = torch.tensor([table[s][j] for j in kept], device=DEV)
                k, v = (x.reshape(-1, D) for x in _exact_values(st["pages"][pg, h // G], c))
                short = (kept[-1] + 1) * block - n  # tokens of the last block that are not there
                if short > 0:
                    k, v = k[:-short], v[:-short]
            z = (k @ st["q"][r, h].double()) / math.sqrt(D)
            lse[r, h] = torch.logsumexp(z, 0)
            out[r, h] = torch.softmax(z, 0) @ v
    res = {"out": out, "lse": lse}
    return res if c["op"] == "attn" else {**res, "sel_idx": None, "sel_cnt": None}
