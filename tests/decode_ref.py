"""The decode path in 64 bits, on the CPU, from the definitions in include/stem.h (it shares no code
with the library): page layout, quantisation, block summaries, selection and attention."""

from __future__ import annotations

import functools
import math

import numpy as np
import torch

BITS = {"bf16": 16, "q8": 8, "q4": 4}
OFFSET = {"q8": 128, "q4": 8}
QMAX = {"q8": 127, "q4": 7}


def tile_bytes(fmt, D):
    return 16 * D * 2 * BITS[fmt] // 8 + (0 if fmt == "bf16" else 16 * 4 * (D // 32))


def page_bytes(fmt, D, block):
    return tile_bytes(fmt, D) * (block // 16)


@functools.lru_cache(maxsize=None)
def bit_of(fmt, D):
    """(K, V): first bit of the code of (token of the tile, channel) within a tile: [16, D] each."""
    W = {"q4": 1, "q8": 2, "bf16": 4}[fmt]
    size = 16 * D * BITS[fmt] // 8
    out = []
    for which in range(2):
        a = np.zeros((16, D), dtype=np.int64)
        for r in range(16):
            for d in range(D):
                x = d % 32
                if which == 0:
                    lane, e = (r % 8) * 4 + x // 8, x % 8
                    w, bit = {"q4": (0, 16 * (e % 2) + 4 * (e // 2)),
                              "q8": (e // 4, 16 * (e % 2) + 8 * (e % 4 // 2)),
                              "bf16": (e // 2, 16 * (e % 2))}[fmt]
                else:
                    lane, e = (x // 4) * 4 + (r % 8) // 2, x % 4
                    w, bit = {"q4": (0, 16 * (r % 2) + 4 * e),
                              "q8": (e // 2, 16 * (r % 2) + 8 * (e % 2)),
                              "bf16": (e, 16 * (r % 2))}[fmt]
                n = ((r // 8) * (D // 32) + d // 32) * W + w
                byte = which * size + (n // 4 * 32 + lane) * 16 + n % 4 * 4
                a[r, d] = byte * 8 + bit
        out.append(a)
    return out


def quantise(x, fmt):
    """(codes without offset, bf16 scales, values in float64) of x [..., D] (float32 or bfloat16)."""
    g = x.float().reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    amax = g.abs().amax(-1)
    amax = torch.where(torch.isnan(g).any(-1), torch.full_like(amax, float("nan")), amax)
    s = (amax / QMAX[fmt]).to(torch.bfloat16)
    s = torch.where(torch.isfinite(amax), s, torch.full_like(s, float("nan")))
    f = s.float()[..., None]
    c = torch.where(f > 0, torch.round(g / f).clamp(-QMAX[fmt], QMAX[fmt]), torch.zeros_like(g))
    v = c.double() * s.double()[..., None]
    return c.reshape(x.shape).long(), s, v.reshape(x.shape)


def put_row(page, fmt, D, token, k, v):
    """Write the K and V row (D elements) of a token into a page record (uint8 numpy array)."""
    base = token // 16 * tile_bytes(fmt, D)
    r = token % 16
    size = 16 * D * BITS[fmt] // 8
    for which, x in enumerate((k, v)):
        bits = bit_of(fmt, D)[which][r] + base * 8
        at, sh = bits // 8, bits % 8
        if fmt == "bf16":
            u = x.to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16).astype(np.int64)
            page[at] = u & 255
            page[at + 1] = u >> 8
            continue
        c, s, _ = quantise(x, fmt)
        c = c.numpy() + OFFSET[fmt]
        if fmt == "q8":
            page[at] = c
        else:
            for a, b, y in zip(at, sh, c):
                page[a] = (int(page[a]) & ~(15 << int(b)) & 255) | int(y) << int(b)
        o = base + 2 * size + r * 4 * (D // 32) + which * 2 * (D // 32)
        page[o:o + 2 * (D // 32)] = s.contiguous().view(torch.int16).numpy().view(np.uint8)


def get_rows(page, fmt, D, tokens):
    """K and V values [len(tokens), D] float64 that a page record stands for."""
    page = np.asarray(page)
    tokens = np.asarray(tokens)
    base = (tokens // 16 * tile_bytes(fmt, D))[:, None]
    r = tokens % 16
    size = 16 * D * BITS[fmt] // 8
    out = []
    for which in range(2):
        bits = bit_of(fmt, D)[which][r] + base * 8
        at, sh = bits // 8, bits % 8
        if fmt == "bf16":
            u = page[at].astype(np.uint32) | page[at + 1].astype(np.uint32) << 8
            out.append(torch.from_numpy((u << 16).view(np.float32).astype(np.float64)))
            continue
        c = (page[at].astype(np.int64) >> sh & ((1 << BITS[fmt]) - 1)) - OFFSET[fmt]
        g = np.arange(D) // 32
        o = base + 2 * size + r[:, None] * 4 * (D // 32) + which * 2 * (D // 32) + 2 * g
        u = page[o].astype(np.uint32) | page[o + 1].astype(np.uint32) << 8
        s = (u << 16).view(np.float32).astype(np.float64)
        out.append(torch.from_numpy(c * s))
    return out


def summaries(k, v, vsum):
    n = v.square().sum(-1).sqrt()
    return k.mean(-2), (n.amax(-1) if vsum == "max" else n.mean(-1))


def keys(q, kb, n, share, metric, beta, clamp):
    """Ranking keys [heads or 1, blocks] of queries q [G, D] against summaries of blocks 0 .. i - 1."""
    s = q.double() @ kb.double().T / math.sqrt(q.shape[1])
    n = n.double()
    if metric == "additive":
        e = 2 * torch.log(n)
        e = torch.where(e < 0, torch.zeros_like(e), e) if clamp else e
        x = s + (beta * e if beta else 0.0)
        return x.sum(0, keepdim=True) if share == "group" else x
    if share == "group":
        z = s - torch.logsumexp(s, -1, keepdim=True)
        return (torch.logsumexp(z, 0) + torch.log(n))[None]
    return s + torch.log(n)


def select(q, kb, n, last, k, share, metric, beta=0.0, clamp=True):
    """Kept blocks (ascending) for each head of q [G, D]; kb, n: summaries of blocks 0 .. last - 1.
    Returns (lists, smallest gap between a kept and a dropped candidate's keys)."""
    G = q.shape[0]
    if last < 0:
        return [[] for _ in range(G)], math.inf
    if k >= last + 1:
        return [list(range(last + 1)) for _ in range(G)], math.inf
    key = keys(q, kb, n, share, metric, beta, clamp)
    lists, gap = [], math.inf
    for x in key.tolist():
        x = [-math.inf if math.isnan(y) else y for y in x]
        order = sorted(range(1, last), key=lambda j: (-x[j], j))
        inn, out = order[:k - 2], order[k - 2:]
        if inn and out and x[inn[-1]] != x[out[0]]:
            gap = min(gap, x[inn[-1]] - x[out[0]])
        lists.append(sorted([0, last] + inn))
    return (lists * G if share == "group" else lists), gap


def attend(q, k, v):
    """(out, lse) of one query q [D] over k, v [tokens, D], float64."""
    if k.shape[0] == 0:
        return torch.zeros_like(q, dtype=torch.float64), -math.inf
    z = k @ q.double() / math.sqrt(q.shape[0])
    return torch.softmax(z, 0) @ v, float(torch.logsumexp(z, 0))


class Cache:
    """A paged cache on the CPU: the same buffers as the library's, and what to do with them."""

    def __init__(self, num_pages, Hkv, D, block, fmt, table, vsum="mean", fill=0):
        self.pages = np.full((num_pages, Hkv, page_bytes(fmt, D, block)), fill, dtype=np.uint8)
        self.kbar = torch.zeros(num_pages, Hkv, D, dtype=torch.float64)
        self.vnorm = torch.zeros(num_pages, Hkv, dtype=torch.float64)
        self.table, self.block, self.fmt, self.vsum, self.D, self.Hkv = (
            table, block, fmt, vsum, D, Hkv)

    def append(self, k, v, pos, count):
        """k, v [nseq, Hkv, T, D]; pos, count: lists."""
        for s in range(len(pos)):
            for t in range(count[s]):
                j, slot = divmod(pos[s] + t, self.block)
                p = int(self.table[s, j])
                for h in range(self.Hkv):
                    put_row(self.pages[p, h], self.fmt, self.D, slot, k[s, h, t], v[s, h, t])
                    if slot == self.block - 1:
                        rows = get_rows(self.pages[p, h], self.fmt, self.D, range(self.block))
                        self.kbar[p, h], self.vnorm[p, h] = summaries(*rows, self.vsum)

    def tokens(self, s, h, js, n):
        """K and V of the tokens below n of blocks js of sequence s, head h."""
        ks, vs = [], []
        for j in js:
            m = min(self.block, n - j * self.block)
            k, v = get_rows(self.pages[int(self.table[s, j]), h], self.fmt, self.D, range(m))
            ks.append(k)
            vs.append(v)
        if not ks:
            z = torch.zeros(0, self.D, dtype=torch.float64)
            return z, z
        return torch.cat(ks), torch.cat(vs)


def attn_tolerance(q, k, v, fmt, out):
    """Elementwise bound on the error of the library's attention of q [D] over k, v [tokens, D],
    and of its lse. With u = 2^-22 for each float32 step on the tensor cores (they may truncate):
      logits: a chain of D products and the D/32 scaled group sums, whose terms are at most
        |q_d| * top, top the largest magnitude that an offset code can stand for (twice the group's
        largest value; the value itself at 16 bits), then the scale: relative u each;
      weights: exp2 and its argument's rounding, one rounding to fp16 (2^-11) or bf16 (2^-8), the
        latter also in the normaliser; the running rescale: a float32 rounding a tile;
      sums over tokens: one u a token on the magnitude of what is added (offset codes again);
      4- and 8-bit codes enter the MMA as fp16 subnormals. The tensor pipe cuts each product at
        2^-25 of the largest product of its chain of 16, and takes a subnormal's exponent for -14
        (measured: with weight 2^14 and code * 2^-24 at the top, 2^-25 beside it is kept and 2^-26
        lost). In code steps that is 2^(e - 14 - 25 + 24) = 2^-15 of the largest factor 2^e. So a
        group's value sum loses at most 16 * 2^-15 = 2^-11 scales times the largest weight of each
        tile, and a logit at most D * 2^-15 * max|q| scales;
      the output's own rounding to bf16, 2^-8 of it.
    """
    u = 2.0 ** -22
    n, D = k.shape
    if n == 0:
        return torch.zeros_like(out), 0.0
    if fmt == "bf16":
        kt, vt = k.abs(), v.abs()
    else:  # code + offset is at most 2 * offset, the scale |largest| / QMAX
        up = 2.0 * OFFSET[fmt] / QMAX[fmt]
        kt = up * k.abs().reshape(n, -1, 32).amax(-1, keepdim=True).expand(-1, -1, 32).reshape(n, D)
        vt = up * v.abs().reshape(n, -1, 32).amax(-1, keepdim=True).expand(-1, -1, 32).reshape(n, D)
    z = k @ q.double() / math.sqrt(D)
    dz = float(((D + D // 32 + 4) * u * (kt @ q.double().abs()) / math.sqrt(D)).max())
    dz += 4 * u * float(z.abs().max()) + 8 * u
    cut = 0.0
    if fmt != "bf16":
        step = 0.5 / OFFSET[fmt]  # a scale, as a share of kt and vt
        dz += D * 2.0 ** -15 * float(q.abs().max()) * float(kt.max()) * step / math.sqrt(D)
        cut = 2.0 ** -11 * step
    w = torch.softmax(z, 0)
    rel = 2 * dz + (2.0 ** -11 if fmt != "bf16" else 2.0 ** -7) + (n // 16 + 8) * 2 * u
    tol = (w @ v.abs()) * rel + (w @ vt) * ((n + 32) * u + cut) + out.abs() * 2.0 ** -8 + 1e-30
    dl = dz + (2.0 ** -8 if fmt == "bf16" else 0.0) + (n // 16 + n % 16 + 16) * u
    return tol, dl
