"""The decode path on a B200 against its definition in 64 bits (tests/decode_ref.py): writing and
reading the paged cache, the block selection of single query tokens, their attention, and a run of
all of them as a generating model would use them."""

import math

import numpy as np
import pytest
import torch

from block_sparse_causal_pooling_b200 import decode as S
from block_sparse_causal_pooling_b200 import stem as base
from tests import decode_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
FORMATS = ["bf16", "q8", "q4"]
SHAPES = [(64, 64), (128, 64), (64, 128), (128, 128)]  # D, block


def make_table(nblocks, max_blocks, spare=2, seed=0):
    """Disjoint pages in a shuffled order; -1 past each sequence's blocks."""
    total = sum(nblocks) + spare
    order = np.random.RandomState(seed).permutation(total).astype(np.int32)
    t = np.full((len(nblocks), max_blocks), -1, dtype=np.int32)
    at = 0
    for s, n in enumerate(nblocks):
        t[s, :n] = order[at:at + n]
        at += n
    return t, total


def rows(g, *shape, dtype=torch.bfloat16):
    x = torch.randn(*shape, generator=g) * torch.exp(0.7 * torch.randn(*shape[:-1], 1, generator=g))
    return x.to(dtype)


def pair(num_pages, Hkv, D, block, fmt, table, vsum="mean", fill=0xFF):
    """The same cache on the GPU and in the reference, unwritten bytes `fill` (0xff: NaN rows)."""
    gpu = S.PagedCache.alloc(num_pages, Hkv, D, block, fmt, torch.from_numpy(table).to(DEV), vsum)
    gpu.pages.fill_(fill)
    return gpu, ref.Cache(num_pages, Hkv, D, block, fmt, table, vsum, fill)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def status_word():
    return torch.full((1,), 7, dtype=torch.int32, device=DEV)


def check_pages(gpu, cpu):
    assert np.array_equal(gpu.pages.cpu().numpy(), cpu.pages)


def check_summaries(gpu, cpu, blocks):
    """float32 sums of a block's rows: 8 tiles of pairs, a tree of 8 pairs and a division for kbar;
    for vnorm 12 steps of the square sum halved by the root, the root, and the same mean."""
    u = 2.0 ** -24
    for p, size in blocks:
        for h in range(cpu.Hkv):
            k, v = ref.get_rows(cpu.pages[p, h], cpu.fmt, cpu.D, range(cpu.block))
            tol = 14 * u * k.abs().mean(0) + 1e-30
            assert torch.all((gpu.kbar[p, h].cpu().double() - cpu.kbar[p, h]).abs() <= tol)
            d = abs(float(gpu.vnorm[p, h]) - float(cpu.vnorm[p, h]))
            assert d <= 24 * u * float(cpu.vnorm[p, h]) + 1e-30


# ------------------------------------------------------------------ the cache


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D,block", SHAPES)
def test_append_writes_the_defined_bytes(fmt, D, block):
    """Ragged chunks at odd offsets, an empty sequence, token-major strides; every byte of the cache
    afterwards, the other bytes left as they were."""
    g = torch.Generator().manual_seed(D + block)
    Hkv, pos, count = 2, [0, 5, block - 1, 3, 2 * block], [block + 3, 2, 2, 0, 1]
    nb = [-(-(p + c) // block) if c else 1 for p, c in zip(pos, count)]
    table, pages = make_table(nb, max(nb) + 1)
    gpu, cpu = pair(pages, Hkv, D, block, fmt, table, fill=0x11)
    T = max(count)
    k, v = (rows(g, len(pos), T, Hkv, D).transpose(1, 2) for _ in range(2))
    st = status_word()
    S.stem_cache_append(gpu, k.to(DEV), v.to(DEV), i32(pos), i32(count), status=st)
    cpu.append(k, v, pos, count)
    assert int(st) == 0
    check_pages(gpu, cpu)
    full = [(int(table[s, j]), block) for s in range(len(pos)) for j in range(nb[s])
            if count[s] and pos[s] < (j + 1) * block <= pos[s] + count[s]]
    assert full
    check_summaries(gpu, cpu, full)
    # blocks that are not complete keep the summaries they had
    left = set(range(pages)) - {p for p, _ in full}
    for p in left:
        assert not gpu.kbar[p].any() and not gpu.vnorm[p].any()
    # and back
    out = [torch.full((len(pos), Hkv, T, D), 3.0, dtype=torch.bfloat16, device=DEV) for _ in "kv"]
    S.stem_cache_read(gpu, i32(pos), i32(count), *out)
    wide = S.stem_cache_read(gpu, i32(pos), i32(count), T=T, dtype=torch.float32)
    for x, y, src in zip(out, wide, (k, v)):
        for s in range(len(pos)):
            n = count[s]
            want = src[s, :, :n].double() if fmt == "bf16" else ref.quantise(src[s, :, :n], fmt)[2]
            assert torch.equal(y[s, :, :n].cpu().double(), want)
            assert torch.equal(x[s, :, :n].cpu(), want.float().to(torch.bfloat16))
            assert (x[s, :, n:] == 3.0).all() and not y[s, :, n:].any()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("vsum", ["mean", "max"])
def test_token_by_token_equals_one_call(fmt, vsum):
    """However a sequence arrives, the cache and its summaries hold the same bits; and taking tokens
    back by writing an earlier position again gives what was never taken back."""
    g = torch.Generator().manual_seed(5)
    D, block, Hkv, n = 128, 64, 2, 150
    k, v = rows(g, 1, Hkv, n, D).to(DEV), rows(g, 1, Hkv, n, D).to(DEV)
    table, pages = make_table([3], 3)
    caches = []
    for steps in ([n], [1] * n, [63, 1, 1, 64, 20, 1], "back"):
        c = S.PagedCache.alloc(pages, Hkv, D, block, fmt, torch.from_numpy(table).to(DEV), vsum)
        if steps == "back":
            S.stem_cache_append(c, k[:, :, :140], v[:, :, :140], i32([0]))
            S.stem_cache_append(c, v[:, :, 100:140], k[:, :, 100:140], i32([100]))  # rejected
            S.stem_cache_append(c, k[:, :, 100:], v[:, :, 100:], i32([100]))
        else:
            at = 0
            for m in steps:
                S.stem_cache_append(c, k[:, :, at:at + m], v[:, :, at:at + m], i32([at]))
                at += m
        caches.append(c)
    for c in caches[1:]:
        assert torch.equal(c.pages, caches[0].pages)
        assert torch.equal(c.kbar, caches[0].kbar) and torch.equal(c.vnorm, caches[0].vnorm)
    assert caches[0].kbar.any() and caches[0].vnorm.any()


@pytest.mark.parametrize("fmt", ["q8", "q4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantising_extreme_rows(fmt, dtype):
    """Zeros, subnormals, the type's largest values, infinities and NaN, ties, negative zero."""
    D, block = 64, 64
    big = torch.finfo(torch.bfloat16).max
    x = torch.zeros(1, 1, 12, D)
    x[0, 0, 1] = 1e-40
    x[0, 0, 2, :32] = torch.linspace(-big, big, 32)
    x[0, 0, 3, 5] = float("inf")
    x[0, 0, 4, 40] = float("nan")
    x[0, 0, 5] = -0.0
    x[0, 0, 6] = torch.arange(D) - 31.5
    x[0, 0, 7, 0] = 7.0 if fmt == "q4" else 127.0  # scale 1: halves are ties
    x[0, 0, 7, 1:32] = torch.arange(31) * 0.5 - 6.75 + 0.25
    x[0, 0, 8, 3] = float("-inf")
    x[0, 0, 9] = 2.0 ** -126
    x[0, 0, 10, 7] = 3e-39
    x[0, 0, 11] = torch.randn(D, generator=torch.Generator().manual_seed(1))
    x = x.to(dtype)
    table, pages = make_table([1], 1)
    gpu, cpu = pair(pages, 1, D, block, fmt, table)
    S.stem_cache_append(gpu, x.to(DEV), x.flip(2).contiguous().to(DEV), i32([0]))
    cpu.append(x, x.flip(2), [0], [12])
    check_pages(gpu, cpu)
    k, v = S.stem_cache_read(gpu, i32([0]), T=12, dtype=torch.float32)
    want = ref.quantise(x, fmt)[2].float()
    assert torch.equal(torch.isnan(k.cpu()), torch.isnan(want))
    # rows 3, 4 and 8 have one group each that is not finite, and so has row 2: linspace's step,
    # twice the largest number, overflows
    assert torch.isnan(want).sum() == 4 * 32
    assert torch.equal(k.cpu().nan_to_num(9.0), want.nan_to_num(9.0))
    assert torch.equal(v.cpu().flip(2).nan_to_num(9.0), want.nan_to_num(9.0))


@pytest.mark.parametrize("fmt", ["q8", "q4"])
def test_quantising_the_largest_numbers(fmt):
    """Rows up to the type's largest number: scale and codes stay finite (a value may round up past
    it, as scale * code can)."""
    D, block = 64, 64
    big = torch.finfo(torch.bfloat16).max
    x = (torch.linspace(-1, 1, 4 * D).reshape(1, 1, 4, D) * big).to(torch.bfloat16)
    assert torch.isfinite(x).all()
    table, pages = make_table([1], 1)
    gpu, cpu = pair(pages, 1, D, block, fmt, table)
    S.stem_cache_append(gpu, x.to(DEV), -x.to(DEV), i32([0]))
    cpu.append(x, -x, [0], [4])
    check_pages(gpu, cpu)
    k, _ = S.stem_cache_read(gpu, i32([0]), T=4, dtype=torch.float32)
    want = ref.quantise(x, fmt)[2].float()
    assert not torch.isnan(k).any() and torch.equal(k.cpu(), want)


def test_float32_rows_in_a_bf16_cache_are_rounded_once():
    g = torch.Generator().manual_seed(2)
    x = torch.randn(1, 1, 20, 64, generator=g)
    table, pages = make_table([1], 1)
    gpu, cpu = pair(pages, 1, 64, 64, "bf16", table)
    S.stem_cache_append(gpu, x.to(DEV), -x.to(DEV), i32([0]))
    k, v = S.stem_cache_read(gpu, i32([0]), T=20)
    assert torch.equal(k.cpu(), x.to(torch.bfloat16)) and torch.equal(v, -k)


def test_bad_positions_and_pages_are_reported_and_skipped():
    D, block = 64, 64
    table = np.array([[0, 1], [99, 2], [3, -1]], dtype=np.int32)
    x = torch.ones(3, 1, 70, D, dtype=torch.bfloat16, device=DEV)
    for pos, count, written in [([0, 0, 0], [10, 10, 10], [0, 3]), ([-1, 64, 0], [1, 1, 1], [2, 3]),
                                ([128, 100, 64], [1, 70, 1], []), ([0, 0, 0], [-3, 71, 0], [])]:
        gpu, _ = pair(5, 1, D, block, "q8", table, fill=0x33)
        st = status_word()
        S.stem_cache_append(gpu, x, x, i32(pos), i32(count), status=st)
        assert int(st) == base.STEM_ERR_ARG
        touched = [p for p in range(5) if (gpu.pages[p] != 0x33).any()]
        assert touched == written
        st = status_word()
        k, v = S.stem_cache_read(gpu, i32(pos), i32(count), T=70, status=st)
        assert int(st) == base.STEM_ERR_ARG


# ------------------------------------------------------------------ selection


def fill_summaries(gpu, g, scale=1.0):
    n, Hkv, D = gpu.kbar.shape
    kb = (torch.randn(n, Hkv, D, generator=g) * scale).float()
    vn = torch.exp(0.5 * torch.randn(n, Hkv, generator=g)).float() * 3
    gpu.kbar.copy_(kb)
    gpu.vnorm.copy_(vn)
    return kb, vn


def check_select(gpu, q, row_seq, lens, budget, kb, vn, table, share, metric, beta, clamp, idx, cnt,
                 kcap):
    R, Hq, D = q.shape
    Hkv = kb.shape[1]
    G = Hq // Hkv
    idx, cnt = idx.cpu(), cnt.cpu()
    for r in range(R):
        last = -(-lens[r] // gpu.block) - 1
        k = min(budget[last], kcap) if last >= 0 else 0
        pg = [int(table[row_seq[r], j]) for j in range(max(last, 0))]
        for kv in range(Hkv):
            lists, gap = ref.select(q[r, kv * G:(kv + 1) * G], kb[pg, kv], vn[pg, kv], last, k, share,
                                    metric, beta, clamp)
            assert gap > 1e-11  # the inputs have no near-ties that double could decide either way
            for h in range(G):
                got = idx[r, kv * G + h].tolist()
                n = int(cnt[r, kv * G + h])
                assert got[:n] == lists[h], (r, kv, h)
                assert got[n:] == [-1] * (kcap - n)


@pytest.mark.parametrize("share", ["head", "group"])
@pytest.mark.parametrize("metric,beta,clamp", [("product", 0.0, True), ("additive", 0.2, True),
                                               ("additive", 1.5, False), ("additive", 0.0, True)])
@pytest.mark.parametrize("D,G", [(64, 1), (128, 4), (128, 7), (64, 9)])
def test_select_matches_the_definition(share, metric, beta, clamp, D, G):
    g = torch.Generator().manual_seed(G * 10 + D)
    block, Hkv = 64, 2
    lens_seq = [64 * 40, 1, 64, 65, 64 * 300 - 7, 64 * 97 + 1, 128]
    nb = [-(-n // block) for n in lens_seq]
    table, pages = make_table(nb, max(nb))
    gpu, _ = pair(pages, Hkv, D, block, "q4", table)
    kb, vn = fill_summaries(gpu, g)
    row_seq = [0, 1, 2, 3, 4, 5, 6, 4, 4, 0, 5]
    lens = [lens_seq[s] for s in row_seq]
    lens[7], lens[8], lens[9] = 64 * 299 + 1, 64 * 150, 0
    m = S.make_method("exp", rho_min=0.1, tau=8.0, k_min=3, metric=metric, beta=beta, clamp=clamp,
                      share=share)
    budget, kcap = S.stem_decode_budget(max(nb), m, DEV)
    q = rows(g, len(lens), Hkv * G, D)
    st = status_word()
    idx, cnt = S.stem_decode_select(gpu, q.to(DEV), i32(lens), budget, kcap, m, rows=i32(row_seq),
                                    status=st)
    assert int(st) == 0
    check_select(gpu, q, row_seq, lens, budget.tolist(), kb, vn, table, share, metric,
                 float(np.float32(beta)), clamp, idx, cnt, kcap)


@pytest.mark.parametrize("share", ["head", "group"])
@pytest.mark.parametrize("nb", [513, 4096])
def test_select_long_contexts(share, nb):
    g = torch.Generator().manual_seed(nb)
    D, block, Hkv, G = 64, 64, 1, 2
    table, pages = make_table([nb], nb, spare=0)
    gpu, _ = pair(pages, Hkv, D, block, "q4", table)
    kb, vn = fill_summaries(gpu, g, scale=0.05)
    q = rows(g, 2, 2, D)
    lens = [nb * block, nb * block - 70]
    for kw in (dict(rho_min=0.02, tau=64.0, k_min=2), dict(rho_min=0.9, tau=1.0, k_min=2),
               dict(rho_min=1.0, tau=1.0, k_min=2), dict(rho_min=1e-4, tau=1.0, k_min=1)):
        m = S.make_method("exp", share=share, **kw)
        budget, kcap = S.stem_decode_budget(nb, m, DEV)
        idx, cnt = S.stem_decode_select(gpu, q.to(DEV), i32(lens), budget, kcap, m, rows=i32([0, 0]))
        check_select(gpu, q, [0, 0], lens, budget.tolist(), kb, vn, table, share, "product", 0.0,
                     True, idx, cnt, kcap)


@pytest.mark.parametrize("share", ["head", "group"])
@pytest.mark.parametrize("nb,G,D", [(300, 4, 128), (30, 9, 64), (700, 2, 64)])
def test_select_of_many_rows(share, nb, G, D):
    """More rows than run at once (a kernel with fewer registers) choose as the definition does, and
    as the same rows do in a small call."""
    g = torch.Generator().manual_seed(nb)
    block, Hkv, few = 64, 2, 12
    table, pages = make_table([nb], nb, spare=0)
    gpu, _ = pair(pages, Hkv, D, block, "q4", table)
    kb, vn = fill_summaries(gpu, g)
    q = rows(g, few, Hkv * G, D)
    lens = [nb * block - 64 * (nb // few) * r - 5 * r for r in range(few)]
    m = S.make_method("exp", rho_min=0.1, tau=8.0, k_min=3, share=share)
    budget, kcap = S.stem_decode_budget(nb, m, DEV)
    times = 400 // few
    st = status_word()
    idx, cnt = S.stem_decode_select(gpu, q.repeat(times, 1, 1).to(DEV), i32(lens * times), budget,
                                    kcap, m, rows=i32([0] * (few * times)), status=st)
    assert int(st) == 0
    check_select(gpu, q, [0] * few, lens, budget.tolist(), kb, vn, table, share, "product", 0.0, True,
                 idx[:few], cnt[:few], kcap)
    one = S.stem_decode_select(gpu, q.to(DEV), i32(lens), budget, kcap, m, rows=i32([0] * few))
    assert torch.equal(idx, one[0].repeat(times, 1, 1))
    assert torch.equal(cnt, one[1].repeat(times, 1))


@pytest.mark.parametrize("share", ["head", "group"])
def test_select_ties_and_odd_summaries(share):
    """Blocks that share a page tie exactly: the lower index wins. Zero V norms (ln 0), NaN and
    infinite summaries rank as the definition says."""
    D, block, G = 128, 64, 3
    nb = 64
    table = (np.arange(nb, dtype=np.int32) % 5)[None].copy()
    gpu, _ = pair(5, 1, D, block, "q8", table)
    g = torch.Generator().manual_seed(3)
    kb, vn = fill_summaries(gpu, g)
    vn[1] = 0.0
    kb[2, 0, 7] = float("nan")
    gpu.kbar.copy_(kb)
    gpu.vnorm.copy_(vn)
    q = rows(g, 1, G, D)
    for metric in ("product", "additive"):
        for k in (2, 3, 9, 20, 45, 63, 64):
            if share == "group" and metric == "product":
                kb[2, 0, 7] = 0.5  # a NaN score would make the whole softmax NaN
                gpu.kbar.copy_(kb)
            m = S.make_method("exp", rho_min=1.0, tau=1.0, metric=metric, beta=0.3, clamp=False,
                              share=share)
            budget = torch.full((nb,), k, dtype=torch.int32, device=DEV)
            idx, cnt = S.stem_decode_select(gpu, q.to(DEV), i32([nb * block]), budget, 64, m)
            lists, _ = ref.select(q[0], kb[table[0, :nb - 1], 0], vn[table[0, :nb - 1], 0], nb - 1, k,
                                  share, metric, float(np.float32(0.3)), False)
            for h in range(G):
                assert idx[0, h, :k].tolist() == lists[h]
                assert int(cnt[0, h]) == k


@pytest.mark.parametrize("share", ["head", "group"])
@pytest.mark.parametrize("metric", ["product", "additive"])
@pytest.mark.parametrize("nb,G,D", [(40, 1, 64), (200, 4, 128), (700, 8, 64), (1500, 11, 128)])
def test_select_among_blocks_that_nearly_tie(share, metric, nb, G, D):
    """Summaries that differ in their last digits: keys closer than float32 arithmetic can tell apart,
    for all rows or for some, decided as double precision decides."""
    g = torch.Generator().manual_seed(nb)
    table, pages = make_table([nb], nb, spare=0)
    gpu, _ = pair(pages, 1, D, 64, "q4", table)
    for spread, some in ((1e-6, 1.0), (3e-5, 1.0), (1e-6, 0.3)):
        kb, vn = fill_summaries(gpu, g)
        near = torch.rand(pages, 1, 1, generator=g) < some
        kb = torch.where(near, kb[:1] + spread * kb, kb)
        vn = torch.where(near[..., 0], vn[:1] * (1 + spread * torch.randn(pages, 1, generator=g)), vn)
        gpu.kbar.copy_(kb)
        gpu.vnorm.copy_(vn)
        q = rows(g, 4, G, D)
        lens = [nb * 64, nb * 64 - 100, nb * 40, 64 * 9 + 1]
        for rho in (0.05, 0.5):
            m = S.make_method("exp", rho_min=rho, tau=2.0, k_min=3, share=share, metric=metric, beta=0.2)
            budget, kcap = S.stem_decode_budget(nb, m, DEV)
            idx, cnt = S.stem_decode_select(gpu, q.to(DEV), i32(lens), budget, kcap, m,
                                            rows=i32([0] * 4))
            check_select(gpu, q, [0] * 4, lens, budget.tolist(), kb, vn, table, share, metric,
                         float(np.float32(0.2)), True, idx, cnt, kcap)


def test_select_with_infinite_summaries():
    """Infinite scores: first where they are +infinity, last where -infinity or not a number."""
    g = torch.Generator().manual_seed(21)
    D, nb = 64, 90
    table, pages = make_table([nb], nb, spare=0)
    gpu, _ = pair(pages, 1, D, 64, "q8", table)
    kb, vn = fill_summaries(gpu, g)
    q = rows(g, 1, 2, D)
    kb[5, 0, 3], kb[17, 0, 3], kb[40, 0, 3] = float("inf"), float("-inf"), float("nan")
    vn[30], vn[31] = float("inf"), 0.0
    gpu.kbar.copy_(kb)
    gpu.vnorm.copy_(vn)
    for k in (3, 4, 9, 60, 87, 88):
        m = S.make_method("exp", rho_min=1.0, tau=1.0)
        budget = torch.full((nb,), k, dtype=torch.int32, device=DEV)
        idx, cnt = S.stem_decode_select(gpu, q.to(DEV), i32([nb * 64]), budget, k, m)
        pg = table[0, :nb - 1]
        lists, _ = ref.select(q[0], kb[pg, 0], vn[pg, 0], nb - 1, k, "head", "product")
        for h in range(2):
            assert idx[0, h].tolist() == lists[h] and int(cnt[0, h]) == k


def test_select_reports_bad_rows_budgets_and_pages():
    D, block, nb = 64, 64, 8
    table = np.arange(2 * nb, dtype=np.int32).reshape(2, nb)
    gpu, _ = pair(2 * nb, 1, D, block, "q4", table)
    fill_summaries(gpu, torch.Generator().manual_seed(1))
    q = torch.randn(3, 2, D).to(torch.bfloat16).to(DEV)
    m = S.make_method("exp", rho_min=0.5, tau=2.0, k_min=2)
    budget, kcap = S.stem_decode_budget(nb, m, DEV)

    def go(lens, rows_, budget=budget, kcap=kcap):
        st = status_word()
        idx, cnt = S.stem_decode_select(gpu, q, i32(lens), budget, kcap, m, rows=i32(rows_),
                                        status=st)
        return int(st), idx.cpu(), cnt.cpu()

    ok = go([500, 512, 1], [0, 1, 1])
    assert ok[0] == 0
    for lens, rows_ in (([500, 513, 1], [0, 1, 1]), ([500, 512, 1], [0, 2, 1]),
                        ([500, -1, 1], [0, 1, 1]), ([500, 512, 1], [0, -1, 1])):
        st, idx, cnt = go(lens, rows_)
        assert st == base.STEM_ERR_ARG
        assert not cnt[1].any() and (idx[1] == -1).all()  # the bad row keeps nothing
        assert torch.equal(idx[0], ok[1][0]) and torch.equal(idx[2], ok[1][2])  # the others stand
    st, idx, cnt = go([500, 512, 1], [0, 1, 1], budget=torch.full_like(budget, 100))
    assert st == base.STEM_ERR_ARG and int(cnt.max()) <= kcap
    st, idx, cnt = go([500, 512, 1], [0, 1, 1], kcap=2)
    assert st == base.STEM_ERR_ARG and int(cnt.max()) == 2
    gpu.table[0, 3] = 77
    st, idx, cnt = go([500, 512, 1], [0, 1, 1])
    assert st == base.STEM_ERR_ARG and 3 not in idx[0, 0, :int(cnt[0, 0])].tolist()


# ------------------------------------------------------------------ attention


def filled(fmt, D, block, Hkv, lens, g, vsum="mean", max_blocks=None, fill=0xFF):
    nb = [max(-(-n // block), 1) for n in lens]
    table, pages = make_table(nb, max_blocks or max(nb))
    gpu, cpu = pair(pages, Hkv, D, block, fmt, table, vsum, fill)
    T = max(lens)
    k, v = rows(g, len(lens), Hkv, T, D), rows(g, len(lens), Hkv, T, D)
    S.stem_cache_append(gpu, k.to(DEV), v.to(DEV), i32([0] * len(lens)), i32(lens))
    cpu.pages[:] = gpu.pages.cpu().numpy()  # (the bytes themselves are tested above)
    cpu.kbar, cpu.vnorm = gpu.kbar.cpu().double(), gpu.vnorm.cpu().double()
    return gpu, cpu


def random_lists(g, lens, row_seq, Hq, G, block, share, most):
    out = []
    for r in range(len(lens)):
        last = -(-lens[r] // block) - 1
        heads = []
        for h in range(Hq):
            if share == "group" and h % G:
                heads.append(heads[-1])
            elif last < 0:
                heads.append([])
            else:
                n = int(torch.randint(1, min(last + 1, most) + 1, (1,), generator=g))
                pick = torch.randperm(last + 1, generator=g)[:n].tolist()
                heads.append(sorted(set(pick) | {last}) if h % 3 else sorted(pick))
        out.append(heads)
    return out


def as_tensors(lists, kcap):
    R, Hq = len(lists), len(lists[0])
    idx = torch.full((R, Hq, kcap), 12345, dtype=torch.int32)  # past the count: anything
    cnt = torch.zeros(R, Hq, dtype=torch.int32)
    for r in range(R):
        for h in range(Hq):
            idx[r, h, :len(lists[r][h])] = torch.tensor(lists[r][h], dtype=torch.int32)
            cnt[r, h] = len(lists[r][h])
    return idx.to(DEV), cnt.to(DEV)


def check_attn(cpu, fmt, q, row_seq, lens, lists, out, lse):
    R, Hq, D = q.shape
    G = Hq // cpu.Hkv
    out, lse = out.cpu().double(), lse.cpu().double()
    for r in range(R):
        for h in range(Hq):
            k, v = cpu.tokens(row_seq[r], h // G, lists[r][h], lens[r])
            o, z = ref.attend(q[r, h], k, v)
            tol, dl = ref.attn_tolerance(q[r, h], k, v, fmt, o)
            assert torch.all((out[r, h] - o).abs() <= tol), (r, h, float((out[r, h] - o).abs().max()))
            if k.shape[0] == 0:
                assert float(lse[r, h]) == -math.inf and not out[r, h].any()
            else:
                assert abs(float(lse[r, h]) - z) <= dl, (r, h)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D,block", SHAPES)
@pytest.mark.parametrize("share,G", [("head", 1), ("head", 4), ("group", 7), ("group", 8),
                                     ("head", 3)])
def test_attention_matches_the_definition(fmt, D, block, share, G):
    g = torch.Generator().manual_seed(G + D)
    Hkv = 2
    lens_seq = [5 * block + 17, 1, block, 2 * block + 1, 15, 3 * block - 1]
    gpu, cpu = filled(fmt, D, block, Hkv, lens_seq, g)
    row_seq = [0, 1, 2, 3, 4, 5, 0, 3]
    lens = [lens_seq[s] for s in row_seq]
    lens[6], lens[7] = 3 * block + 16, 0
    lists = random_lists(g, lens, row_seq, Hkv * G, G, block, share, 6)
    idx, cnt = as_tensors(lists, 6)
    q = rows(g, len(lens), Hkv * G, D)
    st = status_word()
    out, lse = S.stem_decode_attn(gpu, q.to(DEV), i32(lens), idx, cnt, share=share, rows=i32(row_seq),
                                  status=st)
    assert int(st) == 0
    check_attn(cpu, fmt, q, row_seq, lens, lists, out, lse)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("share,G", [("group", 12), ("head", 17)])
def test_attention_of_more_heads_than_a_tile_holds(fmt, share, G):
    g = torch.Generator().manual_seed(G)
    gpu, cpu = filled(fmt, 64, 64, 1, [200, 63], g)
    lens = [200, 63]
    lists = random_lists(g, lens, [0, 1], G, G, 64, share, 4)
    idx, cnt = as_tensors(lists, 4)
    q = rows(g, 2, G, 64)
    out, lse = S.stem_decode_attn(gpu, q.to(DEV), i32(lens), idx, cnt, share=share)
    check_attn(cpu, fmt, q, [0, 1], lens, lists, out, lse)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows_per_seq", [1, 200])
def test_attention_over_whole_long_sequences(fmt, rows_per_seq):
    """Every block kept, a list long enough to be split over many CTAs or over none."""
    g = torch.Generator().manual_seed(9)
    D, block, n = 128, 128, 128 * 20 + 77
    gpu, cpu = filled(fmt, D, block, 1, [n], g)
    nb = 21
    R = rows_per_seq
    lens = [n] * R
    lists = [[list(range(nb))] * 2] * R
    idx, cnt = as_tensors(lists, nb)
    q = rows(g, R, 2, D)
    out, lse = S.stem_decode_attn(gpu, q.to(DEV), i32(lens), idx, cnt, share="group",
                                  rows=i32([0] * R))
    some = [0] if R == 1 else [0, 57, R - 1]
    check_attn(cpu, fmt, q[some], [0] * len(some), [n] * len(some), [lists[r] for r in some],
               out[some], lse[some])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("lens,share", [([200 * 64 - 5], "group"),  # many parts, joined by a kernel
                                        ([600 * 64, 64 * 31 + 7, 1, 64 * 390], "group"),
                                        ([64 * 150, 64 * 90 + 33], "head")])
def test_attention_over_lists_of_many_parts(fmt, lens, share):
    """A few long items: every block of ragged sequences, split over all the CTAs that there are."""
    g = torch.Generator().manual_seed(len(lens))
    D, block, G = 64, 64, 2
    gpu, cpu = filled(fmt, D, block, 1, lens, g)
    nb = [-(-n // block) for n in lens]
    lists = [[list(range(n))] * G for n in nb]
    if share == "head":
        lists = [[x[0], x[0][::2]] for x in lists]
    idx, cnt = as_tensors(lists, max(nb))
    q = rows(g, len(lens), G, D)
    out, lse = S.stem_decode_attn(gpu, q.to(DEV), i32(lens), idx, cnt, share=share)
    check_attn(cpu, fmt, q, list(range(len(lens))), lens, lists, out, lse)


@pytest.mark.parametrize("fmt", FORMATS)
def test_attention_with_long_parts(fmt):
    """So many rows that a CTA's part is longer than what it stages at a time, and rows between them
    that keep nothing."""
    g = torch.Generator().manual_seed(31)
    D, block, nb, R = 64, 64, 300, 700
    gpu, cpu = filled(fmt, D, block, 1, [nb * block - 9], g)
    lens = [0 if r % 5 == 3 else (nb * block - 9 if r % 2 else 64 * 77) for r in range(R)]
    every = [-(-n // block) for n in lens]
    idx = torch.arange(nb, dtype=torch.int32, device=DEV).expand(R, 1, nb).contiguous()
    cnt = i32(every)[:, None].contiguous()
    q = rows(g, R, 1, D)
    out, lse = S.stem_decode_attn(gpu, q.to(DEV), i32(lens), idx, cnt, share="group",
                                  rows=i32([0] * R))
    some = [0, 1, 3, 350, 351, R - 1]
    check_attn(cpu, fmt, q[some], [0] * len(some), [lens[r] for r in some],
               [[list(range(every[r]))] for r in some], out[some], lse[some])
    none = [r for r in range(R) if lens[r] == 0]
    assert not out[none].any() and (lse[none] == -math.inf).all()
    same = [r for r in range(R) if lens[r] == 64 * 77 and r % 5 != 3]
    at = slice(same[7], same[7] + 1)
    one = S.stem_decode_attn(gpu, q[at].to(DEV), i32([64 * 77]), idx[:1], cnt[at], share="group")
    assert torch.allclose(one[0].float(), out[at].float(), rtol=2 ** -6, atol=1e-3)


@pytest.mark.parametrize("fmt", ["q8", "q4"])
def test_every_quotient_of_two_bfloat16_significands(fmt):
    """All 128 significands of the largest element against all of the others', at several ratios:
    codes equal those of the division in 64 bits (ties to even)."""
    D, block = 64, 64
    top = torch.arange(128, 256, dtype=torch.float64).repeat_interleave(5)  # largest of the group
    scale = (top.float() / ref.QMAX[fmt]).to(torch.bfloat16).double()
    vals = torch.arange(128, 256, dtype=torch.float64)
    blocks = []
    for i in range(top.numel()):
        r = 2.0 ** -(i % 5)
        x = vals[torch.randperm(128, generator=torch.Generator().manual_seed(i))] * r
        x = torch.minimum(x, top[i])
        for part in x.reshape(-1, 31)[:4] if x.numel() % 31 == 0 else x[:124].reshape(4, 31):
            blocks.append((torch.cat([top[i:i + 1], part]), scale[i]))
    x = torch.stack([b[0] for b in blocks])
    s = torch.stack([b[1] for b in blocks])
    want = torch.round(x / s[:, None]).clamp(-ref.QMAX[fmt], ref.QMAX[fmt]) * s[:, None]
    k = x.reshape(1, 1, -1, D).to(torch.bfloat16)
    T = k.shape[2]
    table, pages = make_table([-(-T // block)], -(-T // block))
    gpu, _ = pair(pages, 1, D, block, fmt, table)
    S.stem_cache_append(gpu, k.to(DEV), -k.to(DEV), i32([0]))
    got, neg = S.stem_cache_read(gpu, i32([0]), T=T, dtype=torch.float32)
    assert torch.equal(got.cpu().double().reshape(-1, 32), want)
    assert torch.equal(neg, -got)


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_head_is_untouched_by_blocks_it_does_not_keep(fmt):
    """Per-head lists: NaN and infinities in a block that one head keeps reach that head alone."""
    g = torch.Generator().manual_seed(4)
    D, block, G = 128, 64, 4
    lens = [4 * block]
    gpu, cpu = filled(fmt, D, block, 1, lens, g)
    x = rows(g, 1, 1, block, D)
    bad = x.clone()
    bad[0, 0, 3, 5], bad[0, 0, 9, 100] = float("nan"), float("inf")
    S.stem_cache_append(gpu, x.to(DEV), bad.to(DEV), i32([block]))
    cpu.pages[:] = gpu.pages.cpu().numpy()
    lists = [[[0, 3], [0, 1, 3], [2, 3], [3]]]
    idx, cnt = as_tensors(lists, 4)
    q = rows(g, 1, G, D)
    out, lse = S.stem_decode_attn(gpu, q.to(DEV), i32(lens), idx, cnt, share="head")
    keep = [0, 2, 3]
    k_out, k_lse = out[:, keep], lse[:, keep]
    assert torch.isfinite(k_out).all() and torch.isfinite(lse).all()
    for h in keep:
        k, v = cpu.tokens(0, 0, lists[0][h], lens[0])
        o, z = ref.attend(q[0, h], k, v)
        tol, dl = ref.attn_tolerance(q[0, h], k, v, fmt, o)
        assert torch.all((out[0, h].cpu().double() - o).abs() <= tol)
        assert abs(float(lse[0, h]) - z) <= dl
    assert torch.isnan(out[0, 1, 5]) and not torch.isfinite(out[0, 1, 100])


@pytest.mark.parametrize("fmt", ["q8", "q4"])
def test_value_scales_over_the_whole_range(fmt):
    """V rows from 1e-37 to 1e37: the weights' power of two follows the largest seen."""
    g = torch.Generator().manual_seed(6)
    D, block, n = 64, 64, 192
    for mags in ([1e37, 1.0, 1e-37], [1e-37, 1e-30, 1e-20], [1e-37, 1.0, 1e37]):
        table, pages = make_table([3], 3)
        gpu, cpu = pair(pages, 1, D, block, fmt, table)
        k, v = rows(g, 1, 1, n, D), torch.randn(1, 1, n, D, generator=g)
        v = (v * torch.tensor(mags).repeat_interleave(64)[None, None, :, None]).to(torch.bfloat16)
        S.stem_cache_append(gpu, k.to(DEV), v.to(DEV), i32([0]))
        cpu.pages[:] = gpu.pages.cpu().numpy()
        q = rows(g, 1, 2, D)
        for lists in ([[[0, 1, 2], [0, 1, 2]]], [[[0], [1, 2]]], [[[2], [0, 1]]]):
            idx, cnt = as_tensors(lists, 3)
            out, lse = S.stem_decode_attn(gpu, q.to(DEV), i32([n]), idx, cnt)
            for h in range(2):
                kk, vv = cpu.tokens(0, 0, lists[0][h], n)
                o, z = ref.attend(q[0, h], kk, vv)
                tol, _ = ref.attn_tolerance(q[0, h], kk, vv, fmt, o)
                # a weight far below the tile's largest scale may round to 0: 2^-24 of 2^14 of it
                top = vv.abs().max() * 2.0 ** -30
                assert torch.all((out[0, h].cpu().double() - o).abs() <= tol + top)


@pytest.mark.parametrize("fmt", FORMATS)
def test_large_queries_and_flat_logits(fmt):
    g = torch.Generator().manual_seed(8)
    gpu, cpu = filled(fmt, 64, 64, 1, [130], g)
    for mag in (0.0, 1e-30, 1e-3, 30.0, 1e4):
        q = (rows(g, 1, 2, 64).float() * mag).to(torch.bfloat16)
        lists = [[[0, 1, 2], [1, 2]]]
        idx, cnt = as_tensors(lists, 3)
        out, lse = S.stem_decode_attn(gpu, q.to(DEV), i32([130]), idx, cnt)
        check_attn(cpu, fmt, q, [0], [130], lists, out, lse)


def test_attention_reports_bad_lists_and_pages():
    g = torch.Generator().manual_seed(8)
    for share in ("head", "group"):
        gpu, cpu = filled("q4", 64, 64, 1, [400], g)
        q = rows(g, 1, 2, 64)
        lens = [400]
        for bad in ([0, 7, 3], [0, -4, 3], [0, 1 << 20, 3]):
            idx, cnt = as_tensors([[bad, bad]], 3)
            st = status_word()
            out, lse = S.stem_decode_attn(gpu, q.to(DEV), i32(lens), idx, cnt, share=share, status=st)
            assert int(st) == base.STEM_ERR_ARG
            check_attn(cpu, "q4", q, [0], lens, [[[0, 3], [0, 3]]], out, lse)
        idx, cnt = as_tensors([[[0, 2, 3], [0, 2, 3]]], 3)
        st = status_word()
        S.stem_decode_attn(gpu, q.to(DEV), i32(lens), idx, torch.full_like(cnt, 9), share=share,
                           status=st)
        assert int(st) == base.STEM_ERR_ARG
        gpu.table[0, 2] = 1 << 30
        st = status_word()
        out, lse = S.stem_decode_attn(gpu, q.to(DEV), i32(lens), idx, cnt, share=share, status=st)
        assert int(st) == base.STEM_ERR_ARG
        check_attn(cpu, "q4", q, [0], lens, [[[0, 3], [0, 3]]], out, lse)


def test_pages_beyond_four_gigabytes():
    """Page offsets need more than 32 bits."""
    D, block, Hkv, fmt = 128, 128, 8, "bf16"
    size = S.stem_cache_page_bytes(D, block, fmt)
    pages = (5 << 30) // (size * Hkv)
    table = np.array([[pages - 1, 0, pages - 2]], dtype=np.int32)
    c = S.PagedCache(torch.empty(pages, Hkv, size, dtype=torch.uint8, device=DEV),
                     torch.empty(pages, Hkv, D, device=DEV), torch.empty(pages, Hkv, device=DEV),
                     torch.from_numpy(table).to(DEV), block, fmt)
    small = S.PagedCache.alloc(3, Hkv, D, block, fmt,
                               torch.tensor([[0, 1, 2]], dtype=torch.int32, device=DEV))
    g = torch.Generator().manual_seed(1)
    k, v = rows(g, 1, Hkv, 300, D).to(DEV), rows(g, 1, Hkv, 300, D).to(DEV)
    q = rows(g, 1, Hkv, D).to(DEV)
    m = S.make_method("exp", rho_min=1.0, tau=1.0)
    budget, kcap = S.stem_decode_budget(3, m, DEV)
    got = []
    for cc in (c, small):
        S.stem_cache_append(cc, k, v, i32([0]))
        got.append(S.stem_decode(cc, q, i32([300]), budget, kcap, m) +
                   S.stem_cache_read(cc, i32([0]), T=300))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert torch.equal(got[0][4], k)


# ------------------------------------------------------------------ together


@pytest.mark.parametrize("fmt,share,metric,vsum", [("bf16", "head", "product", "mean"),
                                                   ("q8", "group", "additive", "max"),
                                                   ("q4", "group", "product", "mean"),
                                                   ("q4", "head", "additive", "max")])
def test_generation_from_a_prefilled_prompt(fmt, share, metric, vsum):
    """A prompt goes through the framework's prefill, its K and V into the cache; then tokens are
    generated one at a time: append, decode. Each step's lists and outputs match the definition, and
    a batch of sequences gives what each gives alone."""
    g = torch.Generator().manual_seed(11)
    D, block, Hkv, G = 64, 64, 2, 2
    prompt, new = [500, 190], 5
    m = S.make_method("exp", rho_min=0.3, tau=3.0, k_min=2, metric=metric, beta=0.2, vsum=vsum,
                      share=share)
    total = [n + new for n in prompt]
    nb = [-(-n // block) for n in total]
    table, pages = make_table(nb, max(nb))
    gpu, cpu = pair(pages, Hkv, D, block, fmt, table, vsum)
    T = max(total)
    k, v = rows(g, 2, Hkv, T, D), rows(g, 2, Hkv, T, D)
    q = rows(g, 2, Hkv * G, T, D)
    for s in range(2):
        n = prompt[s]
        args = [x[s:s + 1, :, :n].contiguous().to(DEV) for x in (q, k, v)]
        out, _, _ = base.stem_prefill_ex(*args, block, 0.0, 0.0, 0, method=m)
        assert torch.isfinite(out).all()
    S.stem_cache_append(gpu, k.to(DEV)[:, :, :max(prompt)], v.to(DEV)[:, :, :max(prompt)],
                        i32([0, 0]), i32(prompt))
    budget, kcap = S.stem_decode_budget(max(nb), m, DEV)
    for t in range(new):
        pos = [n + t for n in prompt]
        kt = torch.stack([k[s, :, pos[s]] for s in range(2)])[:, :, None].to(DEV)
        vt = torch.stack([v[s, :, pos[s]] for s in range(2)])[:, :, None].to(DEV)
        qt = torch.stack([q[s, :, pos[s]] for s in range(2)])
        S.stem_cache_append(gpu, kt, vt, i32(pos))
        lens = [p + 1 for p in pos]
        st = status_word()
        out, lse, idx, cnt = S.stem_decode(gpu, qt.to(DEV), i32(lens), budget, kcap, m, status=st)
        assert int(st) == 0
        cpu.pages[:] = gpu.pages.cpu().numpy()
        check_select(gpu, qt, [0, 1], lens, budget.tolist(), gpu.kbar.cpu(), gpu.vnorm.cpu(), table,
                     share, metric, float(np.float32(0.2)), True, idx, cnt, kcap)
        lists = [[idx[r, h, :int(cnt[r, h])].tolist() for h in range(Hkv * G)] for r in range(2)]
        check_attn(cpu, fmt, qt, [0, 1], lens, lists, out, lse)
        for s in range(2):
            one = S.stem_decode(gpu, qt[s:s + 1].to(DEV), i32([lens[s]]), budget, kcap, m,
                                rows=i32([s]))
            assert torch.equal(one[2], idx[s:s + 1]) and torch.equal(one[3], cnt[s:s + 1])
            assert torch.allclose(one[0].float(), out[s:s + 1].float(), rtol=2 ** -6, atol=1e-3)


def test_captured_steps_replay_with_new_lengths_and_overlap():
    """Two captured steps, each with its own workspace, replayed at once on two streams after the
    lengths, the cache and the queries have changed; and repeated calls give the same bits."""
    g = torch.Generator().manual_seed(12)
    D, block, Hkv, G, n = 128, 64, 2, 4, 900
    gpu, _ = filled("q4", D, block, Hkv, [n], g)
    m = S.make_method("exp", rho_min=0.3, tau=3.0, k_min=2, share="group")
    budget, kcap = S.stem_decode_budget(gpu.max_blocks, m, DEV)
    side, graphs = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for st in side:
        b = dict(q=rows(g, 1, Hkv * G, D).to(DEV), lens=i32([300]),
                 k=rows(g, 1, Hkv, 1, D).to(DEV), pos=i32([299]))
        S.stem_decode(gpu, b["q"], b["lens"], budget, kcap, m)  # warm
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            b["out"] = S.stem_decode(gpu, b["q"], b["lens"], budget, kcap, m)
        graphs.append((graph, b))
    for length in (900, 65, 1, 640):
        for _, b in graphs:
            b["q"].copy_(rows(g, 1, Hkv * G, D))
            b["lens"].fill_(length)
        torch.cuda.synchronize()
        for _ in range(3):
            for st, (graph, _) in zip(side, graphs):
                with torch.cuda.stream(st):
                    graph.replay()
        torch.cuda.synchronize()
        for _, b in graphs:
            want = S.stem_decode(gpu, b["q"], b["lens"], budget, kcap, m)
            for x, y in zip(b["out"], want):
                assert torch.equal(x, y)


def test_the_binding_refuses_wrong_tensors():
    g = torch.Generator().manual_seed(14)
    gpu, _ = filled("q8", 64, 64, 2, [300, 64], g)
    m = S.make_method("exp", rho_min=0.3, tau=3.0, k_min=2)
    budget, kcap = S.stem_decode_budget(gpu.max_blocks, m, DEV)
    q, lens = rows(g, 2, 4, 64).to(DEV), i32([300, 64])

    def no(error, match, fn, *args, **kw):
        with pytest.raises(error, match=match):
            fn(*args, **kw)

    d = (gpu, q, lens, budget, kcap, m)
    no(TypeError, "q must be", S.stem_decode, gpu, q.float(), *d[2:])
    no(ValueError, "contiguous", S.stem_decode, gpu, q.transpose(0, 1).contiguous().transpose(0, 1),
       *d[2:])
    no(ValueError, "cuda", S.stem_decode, gpu, q.cpu(), *d[2:])
    no(TypeError, "lens must be", S.stem_decode, gpu, q, lens.long(), budget, kcap, m)
    no(ValueError, "shape", S.stem_decode, gpu, q, lens[:1], budget, kcap, m)
    no(ValueError, "shape", S.stem_decode, gpu, q, lens, budget[:-1].contiguous(), kcap, m)
    no(ValueError, "kcap", S.stem_decode, gpu, q, lens, budget, 0, m)
    no(S.StemError, "invalid argument", S.stem_decode, gpu, q, lens, budget, 99, m)
    no(ValueError, "both", S.stem_decode_select, *d, sel_idx=torch.empty(2, 4, kcap, device=DEV))
    no(TypeError, "rows must be a tensor", S.stem_decode, *d, rows=[0, 1])
    no(S.StemError, "workspace", S.stem_decode, *d,
       workspace=torch.empty(512, dtype=torch.uint8, device=DEV))
    no(TypeError, "PagedCache", S.stem_decode, None, *d[1:])
    odd = S.make_method("exp", rho_min=0.3, tau=3.0, score="antidiag")
    no(S.StemError, "limits", S.stem_decode, gpu, q, lens, budget, kcap, odd)
    k = torch.zeros(2, 2, 5, 64, dtype=torch.bfloat16, device=DEV)
    no(TypeError, "bfloat16 or float32", S.stem_cache_append, gpu, k.half(), k.half(), i32([0, 0]))
    no(ValueError, "same shape", S.stem_cache_append, gpu, k, k[:, :, :4], i32([0, 0]))
    turned = k.transpose(2, 3).contiguous().transpose(2, 3)
    no(ValueError, "last dimension", S.stem_cache_append, gpu, turned, turned, i32([0, 0]))
    wide = torch.zeros(2, 2, 5, 67, dtype=torch.bfloat16, device=DEV)[..., :64]
    no(S.StemError, "invalid argument", S.stem_cache_append, gpu, wide, wide, i32([0, 0]))
    no(ValueError, "k must be", S.stem_cache_append, gpu, k[:1], k[:1], i32([0, 0]))
    no(ValueError, "T is needed", S.stem_cache_read, gpu, i32([0, 0]))
    one = k[:, :, :1].expand(2, 2, 5, 64)
    no(S.StemError, "invalid argument", S.stem_cache_read, gpu, i32([0, 0]), k=one, v=one)
    S.stem_cache_append(gpu, one, one, i32([64, 0]))  # (many readers are fine)
    idx, cnt = S.stem_decode_select(gpu, q, lens, budget, kcap, m)
    no(TypeError, "sel_cnt must be", S.stem_decode_attn, gpu, q, lens, idx, None)
    no(TypeError, "sel_cnt must be", S.stem_decode_attn, gpu, q, lens, None, cnt)


def test_rows_read_back_on_another_stream():
    """The zeros behind a sequence's rows are written before the rows, on the call's stream: with the
    current stream busy, nothing of it comes after them."""
    g = torch.Generator().manual_seed(15)
    gpu, _ = filled("q4", 64, 64, 2, [300, 64], g)
    want = S.stem_cache_read(gpu, i32([3, 0]), i32([200, 64]), T=200)
    pos, count = i32([3, 0]), i32([200, 64])
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    torch.cuda._sleep(20_000_000)
    got = S.stem_cache_read(gpu, pos, count, T=200, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_another_stream_and_given_buffers():
    g = torch.Generator().manual_seed(13)
    gpu, _ = filled("q8", 64, 64, 2, [300, 64], g)
    m = S.make_method("exp", rho_min=0.3, tau=3.0, k_min=2)
    budget, kcap = S.stem_decode_budget(gpu.max_blocks, m, DEV)
    q, lens = rows(g, 2, 4, 64).to(DEV), i32([300, 64])
    want = S.stem_decode(gpu, q, lens, budget, kcap, m)
    bufs = [torch.empty_like(x) for x in want]
    ws = torch.empty(S.stem_decode_workspace_size(gpu, 2, 4, kcap), dtype=torch.uint8, device=DEV)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    S.stem_decode(gpu, q, lens, budget, kcap, m, out=bufs[0], lse=bufs[1], sel_idx=bufs[2],
                  sel_cnt=bufs[3], workspace=ws, stream=st)
    st.synchronize()
    for x, y in zip(bufs, want):
        assert torch.equal(x, y)
    # what a call makes itself belongs to its stream: freed, it serves that stream again
    made = S.stem_decode(gpu, q, lens, budget, kcap, m, stream=st)
    st.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(made, want))
    ptrs = {x.data_ptr() for x in made}
    del made
    mine = [torch.empty(x.shape, dtype=x.dtype, device=DEV) for x in want]
    assert ptrs.isdisjoint(x.data_ptr() for x in mine)
