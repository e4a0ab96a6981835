"""The decode path on a B200 where sizes, ranges and callers are unlike the ordinary ones: tables wider than
the sequences in them, scores and values far from 1, several threads, against tests/decode_ref.py."""

import math
import os
import subprocess

import numpy as np
import pytest
import torch

from block_sparse_causal_pooling_b200 import build as libbuild
from block_sparse_causal_pooling_b200 import decode as S
from block_sparse_causal_pooling_b200 import stem as base
from tests import decode_ref as ref
from tests import test_gpu_decode as common

pytestmark = pytest.mark.gpu

DEV = common.DEV
HERE = os.path.dirname(os.path.abspath(__file__))
i32, rows, status_word = common.i32, common.rows, common.status_word


# ------------------------------------------------------------------ selection


@pytest.mark.parametrize("share", ["head", "group"])
@pytest.mark.parametrize("metric", ["product", "additive"])
@pytest.mark.parametrize("wide,Hkv", [(100, 20), (300, 20), (700, 2), (4096, 1)])
def test_select_of_short_rows_in_a_wide_table(share, metric, wide, Hkv):
    """Clusters of 2, 4 and 8 CTAs some of which have no block of a row: they are the first to write
    into the others' shared memory, right at the start of a launch. Many launches one after the other,
    each with the same answer."""
    g = torch.Generator().manual_seed(wide)
    D, block, G = 64, 64, 3
    lens = [64 * (wide // 7) - 5, 64 * 3, 64 * (wide // 2)]
    nb = [-(-n // block) for n in lens]
    table, pages = common.make_table(nb, wide)
    gpu, _ = common.pair(pages, Hkv, D, block, "q4", table)
    kb, vn = common.fill_summaries(gpu, g)
    q = rows(g, 3, Hkv * G, D)
    m = S.make_method("exp", rho_min=0.2, tau=4.0, k_min=3, share=share, metric=metric, beta=0.2)
    budget, kcap = S.stem_decode_budget(wide, m, DEV)
    st = status_word()
    dq, dl = q.to(DEV), i32(lens)
    idx, cnt = S.stem_decode_select(gpu, dq, dl, budget, kcap, m, status=st)
    assert int(st) == 0
    common.check_select(gpu, q, [0, 1, 2], lens, budget.tolist(), kb, vn, table, share, metric,
                        float(np.float32(0.2)), True, idx, cnt, kcap)
    again = [S.stem_decode_select(gpu, dq, dl, budget, kcap, m) for _ in range(50)]
    for i, c in again:
        assert torch.equal(i, idx) and torch.equal(c, cnt)


@pytest.mark.parametrize("wide", [100, 200, 700, 4096])
@pytest.mark.parametrize("sign", [-1.0, 1.0])
def test_select_of_scores_far_from_zero(wide, sign):
    """Every score of every head near -960, or near 960, where exp of it is 0 or infinite in 64 bits too:
    what decides are the differences, whatever share of the cluster's CTAs has a block of the row."""
    g = torch.Generator().manual_seed(17)
    D, block, G, n = 64, 64, 4, 100
    table, pages = common.make_table([n], wide)
    gpu, _ = common.pair(pages, 1, D, block, "q4", table)
    kb, vn = common.fill_summaries(gpu, g, scale=0.2)
    kb = kb + sign * 10.0
    gpu.kbar.copy_(kb)
    q = (12.0 + 0.1 * torch.randn(2, G, D, generator=g)).to(torch.bfloat16)
    lens = [n * block - 3, 77 * block]
    m = S.make_method("exp", rho_min=0.2, tau=4.0, k_min=3, share="group")
    budget, kcap = S.stem_decode_budget(wide, m, DEV)
    idx, cnt = S.stem_decode_select(gpu, q.to(DEV), i32(lens), budget, kcap, m, rows=i32([0, 0]))
    common.check_select(gpu, q, [0, 0], lens, budget.tolist(), kb, vn, table, "group", "product", 0.0,
                        True, idx, cnt, kcap)


def test_select_from_two_threads_over_tables_of_different_widths(tmp_path):
    """A narrow table's launch asks for less shared memory than a wide one's, of the same kernel: what
    one thread sets for its launch must not refuse another's."""
    exe, lib = str(tmp_path / "threads"), os.path.dirname(base.LIB_PATH)
    cmd = [libbuild._nvcc()] + libbuild.ARCH + ["-std=c++17", "-I", libbuild.INCLUDE, "-o", exe,
                                                os.path.join(HERE, "decode_threads.cu"), "-L", lib,
                                                "-l:libstem.so", "-Xlinker", "-rpath", "-Xlinker", lib]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout


# ------------------------------------------------------------------ attention


def check_scaled(cpu, fmt, q, lists, n, out, lse):
    """check_attn of one row whose V rows may be of any size. Its tolerance counts a weight's rounding to
    fp16, 2^-11 of it; below fp16's normal range weights may together be off by 2^-12 of their sum in a
    channel group, of values up to the largest of each token's group."""
    D, G = q.shape[2], q.shape[1] // cpu.Hkv
    for h in range(q.shape[1]):
        k, v = cpu.tokens(0, h // G, lists[h], n)
        o, z = ref.attend(q[0, h], k, v)
        tol, dl = ref.attn_tolerance(q[0, h], k, v, fmt, o)
        w = torch.softmax(k @ q[0, h].double() / math.sqrt(D), 0)
        top = v.abs().reshape(-1, D // 32, 32).amax(-1, keepdim=True).expand(-1, -1, 32).reshape(-1, D)
        err = (out[0, h].cpu().double() - o).abs()
        assert torch.all(err <= tol + 2.0 ** -12 * (w @ top)), (h, float((err / (w @ top)).max()))
        assert abs(float(lse[0, h]) - z) <= dl


def one_sequence(fmt, D, block, k, v):
    n = k.shape[2]
    table, pages = common.make_table([-(-n // block)], -(-n // block))
    gpu, cpu = common.pair(pages, k.shape[1], D, block, fmt, table)
    S.stem_cache_append(gpu, k.to(DEV), v.to(DEV), i32([0]))
    cpu.pages[:] = gpu.pages.cpu().numpy()
    return gpu, cpu


@pytest.mark.parametrize("fmt", ["q8", "q4"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("powers", [(0, -9, -14, -20), (0, -30, -30, -30), (-40, 0, -60, 12),
                                    (-60, 40, 0, -19)])
def test_channel_groups_of_unlike_size(fmt, D, powers):
    """Values of each group of 32 channels at a scale of its own: none costs another its digits, however
    the weights are spread over the tokens."""
    g = torch.Generator().manual_seed(33)
    n, block = 1000, 64
    size = 2.0 ** torch.tensor(powers[:D // 32], dtype=torch.float64).repeat_interleave(32)
    k = rows(g, 1, 1, n, D)
    v = (torch.randn(1, 1, n, D, generator=g).double() * size).to(torch.bfloat16)
    gpu, cpu = one_sequence(fmt, D, block, k, v)
    for mag in (0.0, 0.5, 4.0):
        q = (rows(g, 1, 3, D).float() * mag).to(torch.bfloat16)
        lists = [list(range(16)), [0, 3, 15], [15]]
        idx, cnt = common.as_tensors([lists], 16)
        out, lse = S.stem_decode_attn(gpu, q.to(DEV), i32([n]), idx, cnt)
        check_scaled(cpu, fmt, q, lists, n, out, lse)


@pytest.mark.parametrize("fmt", ["q8", "q4"])
@pytest.mark.parametrize("power", [10, 25, 40])
def test_a_large_value_that_hardly_weighs(fmt, power):
    """One token with values 2^power times the others' and next to no weight: the others' digits stay,
    for the heads that keep its block and for those that do not."""
    g = torch.Generator().manual_seed(34)
    D, n, block = 64, 700, 64
    k, v = torch.randn(2, 1, 1, n, D, generator=g)
    q = torch.ones(1, 4, D) + 0.1 * torch.randn(1, 4, D, generator=g)
    at = 333
    k[0, 0, at] = -1.5 * power / 12  # a logit some `power` below the others, in ln
    v[0, 0, at] *= 2.0 ** power
    q, k, v = (x.to(torch.bfloat16) for x in (q, k, v))
    gpu, cpu = one_sequence(fmt, D, block, k, v)
    every = list(range(11))
    lists = [every, every, [b for b in every if b != at // block], [at // block, 10]]
    idx, cnt = common.as_tensors([lists], 11)
    out, lse = S.stem_decode_attn(gpu, q.to(DEV), i32([n]), idx, cnt)
    check_scaled(cpu, fmt, q, lists, n, out, lse)


@pytest.mark.parametrize("fmt", ["q8", "q4"])
def test_values_next_to_the_types_limits(fmt):
    """Values from the smallest normal numbers to ones whose sum over the tokens is just finite, in the
    same row."""
    g = torch.Generator().manual_seed(35)
    D, n, block = 128, 128, 64
    size = 2.0 ** torch.tensor((-120, 112, -100, 0), dtype=torch.float64).repeat_interleave(32)
    k = rows(g, 1, 1, n, D)
    v = (torch.randn(1, 1, n, D, generator=g).double() * size).to(torch.bfloat16)
    gpu, cpu = one_sequence(fmt, D, block, k, v)
    q = rows(g, 1, 2, D)
    lists = [[0, 1], [1]]
    idx, cnt = common.as_tensors([lists], 2)
    out, lse = S.stem_decode_attn(gpu, q.to(DEV), i32([n]), idx, cnt)
    o = out[0].cpu().double()
    for h in range(2):
        kk, vv = cpu.tokens(0, 0, lists[h], n)
        want, _ = ref.attend(q[0, h], kk, vv)
        scaled = ref.attn_tolerance(q[0, h], kk, vv / size, fmt, want / size)[0]
        assert torch.all((o[h] - want).abs() / size <= scaled + 2.0 ** -12 * 8)


def test_an_infinite_value_is_infinite_in_the_output():
    """... of its channel, with the sign of the definition, at 16 bits (the others hold no infinity)."""
    g = torch.Generator().manual_seed(37)
    D, n = 64, 200
    k, v = rows(g, 1, 1, n, D), rows(g, 1, 1, n, D)
    v[0, 0, 70, 3], v[0, 0, 130, 9], v[0, 0, 5, 9] = float("inf"), float("-inf"), float("-inf")
    v[0, 0, 6, 20], v[0, 0, 150, 20] = float("inf"), float("-inf")
    gpu, cpu = one_sequence("bf16", D, 64, k, v)
    q = rows(g, 1, 2, D)
    lists = [[0, 1, 2, 3]] * 2
    idx, cnt = common.as_tensors([lists], 4)
    for share in ("head", "group"):
        out, _ = S.stem_decode_attn(gpu, q.to(DEV), i32([n]), idx, cnt, share=share)
        for h in range(2):
            want, _ = ref.attend(q[0, h], *cpu.tokens(0, 0, lists[h], n))
            got = out[0, h].cpu().double()
            odd = ~torch.isfinite(want)
            assert odd.sum() == 3 and torch.isfinite(got[~odd]).all()
            assert torch.equal(got[odd].nan_to_num(0.0), want[odd].nan_to_num(0.0))
            assert torch.equal(torch.isnan(got), torch.isnan(want))


@pytest.mark.parametrize("D,block", common.SHAPES)
def test_weights_at_16_bits_keep_the_digits_of_float32(D, block):
    """At 16 bits nothing but the output is rounded to bf16: what its own rounding leaves is 2^-15 of the
    weights, beside the float32 steps (of 2^-22, as in attn_tolerance)."""
    g = torch.Generator().manual_seed(36)
    n = 5 * block + 9
    k, v = rows(g, 1, 1, n, D), rows(g, 1, 1, n, D)
    gpu, cpu = one_sequence("bf16", D, block, k, v)
    q = rows(g, 1, 8, D)
    lists = [list(range(6)), [0, 5], [5], [1, 2, 3], [0], [0, 1, 2, 4, 5], [4], [3, 5]]
    idx, cnt = common.as_tensors([lists], 6)
    out, lse = S.stem_decode_attn(gpu, q.to(DEV), i32([n]), idx, cnt)
    u = 2.0 ** -22
    for h in range(8):
        kk, vv = cpu.tokens(0, 0, lists[h], n)
        o, z = ref.attend(q[0, h], kk, vv)
        m = kk.shape[0]
        logits = kk @ q[0, h].double() / math.sqrt(D)
        dz = (D + 4) * u * float((kk.abs() @ q[0, h].double().abs()).max()) / math.sqrt(D)
        dz += 4 * u * float(logits.abs().max()) + 8 * u
        w = torch.softmax(logits, 0)
        tol = (w @ vv.abs()) * (2 * dz + 2.0 ** -15 + 2.0 ** -20 + (m // 16 + m + 40) * 2 * u)
        err = (out[0, h].cpu().double() - o).abs()
        assert torch.all(err <= tol + 2.0 ** -8 * (o.abs() + tol)), (h, float((err / o.abs()).max()))
        assert abs(float(lse[0, h]) - z) <= dz + (m // 16 + m % 16 + 40) * u


@pytest.mark.parametrize("wide", [60, 900])
def test_select_with_the_linear_schedule(wide):
    """Rows of a context keep as many blocks in a wide table as in one that fits."""
    g = torch.Generator().manual_seed(41)
    table, pages = common.make_table([60], wide)
    gpu, _ = common.pair(pages, 1, 64, 64, "q8", table)
    kb, vn = common.fill_summaries(gpu, g)
    q = rows(g, 4, 4, 64)
    lens = [60 * 64, 60 * 64 - 70, 64 * 5, 64]
    m = S.make_method("linear", k_start=40.0, mu=0.3, k_min=2)
    budget, kcap = S.stem_decode_budget(wide, m, DEV)
    idx, cnt = S.stem_decode_select(gpu, q.to(DEV), i32(lens), budget, kcap, m, rows=i32([0] * 4))
    most = math.ceil(40.0 * float(np.float32(0.3)))  # 13: the float 0.3 is above 0.3
    assert cnt.cpu().tolist() == [[most] * 4, [most] * 4, [5] * 4, [1] * 4]
    common.check_select(gpu, q, [0] * 4, lens, budget.tolist(), kb, vn, table, "head", "product", 0.0,
                        True, idx, cnt, kcap)


# ------------------------------------------------------------------ the cache


@pytest.mark.parametrize("axis", [0, 1, 2])
def test_rows_whose_strides_differ_along_an_axis_of_one(axis):
    """K as it comes and V as a transposed view hold one layout where an axis has one row."""
    g = torch.Generator().manual_seed(42)
    shape = [2, 3, 4]
    shape[axis] = 1
    B, H, T = shape
    D = 64
    table, pages = common.make_table([1] * B, 1)
    k, v = rows(g, B, H, T, D).to(DEV), rows(g, B, H, T, D).to(DEV)
    step = list(v.stride())
    step[axis] = {0: 3, 1: 7, 2: 5}[axis]
    odd = torch.as_strided(v, v.shape, step)
    assert torch.equal(odd, v) and odd.stride() != k.stride()
    got = []
    for vv in (v, odd):
        gpu, _ = common.pair(pages, H, D, 64, "q8", table)
        S.stem_cache_append(gpu, k, vv, i32([0] * B))
        got.append(S.stem_cache_read(gpu, i32([0] * B), T=T))
        into = [torch.as_strided(torch.zeros_like(v), v.shape, step), torch.zeros_like(v)]
        S.stem_cache_read(gpu, i32([0] * B), k=into[0], v=into[1])
        assert torch.equal(into[0], got[-1][0]) and torch.equal(into[1], got[-1][1])
    for x, y in zip(*got):
        assert torch.equal(x, y)
    one = rows(g, 2, 3, 1, D).to(DEV)
    turned = one.transpose(1, 2).contiguous().transpose(1, 2)  # [B, 1, H, D] seen as [B, H, 1, D]
    table, pages = common.make_table([1, 1], 1)
    gpu, cpu = common.pair(pages, 3, D, 64, "bf16", table)
    S.stem_cache_append(gpu, one, turned, i32([0, 0]))
    k2, v2 = S.stem_cache_read(gpu, i32([0, 0]), T=1)
    assert torch.equal(k2, one) and torch.equal(v2, one)


def test_a_list_longer_than_the_table_is_refused_before_it_is_made():
    """kcap above max_blocks is an invalid argument, not an allocation of that size."""
    g = torch.Generator().manual_seed(43)
    gpu, _ = common.filled("q8", 64, 64, 2, [300, 64], g)
    m = S.make_method("exp", rho_min=0.3, tau=3.0, k_min=2)
    budget, _ = S.stem_decode_budget(gpu.max_blocks, m, DEV)
    q, lens = rows(g, 2, 4, 64).to(DEV), i32([300, 64])
    for call in (S.stem_decode_select, S.stem_decode):
        for kcap in (gpu.max_blocks + 1, 1 << 24, 1 << 40):
            torch.cuda.synchronize()
            torch.cuda.reset_peak_memory_stats()
            before = torch.cuda.memory_allocated()
            with pytest.raises(S.StemError, match="invalid argument"):
                call(gpu, q, lens, budget, kcap, m)
            assert torch.cuda.max_memory_allocated() == before


@pytest.mark.parametrize("fmt", common.FORMATS)
def test_summaries_follow_the_last_token_of_a_block(fmt):
    """A token written again in the middle of a full block changes the token alone; written on to the
    block's end, the summaries are those of the block as it stands."""
    g = torch.Generator().manual_seed(44)
    D, block, n = 64, 64, 128
    k, v = rows(g, 1, 1, n, D).to(DEV), rows(g, 1, 1, n, D).to(DEV)
    new = rows(g, 1, 1, n, D).to(DEV)
    table, pages = common.make_table([2], 2)
    gpu, _ = common.pair(pages, 1, D, block, fmt, table)
    S.stem_cache_append(gpu, k, v, i32([0]))
    kbar, vnorm = gpu.kbar.clone(), gpu.vnorm.clone()
    S.stem_cache_append(gpu, new[:, :, 30:31], new[:, :, 30:31], i32([30]))
    assert torch.equal(gpu.kbar, kbar) and torch.equal(gpu.vnorm, vnorm)
    S.stem_cache_append(gpu, k[:, :, 31:64], v[:, :, 31:64], i32([31]))
    fresh, _ = common.pair(pages, 1, D, block, fmt, table)
    k[:, :, 30], v[:, :, 30] = new[:, :, 30], new[:, :, 30]
    S.stem_cache_append(fresh, k, v, i32([0]))
    assert torch.equal(gpu.pages, fresh.pages)
    assert torch.equal(gpu.kbar, fresh.kbar) and torch.equal(gpu.vnorm, fresh.vnorm)
    assert not torch.equal(gpu.kbar, kbar)
