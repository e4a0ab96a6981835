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
