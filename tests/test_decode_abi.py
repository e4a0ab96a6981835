"""The decode path on the CPU: sizes, the page layout, refusals of the C ABI and of the binding, and
the kernels' index arithmetic on values that only the device reads."""

import ctypes
import json
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from block_sparse_causal_pooling_b200 import build as libbuild
from block_sparse_causal_pooling_b200 import decode as D
from block_sparse_causal_pooling_b200 import stem as S
from tests import decode_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROBE = r"""
import ctypes, json, os, sys
assert os.environ["CUDA_VISIBLE_DEVICES"] == ""
from block_sparse_causal_pooling_b200 import stem as S
L, FAKE = S.lib(), 0x7F0000000000


def cache(**kw):
    c = S.stem_cache_t(FAKE, FAKE, FAKE, FAKE, 100, 2, 128, 128, S.STEM_KV_Q4, 3, 16,
                       S.STEM_VSUM_MEAN)
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c)


def rows(fn, c=None, k=FAKE, v=FAKE, dtype=0, T=4, strides=(2048, 1024, 128), pos=FAKE, count=None,
         status=None):
    st = None if strides is None else (ctypes.c_int64 * 3)(*strides)
    return fn(c or cache(), k, v, dtype, T, st, pos, count, status, None)


KEEP = []


def args(c=None, method=True, **kw):
    cc = S.stem_cache_t.from_buffer_copy((c or cache())._obj)
    m = S.make_method("exp", rho_min=0.1, tau=4.0, k_min=2)
    for k in list(kw):
        if k.startswith("m_"):
            setattr(m, k[2:], kw.pop(k))
    KEEP.extend([cc, m])
    a = S.stem_decode_args_t()
    a.cache, a.method = ctypes.pointer(cc), ctypes.pointer(m) if method else None
    a.q = a.rows = a.lens = a.budget = a.sel_idx = a.sel_cnt = a.out = a.lse = a.workspace = FAKE
    a.R, a.Hq, a.kcap, a.dtype, a.workspace_bytes = 2, 8, 5, 0, 1 << 30
    for k, v in kw.items():
        setattr(a, k, v)
    return ctypes.byref(a)


out = {}
for name in ("stem_cache_append", "stem_cache_read"):
    f = getattr(L, name)
    out[name] = {
        "null cache": f(None, FAKE, FAKE, 0, 4, (ctypes.c_int64 * 3)(1, 1, 1), FAKE, None, None, None),
        "D": rows(f, cache(D=96)), "block": rows(f, cache(block=32)),
        "format": rows(f, cache(format=3)), "Hkv": rows(f, cache(Hkv=0)),
        "pages": rows(f, cache(num_pages=-1)), "nseq": rows(f, cache(nseq=-1)),
        "max_blocks": rows(f, cache(max_blocks=0)), "vsum": rows(f, cache(vsum=2)),
        "dtype": rows(f, dtype=2), "T": rows(f, T=-1), "T above the context": rows(f, T=16 * 128 + 1),
        "strides null": rows(f, strides=None), "stride negative": rows(f, strides=(2048, -128, 128)),
        "stride unaligned": rows(f, strides=(2048, 1024, 132)),
        "k null": rows(f, k=None), "v null": rows(f, v=None), "pos null": rows(f, pos=None),
        "k unaligned": rows(f, k=FAKE + 8), "pages null": rows(f, cache(pages=None)),
        "pages unaligned": rows(f, cache(pages=FAKE + 8)), "kbar null": rows(f, cache(kbar=None)),
        "table null": rows(f, cache(table=None)), "count unaligned": rows(f, count=FAKE + 2),
        "status unaligned": rows(f, status=FAKE + 1),
        "long context UNSUPPORTED": rows(f, cache(max_blocks=4097)),
        "many sequences UNSUPPORTED": rows(f, cache(nseq=65536)),
        "no sequences OK": rows(f, cache(nseq=0)), "no tokens OK": rows(f, T=0),
    }
for name in ("stem_decode_select", "stem_decode_attn", "stem_decode"):
    f = getattr(L, name)
    g = lambda *a, **k: f(args(*a, **k), None)
    r = out[name] = {
        "null": f(None, None), "null cache": g(cache=None), "null method": g(method=False),
        "D": g(cache(D=32)), "heads": g(Hq=7), "no heads": g(Hq=0), "R": g(R=-1), "kcap": g(kcap=0),
        "kcap above": g(kcap=17), "dtype": g(dtype=7), "share": g(m_share=2),
        "q null": g(q=None), "q unaligned": g(q=FAKE + 8), "lens null": g(lens=None),
        "sel_idx null": g(sel_idx=None), "sel_cnt null": g(sel_cnt=None),
        "rows unaligned": g(rows=FAKE + 2), "status unaligned": g(status=FAKE + 2),
        "more rows than sequences": g(rows=None, R=4), "no sequences": g(cache(nseq=0)),
        "pages null": g(cache(pages=None)),
        "f32 UNSUPPORTED": g(dtype=1), "many rows UNSUPPORTED": g(R=65536),
        "no rows OK": g(R=0),
    }
    if name != "stem_decode_attn":
        r.update({"budget null": g(budget=None), "metric": g(m_metric=3),
                  "beta": g(m_metric=1, m_beta=-1.0), "beta nan": g(m_metric=1, m_beta=float("nan")),
                  "clamp": g(m_metric=1, m_clamp=2), "score": g(m_score=2),
                  "score UNSUPPORTED": g(m_score=1)})
    if name != "stem_decode_select":
        r.update({"workspace null WORKSPACE": g(workspace=None),
                  "workspace small WORKSPACE": g(workspace_bytes=4096),
                  "workspace unaligned WORKSPACE": g(workspace=FAKE + 128),
                  "out null": g(out=None), "out unaligned": g(out=FAKE + 8),
                  "lse unaligned": g(lse=FAKE + 2)})
print(json.dumps(out))
"""


def test_refusals_come_before_any_device_work():
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="", PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, "-c", PROBE], env=env, capture_output=True, text=True,
                       timeout=300, cwd=ROOT)
    assert r.returncode == 0, r.stderr
    codes = {"OK": S.STEM_OK, "UNSUPPORTED": S.STEM_ERR_UNSUPPORTED,
             "WORKSPACE": S.STEM_ERR_WORKSPACE}
    for call, res in json.loads(r.stdout.strip().splitlines()[-1]).items():
        for case, got in res.items():
            assert got == codes.get(case.split()[-1], S.STEM_ERR_ARG), (call, case)


def test_rows_read_back_need_places_of_their_own():
    """A stride of 0 would give several rows one place; with one row along it there is no other."""
    code = PROBE.split("out = {}")[0] + """
read, cases = L.stem_cache_read, {}
for n in range(3):
    st = [2048, 1024, 128]
    st[n] = 0
    cases[n] = rows(read, strides=st)
    one = dict(c=cache(nseq=0) if n == 0 else cache(Hkv=1) if n == 1 else cache(), T=1 if n == 2 else 4)
    cases[f"one {n}"] = rows(read, strides=st, **one)
print(json.dumps(cases))
"""
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="", PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True,
                       timeout=300, cwd=ROOT)
    assert r.returncode == 0, r.stderr
    got = json.loads(r.stdout.strip().splitlines()[-1])
    for n in range(3):
        assert got[str(n)] == S.STEM_ERR_ARG, n
        assert got[f"one {n}"] != S.STEM_ERR_ARG, n


def test_sizes():
    for fmt in ("bf16", "q8", "q4"):
        for d in (64, 128):
            for block in (64, 128):
                assert D.stem_cache_page_bytes(d, block, fmt) == ref.page_bytes(fmt, d, block)
    assert D.stem_cache_page_bytes(128, 128, "q4") == 128 * 2 * (64 + 8)  # 4.5 bits a value
    assert D.stem_cache_page_bytes(96, 128, "q4") == 0 and D.stem_cache_page_bytes(64, 16, "q8") == 0
    c = S.stem_cache_t(None, None, None, None, 100, 8, 128, 128, S.STEM_KV_Q4, 3, 1024, 0)
    L = S.lib()
    n = L.stem_decode_workspace_size(ctypes.byref(c), 2, 32, 50)
    # the parts of an item (its CTAs' numerators), lists of 50 blocks a kv head or, per head, 200
    assert n > 2 * 8 * 200 * 8
    assert L.stem_decode_workspace_size(ctypes.byref(c), 4, 32, 50) > n
    assert L.stem_decode_workspace_size(ctypes.byref(c), 0, 32, 50) == 0
    assert L.stem_decode_workspace_size(ctypes.byref(c), 2, 33, 50) == 0
    assert L.stem_decode_workspace_size(ctypes.byref(c), 2, 32, 1025) == 0
    assert L.stem_decode_workspace_size(None, 2, 32, 50) == 0


@pytest.mark.parametrize("fmt", ["bf16", "q8", "q4"])
@pytest.mark.parametrize("d", [64, 128])
def test_reference_layout_is_a_bijection(fmt, d):
    """Every bit of a tile's code areas belongs to exactly one (token, channel) of K or V."""
    bits = np.concatenate([a.reshape(-1) for a in ref.bit_of(fmt, d)])
    width = ref.BITS[fmt]
    assert np.array_equal(np.sort(bits), np.arange(bits.size) * width)
    assert bits.size * width == 16 * d * 2 * width


def test_reference_rows_round_trip():
    g = torch.Generator().manual_seed(0)
    for fmt in ("bf16", "q8", "q4"):
        page = np.zeros(ref.page_bytes(fmt, 64, 64), dtype=np.uint8)
        k, v = (torch.randn(64, 64, generator=g).to(torch.bfloat16) for _ in range(2))
        for t in range(64):
            ref.put_row(page, fmt, 64, t, k[t], v[t])
        for got, x in zip(ref.get_rows(page, fmt, 64, range(64)), (k, v)):
            want = x.double() if fmt == "bf16" else ref.quantise(x, fmt)[2]
            assert torch.equal(got, want)
            if fmt != "bf16":  # half a step of the largest value, and the scale's rounding
                top = x.float().reshape(64, 2, 32).abs().amax(-1, keepdim=True).expand(-1, -1, 32)
                step = (top / ref.QMAX[fmt]).reshape(64, 64).double()
                assert torch.all((got - x.double()).abs() <= step * (0.5 + 2.0 ** -8 * 128))


def test_the_binding_refuses_host_tensors_and_wrong_shapes():
    table = torch.zeros(1, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        D.PagedCache.alloc(4, 2, 64, 64, "q4", table)
    with pytest.raises(ValueError, match="fmt"):
        D.PagedCache.alloc(4, 2, 64, 64, "q5", table)
    with pytest.raises(ValueError, match="64 or 128"):
        D.PagedCache.alloc(4, 2, 80, 64, "q4", table)
    with pytest.raises(ValueError, match="vsum"):
        D.PagedCache(table, torch.zeros(1, 1, 64), table, table, 64, "q4", vsum="sum")


def test_budget_of_a_method():
    m = S.make_method("exp", rho_min=0.1, tau=8.0, k_min=3)
    k, _ = S.stem_budget_m(100, m)
    budget, kcap = D.stem_decode_budget(100, m, "cpu")
    assert torch.equal(budget, k) and kcap == int(k.max())


def test_index_arithmetic_stays_inside_the_buffers(tmp_path):
    exe = str(tmp_path / "bounds")
    cmd = [libbuild._nvcc()] + libbuild.ARCH + ["-std=c++17", "-I", libbuild.INCLUDE, "-I",
                                                libbuild.CSRC, "-o", exe,
                                                os.path.join(ROOT, "tests", "decode_bounds.cu")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout
