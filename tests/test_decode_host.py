"""The host side of the decode path on the CPU: budgets, argument checks and the build of the binding."""

import ctypes
import json
import os
import subprocess
import sys

import pytest
import torch

from block_sparse_causal_pooling_b200 import build as libbuild
from block_sparse_causal_pooling_b200 import decode as D
from block_sparse_causal_pooling_b200 import stem as S
from tests import test_decode_abi as abi


def abi_probe(code):
    """What `code` prints (JSON) after the helpers of test_decode_abi.PROBE, in a process without a GPU."""
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="", PYTHONPATH=abi.ROOT)
    r = subprocess.run([sys.executable, "-c", abi.PROBE.split("out = {}")[0] + code], env=env,
                       capture_output=True, text=True, timeout=300, cwd=abi.ROOT)
    assert r.returncode == 0, r.stderr
    return json.loads(r.stdout.strip().splitlines()[-1])


@pytest.mark.parametrize("k_start,mu,k_min", [(20.0, 0.25, 2), (7.5, 0.9, 3), (300.0, 1.0, 1),
                                              (1.0, 0.01, 1)])
def test_the_linear_schedule_is_that_of_a_context_which_ends_here(k_start, mu, k_min):
    """A token in block i is in the last of i + 1 blocks, whatever the width of the table."""
    m = S.make_method("linear", k_start=k_start, mu=mu, k_min=k_min)
    for width in (1, 2, 3, 50, 400):
        budget, kcap = D.stem_decode_budget(width, m, "cpu")
        want = [int(S.stem_budget_m(i + 1, m)[0][i]) for i in range(width)]
        assert budget.tolist() == want and budget.dtype == torch.int32
        assert kcap == max(want)


def test_the_stride_of_an_axis_of_one_row_is_not_looked_at():
    """It may be anything: unaligned, negative, 0; along an axis of several rows it is refused."""
    got = abi_probe("""
cases = {}
for name in ("stem_cache_append", "stem_cache_read"):
    for n in range(3):
        for bad in (132, -128, 3):
            st = [2048, 1024, 128]
            st[n] = bad
            one = dict(c=cache(nseq=1) if n == 0 else cache(Hkv=1) if n == 1 else cache(),
                       T=1 if n == 2 else 4)
            cases[f"{name} {n} {bad}"] = [rows(getattr(L, name), strides=st),
                                          rows(getattr(L, name), strides=st, **one)]
print(json.dumps(cases))
""")
    assert len(got) == 18
    for case, (several, one) in got.items():
        assert several == S.STEM_ERR_ARG and one != S.STEM_ERR_ARG, case


def test_method_parameters_are_of_their_type():
    """Their memory is read by address: nothing else may stand in for them, above all nothing smaller."""
    for method in (ctypes.c_int32(0), S.stem_cache_t(), None, "exp", 0):
        for call in (D.stem_decode_select, D.stem_decode):
            with pytest.raises(TypeError, match="stem_method_t"):
                call(None, None, None, None, 1, method)


def test_the_binding_is_built_again_for_another_torch_python_or_command(monkeypatch, tmp_path):
    ran = []

    def gxx(cmd, **kw):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    for name, at in (("BIND", "_decode.so"), ("STAMP", "stamp"), ("BUILD", "build")):
        monkeypatch.setattr(libbuild, name, str(tmp_path / at))
    monkeypatch.setattr(libbuild.subprocess, "run", gxx)

    def builds():
        n = len(ran)
        libbuild._build_binding(False)
        return len(ran) - n

    assert builds() == 1 and os.path.exists(libbuild.BIND)
    assert builds() == 0
    os.remove(libbuild.STAMP)
    assert builds() == 1 and builds() == 0
    for change in ((torch, "__version__", "0.0"), (sys, "version", "0.0"),
                   (libbuild, "INCLUDE", libbuild.INCLUDE + "/")):
        monkeypatch.setattr(*change)
        assert builds() == 1 and builds() == 0, change[1]
    monkeypatch.setattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", not torch._C._GLIBCXX_USE_CXX11_ABI)
    assert builds() == 1 and builds() == 0


def test_rows_read_back_may_not_overlap():
    got = abi_probe("""
read, append = L.stem_cache_read, L.stem_cache_append
c = lambda **kw: cache(nseq=3, Hkv=2, D=64, **kw)
cases = {}
# T = 4 rows of 64, element strides of (sequence, head, token)
for ok, st in ((1, (512, 256, 64)), (1, (512, 64, 128)), (1, (64, 1024, 192)), (1, (4096, 2048, 72)),
               (0, (512, 256, 56)), (0, (512, 248, 64)), (0, (504, 256, 64)), (0, (512, 64, 64)),
               (0, (64, 64, 64)), (0, (128, 256, 64)), (0, (512, 256, 8)), (0, (0, 256, 64)),
               (0, (1 << 62, 256, 64)), (1, (1 << 40, 256, 64))):
    cases[f"{ok} {st}"] = [rows(read, c(), strides=st), rows(append, c(), strides=st)]
print(json.dumps(cases))
""")
    for case, (read, append) in got.items():
        assert (read == S.STEM_ERR_ARG) == (case[0] == "0"), case
        assert append != S.STEM_ERR_ARG, case  # (rows that are read may)
