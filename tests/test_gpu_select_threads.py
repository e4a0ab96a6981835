"""Selection calls of two host threads on a B200: the shared-memory limit of a kernel belongs to all
threads, and what one sets for its launch must not refuse another's."""

import os
import subprocess

import pytest

from block_sparse_causal_pooling_b200 import build as libbuild
from block_sparse_causal_pooling_b200 import stem as S

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def test_group_selection_of_two_sizes_from_two_threads(tmp_path):
    exe, lib = str(tmp_path / "threads"), os.path.dirname(S.LIB_PATH)
    cmd = [libbuild._nvcc()] + libbuild.ARCH + ["-std=c++17", "-I", libbuild.INCLUDE, "-o", exe,
                                                os.path.join(HERE, "select_threads.cu"), "-L", lib,
                                                "-l:libstem.so", "-Xlinker", "-rpath", "-Xlinker", lib]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout
