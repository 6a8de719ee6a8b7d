"""The library builds, and host-only calls run, where torch, its headers or a
C++ compiler for the binding's module are missing."""
import importlib.util
import os
import shutil
import subprocess
import sys

import numpy as np
import pytest

import paged_prefix_shared_decode_gb300 as kvp
from paged_prefix_shared_decode_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def small_build(tmp_path, monkeypatch):
    """build() of a library of one unit, in a folder of its own."""
    if not shutil.which(build._nvcc()):
        pytest.skip("no nvcc")
    for name, path in (("OUT_DIR", "out"), ("LIB", "libkvp.so"), ("CALLS", "_calls.so")):
        monkeypatch.setattr(build, name, str(tmp_path / path))
    monkeypatch.setattr(build, "SOURCES", ["radix.cpp"])
    (tmp_path / "_calls.so").write_text("an old one")
    return tmp_path


def test_without_torch(small_build, monkeypatch):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    with pytest.warns(UserWarning, match="_calls.so is not built: No module named 'torch'"):
        build.build()
    assert (small_build / "libkvp.so").exists()


@pytest.mark.parametrize("cxx", ["false", "no-such-compiler"])
def test_without_a_compiler(small_build, monkeypatch, cxx):
    pytest.importorskip("torch")
    monkeypatch.setenv("CXX", cxx)
    with pytest.warns(UserWarning, match="_calls.so is not built"):
        build.build()
    assert (small_build / "libkvp.so").exists() and not (small_build / "_calls.so").exists()


def test_a_library_that_does_not_compile_is_an_error(small_build, monkeypatch):
    monkeypatch.setenv("NVCC", "/bin/false")
    monkeypatch.setattr(build, "_calls_job", lambda *a: None)
    with pytest.raises(RuntimeError, match="compile failed"):
        build.build()


RUN = """
import sys
sys.modules["torch"] = None                 # importing it raises
import numpy as np
import paged_prefix_shared_decode_gb300 as kvp
p = kvp.kv_pool_create(kvp.PoolDesc(1, 64, 16, 2, 64, 8, 8, 3))
for i in range(4):
    kvp.seq_reserve(p, kvp.seq_alloc(p), 20 + i)
kvp.seq_reorder(p, [0, 1, 2], np.array([3, 3, 0]))
kvp.seq_reorder(p, [], [])
assert [kvp.seq_len(p, i) for i in range(4)] == [23, 23, 20, 23]
for dst, src, error in (([0], [1, 2], ValueError), ([1 << 40], [0], ValueError), ([0.5], [0], TypeError),
                        (None, [0], TypeError), (np.zeros((1, 1), np.int32), [0], ValueError), ([0, 0], [1, 2], kvp.KvpError)):
    try:
        kvp.seq_reorder(p, dst, src)
    except error:
        continue
    raise SystemExit((dst, src))
assert [kvp.seq_len(p, i) for i in range(4)] == [23, 23, 20, 23]
try:
    kvp.kvp_page_bounds(0, 0, 0, 1, kvp.AttnDesc(), 0, 0)
except ImportError:
    print("done")
"""


def test_host_calls_without_torch():
    r = subprocess.run([sys.executable, "-c", RUN], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout == "done\n", r.stderr


def test_reorder_without_the_module(monkeypatch):
    def missing():
        raise RuntimeError("_calls.so is not built")
    monkeypatch.setattr(kvp, "_native", missing)
    p = kvp.kv_pool_create(kvp.PoolDesc(1, 64, 16, 2, 64, 8, 8, 3))
    for i in range(3):
        kvp.seq_reserve(p, kvp.seq_alloc(p), 20 + i)
    kvp.seq_reorder(p, np.array([0, 1], np.int64), (2, 0))
    assert [kvp.seq_len(p, i) for i in range(3)] == [22, 20, 22]
    kvp.kv_pool_destroy(p)
