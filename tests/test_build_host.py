"""Building, on CPU: what the C library needs, and what the binding's fast path does."""
import os
import subprocess
import sys

import pytest

from bit_quantized_moe_gemv_b200 import build

PROGRAM = """
import importlib.abc, os, sys
class Refuse(importlib.abc.MetaPathFinder):
    def find_spec(self, name, path=None, target=None):
        if name.split(".")[0] == "torch":
            raise ModuleNotFoundError("No module named 'torch'", name="torch")
sys.meta_path.insert(0, Refuse())
from bit_quantized_moe_gemv_b200 import build
build.OBJ_DIR, build.LIB, build.NATIVE = (os.path.join(sys.argv[1], n) for n in ("obj", "lib.so", "_native.so"))
build.sources = lambda: [os.path.join(build.CSRC, "abi.cu")]
for force in (True, False):
    assert build.build(force=force) == build.LIB and os.path.exists(build.LIB)
    assert not os.path.exists(build.NATIVE)
"""


def test_the_library_builds_without_torch(tmp_path):
    """A user of the C calls has no need of it (one source stands for all)."""
    r = subprocess.run([sys.executable, "-c", PROGRAM, str(tmp_path)], capture_output=True, text=True, cwd=build.ROOT)
    assert r.returncode == 0, r.stderr


def test_the_fast_path_is_built_again_for_another_torch(tmp_path, monkeypatch):
    """It is compiled against torch's and Python's headers, and good for no others."""
    pytest.importorskip("torch")
    monkeypatch.setattr(build, "NATIVE", str(tmp_path / "_native.so"))
    assert build.build_native() == build.NATIVE
    os.utime(build.NATIVE, (2_000_000_000, 2_000_000_000))  # newer than any source
    first = os.stat(build.NATIVE).st_mtime_ns
    build.build_native()
    assert os.stat(build.NATIVE).st_mtime_ns == first
    import importlib.metadata as md
    monkeypatch.setattr(md, "version", lambda name: "0.0.1")
    build.build_native()
    assert os.stat(build.NATIVE).st_mtime_ns != first
