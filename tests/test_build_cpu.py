"""What building needs: the C library stands without PyTorch, without a working binding, and a
variant of it leaves the package's binding alone."""
import os
import subprocess
import sys

import pytest

from gqa_attention_gb300 import build

SOURCE = """#include <cuda_runtime.h>
__global__ void k(int* p) { *p = 1; }
extern "C" int answer() { return 42; }
"""


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A package of one small source in a folder of its own."""
    (tmp_path / "csrc").mkdir()
    (tmp_path / "csrc" / "one.cu").write_text(SOURCE)
    monkeypatch.setattr(build, "CSRC", str(tmp_path / "csrc"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib.so"))
    return dict(lib_path=str(tmp_path / "lib.so"), build_dir=str(tmp_path / "obj"))


def test_library_without_torch(tree, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch fails, as where there is none
    assert os.path.exists(build.build(**tree))


def test_library_where_the_binding_fails(tree, monkeypatch, capsys):
    def fails(force=False):
        raise RuntimeError("no compiler for it")

    monkeypatch.setattr(build, "build_torch_binding", fails)
    assert os.path.exists(build.build(**tree))
    assert "no compiler for it" in capsys.readouterr().err


def test_a_variant_leaves_the_binding_alone(tree, tmp_path, monkeypatch):
    calls = []
    monkeypatch.setattr(build, "build_torch_binding", lambda force=False: calls.append(force))
    build.build(lib_path=str(tmp_path / "variant.so"), build_dir=str(tmp_path / "obj2"))
    assert calls == []
    build.build(**tree)
    assert calls == [False]


def test_a_failing_source_still_raises(tree, tmp_path):
    (tmp_path / "csrc" / "two.cu").write_text("#error no\n")
    with pytest.raises(RuntimeError):
        build.build(**tree)
    assert not os.path.exists(tree["lib_path"])


def test_module_builds_as_a_program():
    r = subprocess.run([sys.executable, "-m", "gqa_attention_gb300.build"], capture_output=True, text=True,
                       cwd=build.ROOT)
    assert r.returncode == 0 and r.stdout.strip().endswith("libgqa_attn.so"), r.stderr
