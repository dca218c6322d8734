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


# ------------------------------------------------------------ a binding of another version --
def test_helpers_ask_whether_the_binding_is_current(monkeypatch):
    from gqa_attention_gb300 import _binding

    build.build()
    calls = []
    real = build.build_torch_binding
    monkeypatch.setattr(build, "build_torch_binding", lambda *a: (calls.append(a), real(*a))[1])
    monkeypatch.setattr(_binding, "_ext", None)
    _binding._torch_binding()
    _binding._torch_binding()
    assert len(calls) == 1


@pytest.mark.parametrize("stamp", [None, "3.9 1.0", "current"])
def test_binding_of_another_version_is_compiled_again(tmp_path, monkeypatch, stamp):
    import torch

    made = tmp_path / "_torch_binding.so"
    made.write_text("old")
    if stamp == "current":
        stamp = f"{sys.version} {torch.__version__}"
    if stamp is not None:
        (tmp_path / "torch_binding.stamp").write_text(stamp)
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "TORCH_BINDING", str(made))

    def compiler(cmd, **kw):
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("new")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build.subprocess, "run", compiler)
    build.build_torch_binding()
    current = stamp == f"{sys.version} {torch.__version__}"
    assert made.read_text() == ("old" if current else "new")
    made.write_text("again")
    build.build_torch_binding()
    assert made.read_text() == "again"
