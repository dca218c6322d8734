"""The block arithmetic of the block-scaled cache's append (csrc/kv_blocks.h), which the kernel
and its launcher share, compiled for the host with overflow checks."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_blocks_of_an_append_up_to_the_largest_sizes(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("no g++")
    exe = tmp_path / "append_blocks"
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror",
                           "-fsanitize=signed-integer-overflow", "-fno-sanitize-recover=all",
                           "-I", os.path.join(ROOT, "gqa_attention_gb300", "csrc"),
                           os.path.join(ROOT, "tests", "c", "append_blocks.cpp"), "-o", str(exe)])
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, out.stdout + out.stderr
    assert "append_blocks: ok" in out.stdout
