"""Which steps of positions need masks, on the CPU under sanitizers
(tests/cache_window_check.cpp)."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "lossless_tensor_compression_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_hidden_positions(tmp_path):
    exe = str(tmp_path / "cache_window_check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-Wall", "-Wextra", "-fsanitize=undefined", "-fno-sanitize-recover=all",
                    "-I", CSRC, os.path.join(HERE, "cache_window_check.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=100)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout
