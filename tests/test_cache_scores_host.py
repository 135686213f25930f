"""The room for written scores, without a GPU: what the rows of a call can see,
not what their tables could hold."""
import ctypes
import os
import shutil
import subprocess

import pytest

from test_cache_host import _lib, cache, seqs

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "lossless_tensor_compression_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_steps_lie_within_the_room(tmp_path):
    exe = str(tmp_path / "cache_scores_check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-Wall", "-Wextra", "-I", CSRC, os.path.join(HERE, "cache_scores_check.cpp"),
                    "-o", exe], check=True)
    r = subprocess.run([exe], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=100)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout


@pytest.mark.parametrize("codes", [0, 1, 3])
def test_a_window_bounds_the_workspace(codes):
    """40 single rows of 32 query heads, tables of 128k positions: with a window of
    1,024 a row's scores are 1,216 numbers, and they are written."""
    L, c = _lib(), cache(codes=codes, heads=8, dim=128, page=64)
    s = seqs(cu=0, n=40, rows=40, width=2048, stride=2048)
    more = [L.ltc_cache_attend_weigh_workspace_size(ctypes.byref(c), s, 32, w) - L.ltc_cache_attend_workspace_size(ctypes.byref(c), s, 32, w)
            for w in (0, 1024, 1 << 20)]
    assert 40 * 32 * 4 <= more[0] < 2 * 40 * 32 * 4      # too many to write down: the sums alone
    assert 40 * 32 * 4 * (1 + 1024 + 40) <= more[1] <= 40 * 32 * 4 * (1 + 1024 + 40 + 192) + 512
    assert more[2] == more[0]
