"""How the attention kernels deal key tiles out to the CTAs, on the CPU: the header that the kernels compile is compiled for
the host and run over drawn lists of items (tests/kv_split_check.cpp)."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_every_tile_is_dealt_once_and_the_ctas_agree_on_the_pieces(tmp_path):
    exe = tmp_path / "kv_split_check"
    subprocess.check_call(["g++", "-std=c++17", "-O2", "-o", str(exe), os.path.join(HERE, "kv_split_check.cpp")])
    out = subprocess.run([str(exe), "4000"], capture_output=True, text=True, timeout=600)
    assert out.returncode == 0, out.stdout + out.stderr
    assert out.stdout.strip().endswith(", 0 failures"), out.stdout
