"""The cache example end to end: prompts, then tokens from a captured graph, each step against 64 bits."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("mode", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("shape", [[], ["--heads", "16", "--kv-heads", "16", "--head-dim", "64", "--page", "16"]])
def test_example(mode, shape):
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "kv_decode.py"), "--check", "--mode", mode,
                        "--hidden", "512", "--steps", "20", "--prompts", "130", "1", "64", "300", *shape],
                       capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr
