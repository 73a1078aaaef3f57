"""The decoder layer example end to end: norm, rotated append, attention, routing, experts and back, prompts and then
tokens from a captured, padded graph, each step's stages and the gradients against 64 bits."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("mode", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("shape", [[], ["--heads", "16", "--kv-heads", "16", "--head-dim", "64", "--rotary", "32", "--page", "16",
                                        "--experts", "60", "--top-k", "6", "--pad", "0"]])
def test_example(mode, shape):
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "decoder_layer.py"), "--check", "--mode", mode, "--hidden", "512",
                        "--expert-dim", "192", "--experts", "8", "--steps", "12", "--prompts", "130", "1", "64", "300", *shape],
                       capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr
