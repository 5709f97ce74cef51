"""The feed-forward example trains and serves (one process, as a user runs it)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
@pytest.mark.parametrize("args", [[], ["--width", "200", "--hidden", "333", "--outputs", "65",
                                       "--tokens", "301", "--steps", "20"]])
def test_example_trains_and_serves(args):
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "feed_forward_block.py"), *args],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-1000:] + r.stderr[-2000:]
    assert "loss" in r.stdout
