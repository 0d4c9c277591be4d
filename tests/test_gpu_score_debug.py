"""The debug build on the attention over 8-bit caches and with capped or biased scores: its checks of tiles and partial
slots, and dead ring rows and unfilled blocks refilled after every commit (test_gpu_debug.py says how)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CASES = ["tests/test_gpu_q8.py", "tests/test_gpu_scores.py", "tests/test_gpu_rope.py", "tests/test_gpu_score_edges.py"]


def test_debug_build_passes_the_score_cases(cuda_device):
    from self_speculative_decode_b200 import build
    env = dict(os.environ, RIPE_LIBRARY=build.build(debug=True))
    probe = subprocess.run([sys.executable, "-c", "from self_speculative_decode_b200 import ripe; "
                            "print(ripe.ripe_build_info())"], env=env, cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert probe.returncode == 0 and probe.stdout.strip() == "1", probe.stderr[-2000:]
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", *CASES],
                       env=env, cwd=ROOT, capture_output=True, text=True, timeout=1800)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
