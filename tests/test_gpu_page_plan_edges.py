"""Plans at the edges of their workspace."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("resident_expert_routed_gb300")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_lane_counts_around_what_shared_memory_holds_without_asking():
    """20 bytes a lane and 512 more: the 48 KB that need no opt-in end between 2,432 and 2,433 lanes. In a process of its own, as
    the opt-in of a larger call would stay."""
    code = """
import numpy as np
from tests.test_gpu_page_plan import State
for lanes in (2431, 2432, 2433, 2457, 2458, 4096):
    s = State(lanes, 3, 3 * lanes, 16, seed=lanes, most=2)
    new = s.rng.randint(-1, 12, lanes)
    s.check(new, int(np.maximum(new, 0).sum()) + 1)
print("planned")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env=dict(os.environ, PYTHONPATH=ROOT), capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "planned" in r.stdout, r.stdout + r.stderr
