"""Plans at the edges of their workspace, and states that cannot be served."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from tests.test_gpu_page_plan import State

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


def planned(s, new, T):
    """(outputs and state as lists, status) of a call."""
    got = s.gpu(new, T)
    bits = moe.moe_device_status()[1]
    return {k: v.cpu().numpy() for k, v in got.items()}, bits, got


@pytest.mark.parametrize("n,held", [(5, True), (48, False), (3000, True), (3000, False)])
def test_a_page_id_outside_the_pool_refuses_its_lane(n, held):
    """In the lane's table, or on the stack when the lane takes it; few tokens and so many that several blocks plan them. The lane
    gets kv_len 0 and no slots at all, though its other pages are good; the lanes around it are served."""
    page, T = 16, 4 * n + 9
    width = (20 + n) // page + 2
    s = State(4, width, 4 * width + 4, page, seed=n, most=0)
    ids = s.rng.permutation(4 * width + 4).astype(np.int32)
    s.held[:], s.rows[:] = 2, 20                               # the second page is half full
    s.table[:, :2] = ids[:8].reshape(4, 2)
    s.free[:], s.n_free = -7, 4 * width - 4
    s.free[:s.n_free] = ids[8:8 + s.n_free]
    need = -(-(20 + n) // page) - 2
    if held:
        s.table[1, 1] = 4 * width + 4                          # the first id past the pool
    else:
        s.free[s.n_free - 1 - need - need // 2] = -2           # one that lane 1 takes
    want, bits, got = planned(s, [n] * 4, T)
    assert bits == moe.MOE_DEV_BAD_PAGE
    assert want["kv_len"].tolist() == [20 + n, 0, 20 + n, 20 + n] and want["rows"].tolist() == [20] * 4
    assert want["cu"].tolist() == [n * i for i in range(5)]
    slots = want["slots"]
    assert (slots[n:2 * n] == -1).all() and (slots[4 * n:] == -1).all()
    for b in (0, 2, 3):
        at = 20 + np.arange(n)
        assert np.array_equal(slots[b * n:(b + 1) * n], want["table"][b, at // page].astype(np.int64) * page + at % page)
        assert np.array_equal(want["positions"][b * n:(b + 1) * n], at)
    # the pages that it took stay with it: again the same answer, and each page is in one place
    assert want["held"].tolist() == [2 + need] * 4 and want["n_free"].tolist() == [s.n_free - 4 * need]
    s.call(got)
    torch.cuda.synchronize()
    assert moe.moe_device_status()[1] == moe.MOE_DEV_BAD_PAGE
    for name in ("rows", "held", "table", "n_free", "kv_len", "cu", "positions", "slots"):
        assert np.array_equal(got[name].cpu().numpy(), want[name]), name


def test_rows_of_a_lane_refused_for_its_pages_do_not_move_on():
    from resident_expert_routed_gb300.decode import DevicePages
    pages = DevicePages(3, 12, 16, 4, 64)
    new = torch.tensor([10, 10, 10], dtype=torch.int32, device="cuda")
    pages.plan(new)
    pages.advance()
    pages.table[1, 0] = 12
    pages.plan(new)
    assert moe.moe_device_status()[1] == moe.MOE_DEV_BAD_PAGE
    pages.advance()
    assert pages.rows.tolist() == [20, 10, 20] and pages.kv_len.tolist() == [20, 0, 20]


def test_a_waiting_lane_whose_state_is_bad_is_refused_too():
    """Pages outside the table, or negative rows: kv_len 0, as for a lane that gets tokens. A waiting lane behind tokens that do not
    fit the batch is not refused: it has none."""
    for rows, held in ((20, 9), (20, -1), (-4, 2)):
        s = State(3, 4, 20, 16, seed=2, most=2)
        s.rows[:], s.held[:] = 20, 2
        s.table[:, :2] = np.arange(6).reshape(3, 2)
        s.free[:14], s.n_free = np.arange(6, 20), 14
        s.rows[1], s.held[1] = rows, held
        want, bits, _ = planned(s, [3, 0, 0], 8)
        assert bits == moe.MOE_DEV_BAD_PAGE and want["kv_len"].tolist() == [23, 0, 20], (rows, held)
        assert want["rows"][1] == rows and want["held"][1] == held
    s.rows[:], s.held[:] = 20, 2
    want, bits, _ = planned(s, [3, 30, 0], 8)
    assert bits == moe.MOE_DEV_NO_PAGES and want["kv_len"].tolist() == [23, 0, 20]
