"""A tree attention whose waits run out: the kernel ends, the status says so, and the next call is correct."""
import numpy as np
import pytest
import torch

from tests.test_gpu_tree_attention import Case

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("resident_expert_routed_gb300")


@pytest.mark.parametrize("lanes,Hq,D", [([(60000, 4)], 8, 128), ([(700, 1)], 4, 64), ([(9000, 5), (3000, 7), (0, 1)], 4, 256),
                                        ([(20000, 16), (50, 2)], 16, 128), ([(8000, 16)] * 3, 8, 64)])
def test_a_bound_below_any_tile_stops_the_kernel(lanes, Hq, D):
    """A bound of 1 ns: between two looks of the watchdog nothing has moved, as a block's first tile takes microseconds."""
    c = Case(lanes, Hq, 2, D, 64, seed=D)
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    kc, ks, vc, vs = (dev(a) for a in c.pool)
    args = (c.q, moe.KvCache(kc, vc, ks, vs), dev(c.table), dev(c.kv_len), dev(c.cu), c.max_nodes, dev(c.mask.view(np.int32)), c.scale)
    out = torch.empty((c.N, Hq, D), dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(moe.moe_tree_attention_workspace_bytes(c.N, Hq, 2, D, len(lanes)), dtype=torch.uint8, device="cuda")
    moe.moe_tree_attention(*args, out, ws)
    want = out.clone()
    assert moe.moe_device_status() == (moe.MOE_OK, 0)
    before = moe.moe_get_wait_limit()
    for _ in range(5):
        moe.moe_set_wait_limit(1)
        try:
            moe.moe_tree_attention(*args, out, ws)
            status = moe.moe_device_status()
        finally:
            moe.moe_set_wait_limit(before)
        assert status == (moe.MOE_ETIMEOUT, moe.MOE_DEV_TIMEOUT)
        out.fill_(9.0)
        moe.moe_tree_attention(*args, out, ws)
        assert moe.moe_device_status() == (moe.MOE_OK, 0)
        assert torch.equal(out, want)
