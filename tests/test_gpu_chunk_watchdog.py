"""A chunk attention whose waits run out: the kernel ends, the status says so, and the next call is correct."""
import pytest
import torch

from tests.test_gpu_chunk_attention import Chunks

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("resident_expert_routed_gb300")


@pytest.mark.parametrize("lanes,Hq,D", [([(60000, 4)], 8, 128), ([(0, 700)], 4, 64), ([(9000, 5), (3000, 70), (0, 1)], 4, 256),
                                        ([(20000, 160), (50, 2)], 16, 128), ([(8000, 16)] * 3, 8, 64)])
def test_a_bound_below_any_tile_stops_the_kernel(lanes, Hq, D):
    """A bound of 1 ns: between two looks nothing has moved, as a block's first tile takes microseconds."""
    c = Chunks(lanes, Hq, 2, D, 64, seed=D)
    cache, table, kv_len, cu, out, lse, ws = c.args()
    call = lambda: moe.moe_chunk_attention(c.q, cache, table, kv_len, cu, c.scale, out, ws, lse=lse)  # noqa: E731
    call()
    want = out.clone()
    assert moe.moe_device_status() == (moe.MOE_OK, 0)
    before = moe.moe_get_wait_limit()
    for _ in range(5):
        moe.moe_set_wait_limit(1)
        try:
            call()
            status = moe.moe_device_status()
        finally:
            moe.moe_set_wait_limit(before)
        assert status == (moe.MOE_ETIMEOUT, moe.MOE_DEV_TIMEOUT)
        out.fill_(9.0)
        call()
        assert moe.moe_device_status() == (moe.MOE_OK, 0)
        assert torch.equal(out, want)
