"""Lanes that a plan refused, at the attention and at the layer."""
import pytest
import torch

from tests.test_gpu_chunk_attention import Chunks

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("resident_expert_routed_gb300")


def test_a_lane_that_the_plan_refused_gets_zeros_and_is_no_bad_page():
    """kv_len 0 with tokens, as moe_page_plan gives it: the status stays clean, which tells a pool that ran out from a table that is wrong."""
    c = Chunks([(100, 50), (20, 30), (60, 10), (7, 1)], 4, 2, 64, 16, seed=17)
    want = c.gpu()
    for refused in ([1], [0, 3], [0, 1, 2, 3]):
        lens = c.kv_len.copy()
        c.kv_len[refused] = 0
        out, lse = c.gpu()
        assert moe.moe_device_status() == (moe.MOE_OK, 0)
        for b in range(4):
            rows = slice(c.cu[b], c.cu[b + 1])
            if b in refused:
                assert (out[rows] == 0).all() and torch.isneginf(lse[rows]).all()
            else:
                assert torch.equal(out[rows], want[0][rows]) and torch.equal(lse[rows], want[1][rows])
        c.kv_len = lens
    c.kv_len[1] = 29                                           # some rows, but not the tokens': that is an error
    c.gpu()
    assert moe.moe_device_status() == (moe.MOE_EDEVICE, moe.MOE_DEV_BAD_PAGE)


def test_a_layer_without_pages_says_so_and_nothing_else():
    from examples.tree_decode import build
    from resident_expert_routed_gb300.decode import DevicePages
    layer, pages = build(2, 64, 3), DevicePages(2, 3, 16, 8, 64)
    pages.plan(torch.tensor([40, 20], dtype=torch.int32, device="cuda"))
    layer.chunk(torch.randn(60, 256, device="cuda").bfloat16(), pages)
    assert moe.moe_device_status() == (moe.MOE_EDEVICE, moe.MOE_DEV_NO_PAGES)
    assert (layer.out[40:60] == 0).all()
