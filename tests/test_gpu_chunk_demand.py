"""Demand of a chunk's tokens: those that were served count, and no others. A padded batch, captured; a refused lane."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("resident_expert_routed_gb300")


def picks(layer, rows):
    """The demand that these rows of the last call add up to, by expert, in units of 2^-40 (fp32 scores are exact in 64 bits)."""
    e, s = layer.buf.want_e[rows].cpu().numpy(), layer.buf.want_s[rows].cpu().numpy()
    got = np.zeros(layer.moe_args[4].shape[1], np.int64)
    np.add.at(got, e.ravel(), np.rint(s.astype(np.float64) * 2.0 ** 40).astype(np.int64).ravel())
    return got


def test_a_captured_batch_of_one_size_counts_its_tokens_alone():
    """64 rows of hidden states whatever the lanes get; the rest holds something large. Each replay adds its tokens' demand."""
    from examples.tree_decode import build
    from resident_expert_routed_gb300.decode import DevicePages
    T = 64
    layer, pages = build(3, T, 40), DevicePages(3, 40, 16, 12, T)
    demand, miss = layer.moe_args[4], layer.moe_args[5]
    n_new = torch.zeros(3, dtype=torch.int32, device="cuda")
    hidden = torch.zeros((T, 256), dtype=torch.bfloat16, device="cuda")

    def body():
        pages.plan(n_new)
        out = layer.chunk(hidden, pages)
        pages.advance()
        return out

    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        body()                                                 # every lane waits
    side.synchronize()
    assert demand.sum().item() == 0 and (miss == 0).all()
    with torch.cuda.graph(graph, stream=side):
        out = body()
    gen = torch.Generator(device="cuda").manual_seed(5)
    for new in ([20, 7, 0], [1, 1, 30], [0, 0, 0], [40, 0, 24], [1, 1, 1]):
        n = sum(new)
        hidden.copy_(torch.randn((T, 256), generator=gen, device="cuda"))
        hidden[n:] = 3e4
        n_new.copy_(torch.tensor(new, dtype=torch.int32))
        demand.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert moe.moe_device_status() == (moe.MOE_OK, 0)
        assert np.array_equal(demand[0].cpu().numpy(), picks(layer, slice(0, n))), new
        assert torch.isfinite(out[:n]).all()
    assert pages.rows.tolist() == [62, 9, 55]


def test_a_refused_lanes_tokens_are_no_demand():
    from examples.tree_decode import build
    from resident_expert_routed_gb300.decode import DevicePages
    layer, pages = build(3, 80, 4), DevicePages(3, 4, 16, 8, 80)
    pages.plan(torch.tensor([30, 40, 10], dtype=torch.int32, device="cuda"))       # 2, 3 and 1 pages of 4: the second and third are refused
    layer.chunk(torch.randn(80, 256, device="cuda").bfloat16(), pages)
    assert np.array_equal(layer.moe_args[4][0].cpu().numpy(), picks(layer, slice(0, 30)))
    assert moe.moe_device_status()[1] & moe.MOE_DEV_NO_PAGES


def test_a_batch_larger_than_its_places_is_refused_before_anything_is_written():
    from examples.tree_decode import build
    from resident_expert_routed_gb300.decode import DevicePages
    hidden = torch.randn(65, 256, device="cuda").bfloat16()
    for tokens, planned in ((64, 80), (80, 64)):
        layer, pages = build(1, tokens, 8), DevicePages(1, 8, 16, 8, planned)
        pages.plan(torch.tensor([60], dtype=torch.int32, device="cuda"))
        with pytest.raises(ValueError):
            layer.chunk(hidden, pages)
        assert (layer.cache.k_codes == 0).all() and (layer.moe_args[4] == 0).all()
