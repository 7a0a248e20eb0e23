"""The cache, the attention and the expert layer together, as a decode loop uses them; and how the attention's kernel
ends when its waits run out, beside other work and again and again."""
import numpy as np
import pytest
import torch

from tests import kv_reference as ref
from tests.test_gpu_tree_attention import Case

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("resident_expert_routed_gb300")


def test_example_keeps_what_it_accepted():
    from examples import tree_decode
    layer, pages, k, v = tree_decode.main(steps=6, lanes=3, seed=3)
    again, pages2, k2, v2 = tree_decode.main(steps=6, lanes=3, seed=3)
    assert pages.rows == pages2.rows and sum(pages.rows) > 66
    assert torch.equal(k, k2) and torch.equal(v, v2)
    assert torch.isfinite(k).all() and torch.isfinite(v).all() and not (k == 0).all(-1).any()


def test_a_drafted_path_gives_what_single_tokens_give():
    """A path of a tree, checked at once, against the same tokens one by one: the same hidden states and cache, up to
    the roundings of the products' batch sizes and the probabilities (bf16 outputs of order 1: 2^-6)."""
    from examples.tree_decode import build
    from resident_expert_routed_gb300.decode import LanePages, Step
    torch.manual_seed(0)
    parents, path = [-1, 0, 0, 1, 2, 4, 3, 5], [0, 2, 4, 5, 7]
    prompt = torch.randn(40, 256, device="cuda").bfloat16()
    drafted = torch.randn(8, 256, device="cuda").bfloat16()
    outs, caches = [], []
    for tree in (True, False):
        layer, pages = build(1, 64, 8), LanePages(1, 8, 16, 8)
        layer.step(prompt, Step(pages, [list(range(-1, 39))]), tree=False)
        pages.advance(0, 40)
        if tree:
            t = Step(pages, [parents])
            outs.append(layer.step(drafted, t)[path].float())
            layer.keep(t, torch.tensor([path], dtype=torch.int32, device="cuda"), torch.tensor([5], dtype=torch.int32, device="cuda"))
            pages.advance(0, 5)
        else:
            got = []
            for i in path:
                got.append(layer.step(drafted[i:i + 1], Step(pages, [[-1]])).float())
                pages.advance(0, 1)
            outs.append(torch.cat(got))
        k, v = (torch.empty((45, 2, 64), device="cuda") for _ in range(2))
        moe.moe_kv_read(layer.cache, pages.table.cuda(), None, torch.tensor([0, 45], dtype=torch.int32, device="cuda"), k, v)
        caches.append((k, v))
    assert moe.moe_device_status() == (moe.MOE_OK, 0)
    # one e4m3 step where a product's rounding falls on the other side
    for a, b in zip(*caches):
        assert ((a - b).abs() <= 2.0 ** -3 * torch.maximum(a.abs(), b.abs()) + 2.0 ** -6).all()
    scale = outs[1].abs().max()
    assert (outs[0] - outs[1]).abs().max() <= 2.0 ** -4 * scale


def _fixed(c):
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    kc, ks, vc, vs = (dev(a) for a in c.pool)
    args = (c.q, moe.KvCache(kc, vc, ks, vs), dev(c.table), dev(c.kv_len), dev(c.cu), c.max_nodes,
            None if c.mask is None else dev(c.mask.view(np.int32)), c.scale)
    n = moe.moe_tree_attention_workspace_bytes(c.N, c.Hq, c.Hkv, c.D, len(c.lanes))
    return args, (lambda: torch.empty((c.N, c.Hq, c.D), dtype=torch.bfloat16, device="cuda")), (
        lambda: torch.empty(n, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("Hq,nodes,D", [(4, 1, 128), (8, 6, 128), (8, 16, 128), (16, 8, 64), (8, 5, 256)])
def test_the_same_bits_many_times(Hq, nodes, D):
    """Scores that keep passing the reference (keys that grow along the lane), thousands of tiles: warps of a block
    get ahead of one another in every way, and every run has to give the same bits."""
    c = Case([(9000, nodes), (2500, nodes), (130, nodes)], Hq, 2, D, 32, seed=D + nodes, q_gain=4.0)
    for b, (p, n) in enumerate(c.lanes):
        for j in range(0, p, 7):
            page, at = c.row(b, j)
            c.pool[1][page, :, at] = np.minimum(c.pool[1][page, :, at].astype(int) + j * 4 // 9000, 250)
    args, out, ws = _fixed(c)
    o, w = out(), ws()
    moe.moe_tree_attention(*args, o, w)
    c.check(o.double().cpu().numpy(), heads=[0, Hq - 1], lanes=[1, 2])
    outs = [out() for _ in range(40)]
    for x in outs:
        moe.moe_tree_attention(*args, x, w)
    torch.cuda.synchronize()
    assert all(torch.equal(x, o) for x in outs)
    assert moe.moe_device_status() == (moe.MOE_OK, 0)


def test_two_streams_with_a_workspace_each():
    cases = [Case([(3000, 4), (500, 2)], 8, 2, 128, 32, seed=s) for s in (1, 2)]
    fixed = [_fixed(c) for c in cases]
    outs, spaces, streams = [f[1]() for f in fixed], [f[2]() for f in fixed], [torch.cuda.Stream() for _ in fixed]
    torch.cuda.synchronize()
    for _ in range(10):
        for f, o, w, s in zip(fixed, outs, spaces, streams):
            moe.moe_tree_attention(*f[0], o, w, stream=s)
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        c.check(o.double().cpu().numpy(), heads=[0, 5])
    assert moe.moe_device_status() == (moe.MOE_OK, 0)


def test_captured_step_follows_its_tables():
    """Write and attention in one CUDA graph; lengths and slots change between replays."""
    H, D, page, lanes = 2, 128, 16, 4
    cache = moe.KvCache.empty(64, H, page, D)
    table = torch.arange(64, dtype=torch.int32, device="cuda").view(lanes, 16)
    cu = torch.arange(lanes + 1, dtype=torch.int32, device="cuda")
    slots, kv_len = torch.zeros(lanes, dtype=torch.int64, device="cuda"), torch.ones(lanes, dtype=torch.int32, device="cuda")
    qkv = torch.zeros((lanes, 8 + 2 * H, D), dtype=torch.bfloat16, device="cuda")
    out = torch.empty((lanes, 8, D), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(moe.moe_tree_attention_workspace_bytes(lanes, 8, H, D, lanes), dtype=torch.uint8, device="cuda")

    def body():
        moe.moe_kv_write(qkv[:, 8:8 + H], qkv[:, 8 + H:], slots, cache)
        moe.moe_tree_attention(qkv[:, :8], cache, table, kv_len, cu, 1, None, D ** -0.5, out, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        body()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        body()
    gen = np.random.RandomState(0)
    steps = torch.from_numpy(gen.randn(200, lanes, 8 + 2 * H, D)).bfloat16().cuda()
    rows = [[] for _ in range(lanes)]
    for t, x in enumerate(steps):
        qkv.copy_(x)
        slots.copy_(torch.tensor([b * 256 + t for b in range(lanes)]))
        kv_len.fill_(t + 1)
        graph.replay()
        for b in range(lanes):
            rows[b].append(x[b].double().cpu().numpy())
        if t in (0, 15, 16, 127, 128, 199):
            got = out.double().cpu().numpy()
            for b in range(lanes):
                r = np.stack(rows[b])
                k, v = (ref.values(*ref.quantise(a)) for a in (r[:, 8:8 + H], r[:, 8 + H:]))
                for h in (0, 7):
                    o, _, mass = ref.attention(r[-1:, h], k[:, h // 4], v[:, h // 4], np.ones((1, t + 1), bool), D ** -0.5)
                    assert (np.abs(got[b, h] - o[0]) <= 2.0 ** -8 * np.abs(o[0]) + 2.0 ** -8 * mass[0] + 1e-4).all()
    assert moe.moe_device_status() == (moe.MOE_OK, 0)


def test_a_wait_that_runs_out_ends_the_kernel():
    """With a bound too short for any tile the watchdog stops the blocks; the next call is correct."""
    c = Case([(60000, 4)], 8, 2, 128, 64, seed=4)
    args, out, ws = _fixed(c)
    o, w = out(), ws()
    moe.moe_tree_attention(*args, o, w)
    want = o.clone()
    assert moe.moe_device_status() == (moe.MOE_OK, 0)
    before = moe.moe_get_wait_limit()
    moe.moe_set_wait_limit(1)
    try:
        for _ in range(20):
            moe.moe_tree_attention(*args, o, w)
        st, bits = moe.moe_device_status()
    finally:
        moe.moe_set_wait_limit(before)
    assert (st, bits) in ((moe.MOE_ETIMEOUT, moe.MOE_DEV_TIMEOUT), (moe.MOE_OK, 0))
    moe.moe_tree_attention(*args, o, w)
    assert moe.moe_device_status() == (moe.MOE_OK, 0)
    assert torch.equal(o, want)


def test_profile_names_the_kernels():
    c = Case([(2000, 3)], 8, 2, 128, 32, seed=5)
    args, out, ws = _fixed(c)
    x = torch.randn(2, 2, 128, device="cuda")
    moe.moe_profile_reset()
    moe.moe_profile_enable(True)
    try:
        moe.moe_kv_write(x, x, torch.arange(2, device="cuda"), args[1])
        moe.moe_tree_attention(*args, out(), ws())
    finally:
        moe.moe_profile_enable(False)
    got = moe.moe_profile_read()
    assert {"kv_write", "tree_attention", "tree_attention_join"} <= set(got) and all(n == 1 for n, _ in got.values())
