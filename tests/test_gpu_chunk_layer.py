"""Plan, norms and rotation, cache, chunk attention and experts together, as a serving loop uses them."""
import numpy as np
import pytest
import torch

from tests import kv_reference as ref

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("resident_expert_routed_gb300")


def norms(seed=0, norm=True):
    from resident_expert_routed_gb300.decode import HeadNorms
    from resident_expert_routed_gb300.rotary import rotary_frequencies, rotary_turns
    gen = torch.Generator(device="cuda").manual_seed(seed)
    w = [1 + 0.2 * torch.randn(64, generator=gen, device="cuda") if norm else None for _ in range(2)]
    return HeadNorms(rotary_turns(rotary_frequencies(64)), *w)


def rows_of(cache, table, n):
    k, v = (torch.empty((n, 2, 64), device="cuda") for _ in range(2))
    moe.moe_kv_read(cache, table[:1].contiguous(), None, torch.tensor([0, n], dtype=torch.int32, device="cuda"), k, v)
    return k, v


def attended(layer, n):
    """The attention's outputs of the layer's last call. (Behind them the router picks experts: a rounding may pick another one,
    and no bound on what it is given bounds what comes out.)"""
    return layer.out[:n].float().clone()


def near(a, b, most):
    """Outputs of two ways to the same attention, `most` the largest value that they weigh up: one e4m3 step (2^-3) of some values
    where a projection's rounding falls on the other side, an eighth of which and more averages out over a lane's rows; roundings
    of weights and outputs (2^-8 each, of both)."""
    return (a - b).abs().max() <= 2.0 ** -4 * most


def test_the_example_runs_and_its_pages_add_up():
    from examples import chunked_prefill
    layer, pages = chunked_prefill.main(steps=30, seed=3)
    again, pages2 = chunked_prefill.main(steps=30, seed=3)
    for name in ("rows", "held", "table", "n_free"):
        assert torch.equal(getattr(pages, name), getattr(pages2, name))
    assert torch.equal(layer.cache.k_codes, again.cache.k_codes) and torch.equal(layer.cache.v_scales, again.cache.v_scales)


def test_the_example_with_too_few_pages_refuses_and_goes_on():
    from examples.tree_decode import build
    from resident_expert_routed_gb300.decode import DevicePages
    layer, pages = build(2, 64, 3), DevicePages(2, 3, 16, 8, 64)
    n = torch.tensor([40, 20], dtype=torch.int32, device="cuda")
    pages.plan(n)
    hidden = torch.randn(60, 256, device="cuda").bfloat16()
    out = layer.chunk(hidden, pages)
    st, bits = moe.moe_device_status()
    assert bits & moe.MOE_DEV_NO_PAGES and torch.isfinite(out).all()
    pages.advance()
    assert pages.rows.tolist() == [40, 0] and pages.n_free.item() == 0
    pages.plan(torch.tensor([-1, 20], dtype=torch.int32, device="cuda"))
    pages.advance()
    assert pages.rows.tolist() == [0, 20] and moe.moe_device_status() == (moe.MOE_OK, 0)


@pytest.mark.parametrize("with_norms", [False, True])
def test_a_chunk_gives_what_a_chain_gives(with_norms):
    """The same prompt as a chunk over pages planned on the device and as a chain of the tree's kernel over the host's pages: the
    same rows in the cache bit for bit (one batch, the same products), the same outputs up to the attentions' roundings. Each is
    within 2^-8 |o| + (2^-8 + 2 d) sum p |v| of the definition; d, queries held to 2^-13 of their row's largest, is below 2^-8 for
    64 products of size 4 and less; |o| and sum p |v| are at most the largest |v|: 2 (2^-8 + 2^-8 + 2^-7) of it."""
    from examples.tree_decode import build
    from resident_expert_routed_gb300.decode import DevicePages, LanePages, Step
    torch.manual_seed(1)
    prompt = torch.randn(200, 256, device="cuda").bfloat16()
    c = norms() if with_norms else None
    layer, pages = build(1, 256, 16, norms=c), DevicePages(1, 16, 16, 16, 256)
    pages.plan(torch.tensor([200], dtype=torch.int32, device="cuda"))
    layer.chunk(prompt, pages)
    a = attended(layer, 200)
    pages.advance()
    other, host = build(1, 256, 16, norms=c), LanePages(1, 16, 16, 16)
    other.step(prompt, Step(host, [list(range(-1, 199))]), tree=False)
    b = attended(other, 200)
    host.advance(0, 200)
    rows = rows_of(layer.cache, pages.table, 200)
    for x, y in zip(rows, rows_of(other.cache, host.table.cuda(), 200)):
        assert torch.equal(x, y)
    assert (a - b).abs().max() <= 2.0 ** -5 * rows[1].abs().max()
    assert moe.moe_device_status() == (moe.MOE_OK, 0)


def test_pieces_give_what_the_whole_gives():
    """A prompt in three chunks and two single tokens beside another lane, against the prompt at once."""
    from examples.tree_decode import build
    from resident_expert_routed_gb300.decode import DevicePages
    torch.manual_seed(2)
    prompt, noise = torch.randn(150, 256, device="cuda").bfloat16(), torch.randn(64, 256, device="cuda").bfloat16()
    whole, pages = build(1, 256, 32, norms=norms()), DevicePages(1, 32, 16, 16, 256)
    pages.plan(torch.tensor([150], dtype=torch.int32, device="cuda"))
    whole.chunk(prompt, pages)
    want, most = attended(whole, 150), rows_of(whole.cache, pages.table, 150)[1].abs().max()
    layer, pages = build(2, 256, 32, norms=norms()), DevicePages(2, 32, 16, 16, 256)
    at, got = 0, []
    for n, beside in ((60, 7), (1, 0), (1, 3), (80, 1), (8, 20)):
        pages.plan(torch.tensor([n, beside], dtype=torch.int32, device="cuda"))
        layer.chunk(torch.cat([prompt[at:at + n], noise[:beside]]), pages)
        got.append(attended(layer, n))
        pages.advance()
        at += n
    assert pages.rows.tolist() == [150, 31] and near(torch.cat(got), want, most)
    assert moe.moe_device_status() == (moe.MOE_OK, 0)


def test_a_drafted_path_has_the_positions_of_single_tokens():
    """With rotary positions a tree's path, checked at once and kept, gives what its tokens give one by one in chunks."""
    from examples.tree_decode import build
    from resident_expert_routed_gb300.decode import DevicePages, LanePages, Step
    torch.manual_seed(3)
    parents, path = [-1, 0, 0, 1, 2, 4, 3, 5], [0, 2, 4, 5, 7]
    prompt, drafted = torch.randn(40, 256, device="cuda").bfloat16(), torch.randn(8, 256, device="cuda").bfloat16()
    layer, host = build(1, 64, 8, norms=norms()), LanePages(1, 8, 16, 8)
    layer.step(prompt, Step(host, [list(range(-1, 39))]), tree=False)
    host.advance(0, 40)
    t = Step(host, [parents])
    assert t.positions.tolist() == [40, 41, 41, 42, 42, 43, 43, 44]
    layer.step(drafted, t)
    a = attended(layer, 8)[path]
    layer.keep(t, torch.tensor([path], dtype=torch.int32, device="cuda"), torch.tensor([5], dtype=torch.int32, device="cuda"))
    other, pages = build(1, 64, 8, norms=norms()), DevicePages(1, 8, 16, 8, 64)
    one = torch.tensor([1], dtype=torch.int32, device="cuda")
    pages.plan(40 * one)
    other.chunk(prompt, pages)
    pages.advance()
    got = []
    for i in path:
        pages.plan(one)
        other.chunk(drafted[i:i + 1], pages)
        got.append(attended(other, 1))
        pages.advance()
    k0, v0 = rows_of(layer.cache, host.table.cuda(), 45)
    k1, v1 = rows_of(other.cache, pages.table, 45)
    assert near(torch.cat(got), a, v0.abs().max())
    # one e4m3 step where a product's rounding falls on the other side
    for x, y in ((k0, k1), (v0, v1)):
        assert ((x - y).abs() <= 2.0 ** -3 * torch.maximum(x.abs(), y.abs()) + 2.0 ** -6).all()
    assert moe.moe_device_status() == (moe.MOE_OK, 0)


def test_captured_batches_follow_their_lengths():
    """Plan, rotation, write and attention in one graph; what each lane gets changes between replays."""
    lanes, T, H, D, page = 3, 96, 2, 128, 16
    rng = np.random.RandomState(4)
    from resident_expert_routed_gb300.decode import DevicePages
    from resident_expert_routed_gb300.rotary import rotary_frequencies, rotary_turns
    pages, cache = DevicePages(lanes, 64, page, 20, T), moe.KvCache.empty(64, H, page, D)
    f = rotary_frequencies(D)
    turns = rotary_turns(f)
    n_new = torch.zeros(lanes, dtype=torch.int32, device="cuda")
    qkv = torch.zeros((T, 8 + 2 * H, D), dtype=torch.bfloat16, device="cuda")
    q, k = torch.empty((T, 8, D), dtype=torch.bfloat16, device="cuda"), torch.empty((T, H, D), dtype=torch.bfloat16, device="cuda")
    out = torch.empty((T, 8, D), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(moe.moe_chunk_attention_workspace_bytes(T, 8, H, D, lanes), dtype=torch.uint8, device="cuda")

    def body():
        pages.plan(n_new)
        moe.moe_qk_rotate(qkv[:, :8], qkv[:, 8:8 + H], pages.positions, turns, q, k)
        moe.moe_kv_write(k, qkv[:, 8 + H:], pages.slots, cache)
        moe.moe_chunk_attention(q, cache, pages.table, pages.kv_len, pages.cu, D ** -0.5, out, ws)
        pages.advance()

    body()                                                       # (no tokens yet)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        body()
    kept = [[[], []] for _ in range(lanes)]
    for new in ([40, 0, 50], [1, 30, 1], [1, 1, 1], [60, 20, 0], [0, 1, 90]):
        qkv.copy_(torch.from_numpy(rng.randn(T, 8 + 2 * H, D)).bfloat16())
        n_new.copy_(torch.tensor(new, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        at, qh, kh, vh = 0, *(x.double().cpu().numpy() for x in (q, k, qkv[:, 8 + H:]))
        for b, n in enumerate(new):
            for side_, x in zip(kept[b], (kh, vh)):
                side_.extend(x[at:at + n])
            rows = len(kept[b][0])
            kk, vv = (ref.values(*ref.quantise(np.stack(x))) if rows else None for x in kept[b])
            for t in sorted({0, n // 2, n - 1}) if n else ():
                p = rows - n + t
                assert pages.positions[at + t].item() == p
                for h in (0, 7):
                    o, _, mass = ref.attention(qh[at + t:at + t + 1, h], kk[:p + 1, h // 4], vv[:p + 1, h // 4], np.ones((1, p + 1), bool), D ** -0.5)
                    got = out[at + t, h].double().cpu().numpy()
                    # weights' and output's roundings, 2^-8 each; queries held to 2^-13 of their row
                    assert (np.abs(got - o[0]) <= 2.0 ** -8 * np.abs(o[0]) + (2.0 ** -8 + 2.0 ** -8) * mass[0]).all(), (new, b, t)
            at += n
    assert pages.rows.tolist() == [len(x[0]) for x in kept]
    assert moe.moe_device_status() == (moe.MOE_OK, 0)


def test_profile_names_the_kernels():
    from examples.tree_decode import build
    from resident_expert_routed_gb300.decode import DevicePages
    layer, pages = build(1, 64, 8, norms=norms()), DevicePages(1, 8, 16, 8, 64)
    n, hidden = torch.tensor([20], dtype=torch.int32, device="cuda"), torch.randn(20, 256, device="cuda").bfloat16()
    moe.moe_profile_reset()
    moe.moe_profile_enable(True)
    try:
        pages.plan(n)
        layer.chunk(hidden, pages)
    finally:
        moe.moe_profile_enable(False)
    got = moe.moe_profile_read()
    assert {"page_plan", "qk_rotate", "kv_write", "chunk_attention"} <= set(got)
