"""Weights of tree attention far below the largest, value vectors of zeros and of very different size, against the
definition in 64 bits.

Bounds. A weight is held to 2^-9 of itself, or to 2^-28 of the largest weight times its value vector's scale, whichever
is more; the scores and the sums are fp32 (2^-11 of the weights covers their roundings, and the queries'), and the
output is rounded to bf16 once (half a unit: 2^-9 to 2^-8, of which 2^-9 is asked for, as the weights' bound is hardly
reached; and 2^-134 where bf16's steps end). So
  |out - o| <= max(2^-9 |o|, 2^-134) + (2^-9 + 2^-11) sum p |v| + 2^-28 max(p 2^ev) sum |codes|,
each column for itself. A log sum is off by the rounding of the scores and the scale exponents that are
added to them (at most 2^7: 2^-17 each) and a few 2^-22.
"""
import numpy as np
import pytest
import torch

from tests import kv_reference as ref
from tests.test_gpu_tree_attention import Case

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("resident_expert_routed_gb300")


def definition(q, k, codes, scales, see, scale):
    """(out [n, D], lse [n], tolerance [n, D]) of one lane and head: q [n, D], k [L, D] values, codes and scales of v."""
    v, unit = ref.values(codes, scales), 2.0 ** (scales.astype(np.float64) - 127)
    c = np.abs(ref.E4M3[codes])
    out, lse, tol = np.zeros(q.shape), np.full(len(q), -np.inf), np.zeros(q.shape)
    for t in range(len(q)):
        j = np.flatnonzero(see[t])
        if not len(j):
            continue
        s = k[j] @ q[t] * scale
        p = np.exp(s - s.max())
        total = p.sum()
        held = c[j].any(-1)                   # a vector of zeros adds to the sum of weights alone
        most = (p * unit[j])[held].max(initial=0.0)
        out[t], lse[t] = p @ v[j] / total, s.max() + np.log(total)
        tol[t] = np.maximum(2.0 ** -9 * np.abs(out[t]), 2.0 ** -134) + ((2.0 ** -9 + 2.0 ** -11) * (p @ np.abs(v[j])) + 2.0 ** -28 * most * c[j].sum(0)) / total
    return out, lse, tol


def check(c, got, lse, lanes=None):
    k = ref.values(*c.pool[:2])
    G = c.Hq // c.Hkv
    for b, (p, n) in enumerate(c.lanes):
        if lanes is not None and b not in lanes:
            continue
        see = ref.visible(n, p + n, c.mask, c.cu[b])
        kb, codes, scales = (ref.lane_rows(x, c.table[b], p + n) for x in (k, *c.pool[2:]))
        rows = slice(c.cu[b], c.cu[b + 1])
        for h in range(c.Hq):
            o, e, tol = definition(c.q_host[rows, h], kb[:, h // G], codes[:, h // G], scales[:, h // G], see, c.scale)
            off = np.abs(got[rows, h] - o)
            assert (off <= tol).all(), (b, h, float((off / np.maximum(tol, 1e-300)).max()))
            none = np.isneginf(e)
            assert np.array_equal(np.isneginf(lse[rows, h]), none)
            mags = np.abs(c.q_host[rows, h]) @ np.abs(kb[:, h // G]).max(0) * c.scale
            bound = 2.0 ** -16 + 2.0 ** -20 * np.abs(e[~none]) + c.D * 2.0 ** -24 * mags[~none]
            assert (np.abs(lse[rows, h] - e)[~none] <= bound).all(), (b, h, np.abs(lse[rows, h] - e)[~none].max())
    assert moe.moe_device_status() == (moe.MOE_OK, 0)


# ------------------------------------------------------------------ small weights of one size

@pytest.mark.parametrize("bits", [4.3, 8.9, 12.84, 13.5, 15.84, 16.3, 18.55])
@pytest.mark.parametrize("D,G,nodes", [(128, 1, 1), (128, 4, 6), (128, 8, 8), (64, 8, 8), (256, 4, 7)])
def test_a_flat_tail_below_a_peak(bits, D, G, nodes):
    """Two peaks (one for each half of the work on a lane's tiles) before 8,190 rows of one weight each, 2^-bits of a
    peak's; the tail's values have a column of their own. The tail's rows are one page, again and again."""
    H, page, rows, lanes = 8, 128, 8192, 20
    rng = np.random.RandomState(1)
    kc = np.full((3, H, page, D), 0x38, np.uint8)                        # keys of ones, times 2^-8; a peak's are 2^-7
    ks = np.full((3, H, page), 127 - 8, np.uint8)
    ks[:2, :, 0] += 1
    vc, vs = np.empty_like(kc), np.empty_like(ks)
    x = rng.randn(3, H, page, D)
    x[:, :, :, 0], x[:, :, :, 1] = 1.0, 0.0
    x[:2, :, 0, 0], x[:2, :, 0, 1] = 0.0, 1.0
    for i in range(3):
        vc[i], vs[i] = ref.quantise(x[i])
    table = np.full((lanes, rows // page), 2, np.int32)
    table[:, 0], table[:, 1] = 0, 1
    n, Hq = lanes * nodes, G * H
    cu = np.arange(lanes + 1, dtype=np.int32) * nodes
    mask = np.tile((1 << np.arange(nodes, dtype=np.int64)).astype(np.int32), lanes)[:, None]       # its own row, no other node's
    scale = float(bits * np.log(2.0) / (D * 2.0 ** -8))
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    cache = moe.KvCache(dev(kc), dev(vc), dev(ks), dev(vs))
    q = torch.ones((n, Hq, D), dtype=torch.bfloat16, device="cuda")
    out = torch.full((n, Hq, D), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((n, Hq), device="cuda")
    ws = torch.empty(moe.moe_tree_attention_workspace_bytes(n, Hq, H, D, lanes), dtype=torch.uint8, device="cuda")
    moe.moe_tree_attention(q, cache, dev(table), torch.full((lanes,), rows, dtype=torch.int32, device="cuda"), dev(cu), nodes, dev(mask),
                           scale, out, ws, lse=lse)
    got, gl = out.double().cpu().numpy().reshape(lanes, nodes, H, G, D), lse.double().cpu().numpy().reshape(lanes, nodes, H, G)
    assert moe.moe_device_status() == (moe.MOE_OK, 0)
    at, k = np.arange(rows), ref.values(kc, ks)
    see = np.ones((nodes, rows), bool)
    see[:, rows - nodes:] = np.eye(nodes, dtype=bool)
    for h in range(H):
        kl, cl, sl = (a[table[0, at // page], h, at % page] for a in (k, vc, vs))
        o, e, tol = definition(np.ones((nodes, D)), kl, cl, sl, see, scale)
        off = np.abs(got[:, :, h] - o[None, :, None, :])
        assert (off <= tol[None, :, None, :]).all(), (h, float((off / tol[None, :, None, :]).max()))
        # scores of up to 2^5: 2^-20 of them, and the tail's sum
        assert (np.abs(gl[:, :, h] - e[None, :, None]) <= 2.0 ** -16 + 2.0 ** -20 * np.abs(e).max()).all()


def test_a_value_row_that_is_large_in_one_column():
    # the other columns hold what the small rows give, 2^13 below
    c = Case([(900, 3), (300, 2)], 8, 2, 128, 32, seed=21)
    for b, j in ((0, 5), (0, 700), (1, 290)):
        page, at = c.row(b, j)
        c.pool[2][page, :, at], c.pool[3][page, :, at] = 0, 127 + 6
        c.pool[2][page, :, at, 17] = 0x78                                # 256
    check(c, *c.gpu())


# ------------------------------------------------------------------ value vectors of very different size

@pytest.mark.parametrize("sizes", [(-91, 58), (58, -91), (-100, 120), (120, -100), (60, -70), (-70, 60)])
@pytest.mark.parametrize("rows", [256, 700, 9000, 40000])
def test_tiles_of_values_of_very_different_size(sizes, rows):
    """Tiles of which all values are tiny before, after or between tiles of which all are huge: the tiny ones' weights
    still count in full in the sum of weights."""
    c = Case([(rows - 1, 1), (rows // 2, 1)], 2, 1, 128, 128, tree=False, seed=31)
    for b, (p, n) in enumerate(c.lanes):
        for t in range(-(-(p + n) // 128)):
            c.pool[3][c.table[b, t]] = 127 + sizes[t // 2 % 2 if rows < 1000 else t * 4 // -(-rows // 128) % 2]
            if max(sizes) == 120:
                c.pool[2][c.table[b, t]] &= 0x9F                          # codes below 2^-3, so that values stay below 2^118
    check(c, *c.gpu())


@pytest.mark.parametrize("nodes,Hq", [(4, 4), (9, 8), (16, 8)])
def test_a_few_huge_values_among_tiny_ones(nodes, Hq):
    c = Case([(1500, nodes), (300, nodes)], Hq, 2, 64, 32, seed=32)
    c.pool[3][:] = 127 - 95
    for b, j in ((0, 3), (0, 1400), (1, 200)):
        page, at = c.row(b, j)
        c.pool[3][page, :, at] = 127 + 40
    check(c, *c.gpu())


# ------------------------------------------------------------------ value vectors of zeros

def zero_value(c, b, j, head=slice(None), code=0):
    """As the cache holds a vector of zeros: codes 0 (or of the sign alone) and scale 2^0."""
    page, at = c.row(b, j)
    c.pool[2][page, head, at], c.pool[3][page, head, at] = code, 127


@pytest.mark.parametrize("size", [0, -7, -16, -24, -90])
@pytest.mark.parametrize("D,Hq,Hkv,nodes", [(128, 4, 2, 1), (64, 8, 4, 5), (128, 16, 2, 8), (256, 8, 2, 3)])
def test_zero_value_rows(size, D, Hq, Hkv, nodes):
    # values of size 2^size; rows of zeros first, in the middle of a tile, in one head alone, a whole tile, among the drafted nodes
    c = Case([(700, nodes), (7, nodes), (130, nodes), (1900, nodes), (0, nodes)], Hq, Hkv, D, 32, seed=40 + D)
    c.pool[3][:] = np.clip(c.pool[3].astype(int) + size, 27, 247)
    for b, j in ((0, 0), (0, 77), (1, 3), (2, 129), (3, 1899), (4, 0)):
        zero_value(c, b, j)
    for j in range(256, 384):
        zero_value(c, 3, j)
    zero_value(c, 0, 400, head=0, code=0x80)
    check(c, *c.gpu())


@pytest.mark.parametrize("bits", [6.0, 14.0, 16.0, 22.5])
@pytest.mark.parametrize("at", [0, 130, 511])
def test_a_zero_value_with_the_highest_score(bits, at):
    # most of the weight lies on a vector of zeros; what is left keeps its precision
    c = Case([(511, 1)], 2, 1, 128, 64, tree=False, seed=50)
    c.pool[0][:], c.pool[1][:] = 0x38, 127 - 8
    c.q = torch.ones_like(c.q)
    c.q_host = c.q.cpu().double().numpy()
    c.scale = float(bits * np.log(2.0) / 0.5)
    page, row = c.row(0, at)
    c.pool[1][page, 0, row] = 127 - 7
    zero_value(c, 0, at)
    check(c, *c.gpu())


def test_zero_values_alone():
    # nothing else is seen: by single tokens, by a node of a tree, in a lane of a cache that holds nothing yet
    c = Case([(4, 1), (0, 1), (300, 3), (1300, 2)], 4, 2, 128, 16, seed=60)
    for b in (0, 1, 3):
        for j in range(sum(c.lanes[b])):
            zero_value(c, b, j)
    c.lanes[2], c.kv_len[2] = (0, 3), 3              # three nodes without a prefix, the second of which sees itself alone
    zero_value(c, 2, 1)
    c.mask[3, 0] = 0b010
    got, lse = c.gpu()
    check(c, got, lse)
    assert not got[:2].any() and not got[3].any() and not got[5:].any() and np.isfinite(lse).all() and got[2].any()


def test_a_value_row_of_scale_one_is_no_zero():
    # scale 2^0 with codes that are zero but for the last, and infinities in rows that nobody sees
    c = Case([(200, 4)], 4, 2, 128, 16, seed=61)
    for j in (0, 150):
        zero_value(c, 0, j)
        page, at = c.row(0, j)
        c.pool[2][page, :, at, 127] = 0x01
    c.mask[:, 0] = [0b0001, 0b0001, 0b0101, 0b1001]
    zero_value(c, 0, 201)
    check(c, *c.gpu())


def test_written_zeros_are_attended_as_zeros():
    H, page, D = 2, 16, 128
    cache = moe.KvCache.empty(4, H, page, D)
    x = torch.randn(40, 2 * H, D, device="cuda").bfloat16()
    x[:, H:] *= 1e-3
    x[5:9, H:] = 0.0
    x[30, H] = -0.0
    moe.moe_kv_write(x[:, :H], x[:, H:], torch.arange(40, device="cuda"), cache)
    q = torch.randn(1, 4, D, device="cuda").bfloat16()
    out, lse = torch.empty_like(q), torch.empty((1, 4), device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = torch.empty(moe.moe_tree_attention_workspace_bytes(1, 4, H, D, 1), dtype=torch.uint8, device="cuda")
    moe.moe_tree_attention(q, cache, i32(0, 1, 2, 3).view(1, 4), i32(40), i32(0, 1), 1, None, D ** -0.5, out, ws, lse=lse)
    got, host = out.double().cpu().numpy(), [t.cpu().numpy() for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)]
    kc, ks, vc, vs = (ref.lane_rows(a, np.arange(4), 40) for a in host)
    for h in range(4):
        o, e, tol = definition(q[:, h].double().cpu().numpy(), ref.values(kc, ks)[:, h // 2], vc[:, h // 2], vs[:, h // 2],
                               np.ones((1, 40), bool), D ** -0.5)
        assert (np.abs(got[:, h] - o) <= tol).all() and abs(lse[0, h].item() - e[0]) <= 2.0 ** -15
    assert moe.moe_device_status() == (moe.MOE_OK, 0)
