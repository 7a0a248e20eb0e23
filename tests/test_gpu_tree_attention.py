"""Tree attention over the paged 8-bit cache on the GPU, against a plain implementation in 64 bits.

The cache's values are exact on both sides, so what is left are roundings of
the computation. Bounds: p is held with a relative error of at most 2^-8 (8
significant bits), which moves an output by at most 2^-8 of sum p |v|; the
output's own rounding to bf16 is at most 2^-8 of it; weights below 2^-18 of a
tile's largest may be flushed, 128 of them at most 2^-11 of the largest |v|
(taken in full only where one tile holds all the weight). lse: products of e4m3
and bf16 values are exact in fp32, a sum of D of them is off by at most D 2^-24
of the sum of magnitudes; the exponential, the sum and the logarithm add a few
2^-22.
"""
import numpy as np
import pytest
import torch

from tests import kv_reference as ref

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("resident_expert_routed_gb300")


class Case:
    """Lanes of given (prefix rows, nodes) over a cache with random rows; tree masks of random ancestors."""

    def __init__(self, lanes, Hq, Hkv, D, page, tree=True, seed=0, pages_extra=2, q_gain=1.0):
        rng = self.rng = np.random.RandomState(seed)
        self.lanes, self.Hq, self.Hkv, self.D, self.page = lanes, Hq, Hkv, D, page
        total = [p + n for p, n in lanes]
        need = [-(-t // page) for t in total]
        pages = sum(need) + pages_extra
        self.pool = []
        for _ in range(2):
            x = (rng.randn(pages, Hkv, page, D) * np.exp(rng.randn(pages, Hkv, page, 1))).astype(np.float32)
            amax = np.abs(x).max(-1)
            e = np.ceil(np.log2(amax / 448.0)).astype(int)
            codes = ref.round_e4m3(x.astype(np.float64) * 2.0 ** -e[..., None].astype(np.float64))
            self.pool += [codes, (e + 127).astype(np.uint8)]
        self.table = np.full((len(lanes), max(1, max(need))), -1, np.int32)
        ids = rng.permutation(pages)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        self.spare = ids[at:]
        self.kv_len = np.array(total, np.int32)
        self.cu = np.r_[0, np.cumsum([n for _, n in lanes])].astype(np.int32)
        self.N, self.max_nodes = int(self.cu[-1]), max(1, max(n for _, n in lanes))
        q = torch.from_numpy(rng.randn(self.N, Hq, D) * q_gain).bfloat16()
        self.q, self.q_host = q.cuda(), q.double().numpy()
        self.scale = D ** -0.5
        self.mask = None
        if tree:
            self.mask = np.zeros((self.N, -(-self.max_nodes // 32)), np.uint32)
            for b, (_, n) in enumerate(lanes):
                for i in range(n):
                    row = self.mask[self.cu[b] + i]
                    if i:
                        row |= self.mask[self.cu[b] + rng.randint(0, i)]
                    row[i // 32] |= np.uint32(1 << (i % 32))

    def row(self, b, j):
        return self.table[b, j // self.page], j % self.page

    def gpu(self, lse=True, stream=None, workspace=None, q=None):
        kc, ks, vc, vs = (torch.from_numpy(a).cuda() for a in self.pool)
        cache = moe.KvCache(kc, vc, ks, vs)
        dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
        out = torch.full((self.N, self.Hq, self.D), 9.0, dtype=torch.bfloat16, device="cuda")
        l = torch.full((self.N, self.Hq), 9.0, device="cuda") if lse else None
        if workspace is None:
            n = moe.moe_tree_attention_workspace_bytes(self.N, self.Hq, self.Hkv, self.D, len(self.lanes))
            workspace = torch.randint(0, 256, (n,), dtype=torch.uint8, device="cuda")
        args = (self.q if q is None else q, cache, dev(self.table), dev(self.kv_len), dev(self.cu), self.max_nodes,
                None if self.mask is None else dev(self.mask.view(np.int32)), self.scale, out, workspace)
        torch.cuda.synchronize()
        moe.moe_tree_attention(*args, lse=l, stream=stream)
        torch.cuda.synchronize()
        return out.double().cpu().numpy(), None if l is None else l.double().cpu().numpy()

    def check(self, got, lse=None, lanes=None, heads=None):
        k, v = ref.values(*self.pool[:2]), ref.values(*self.pool[2:])
        G = self.Hq // self.Hkv
        for b, (p, n) in enumerate(self.lanes):
            if not n or (lanes is not None and b not in lanes):
                continue
            see = ref.visible(n, p + n, self.mask, self.cu[b])
            kb, vb = (ref.lane_rows(x, self.table[b], p + n) for x in (k, v))
            rows = slice(self.cu[b], self.cu[b + 1])
            for h in range(self.Hq) if heads is None else heads:
                kh, vh = kb[:, h // G], vb[:, h // G]
                o, e, mass = ref.attention(self.q_host[rows, h], kh, vh, see, self.scale)
                g = got[rows, h]
                assert np.array_equal(np.isnan(g), np.isnan(o)), (b, h)
                fine = ~np.isnan(o)
                big = np.nanmax(np.where(see.any(0)[:, None], np.abs(vh), 0.0), initial=0.0)
                tol = 2.0 ** -8 * np.abs(o) + 2.0 ** -8 * mass + 2.0 ** -11 * big * 2.0 ** -4 + 1e-30
                off = np.abs(g - o)
                assert (off[fine] <= tol[fine]).all(), (b, h, np.nanmax(off / tol))
                if lse is not None:
                    x = lse[rows, h]
                    assert np.array_equal(np.isnan(x), np.isnan(e)) and np.array_equal(np.isneginf(x), np.isneginf(e))
                    ok = np.isfinite(e)
                    mags = np.abs(self.q_host[rows, h]) @ np.nan_to_num(np.abs(kh)).max(0) * self.scale
                    bound = 2.0 ** -20 * (1 + np.abs(e)) + self.D * 2.0 ** -24 * mags
                    assert (np.abs(x - e)[ok] <= bound[ok]).all(), (b, h, np.abs(x - e)[ok].max())


def run_and_check(c, **kw):
    got, lse = c.gpu()
    c.check(got, lse, **kw)
    assert moe.moe_device_status() == (moe.MOE_OK, 0)
    return got, lse


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 63, 127, 128, 129, 255, 257, 700])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 64), (256, 32)])
def test_single_token(rows, D, page):
    run_and_check(Case([(rows - 1, 1)], 4, 2, D, page, tree=False, seed=rows))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (6, 2), (5, 1), (16, 1), (40, 8), (24, 1), (64, 8), (100, 1)])
@pytest.mark.parametrize("nodes", [1, 3, 17])
def test_head_layouts(Hq, Hkv, nodes):
    run_and_check(Case([(150, nodes), (3, nodes)], Hq, Hkv, 128, 16, seed=Hq + nodes))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 32, 128, 256, 1024])
@pytest.mark.parametrize("tree", [True, False])
def test_ragged_lanes(D, page, tree):
    lanes = [(300, 5), (0, 7), (1, 1), (127, 1), (129, 16), (40, 0), (0, 1), (255, 9), (0, 0), (513, 3)]
    run_and_check(Case(lanes, 8, 2, D, page, tree=tree, seed=D + page))


@pytest.mark.parametrize("nodes", [31, 32, 33, 64, 65, 130, 300])
@pytest.mark.parametrize("tree", [True, False])
def test_wide_trees(nodes, tree):
    run_and_check(Case([(70, nodes), (0, nodes - 1)], 4, 2, 128, 16, tree=tree, seed=nodes))


def test_many_lanes():
    rng = np.random.RandomState(0)
    lanes = [(int(rng.randint(0, 400)), int(rng.randint(0, 4))) for _ in range(300)]
    run_and_check(Case(lanes, 4, 2, 64, 32, seed=1))


@pytest.mark.parametrize("D,Hq,Hkv,nodes", [(128, 8, 1, 1), (128, 16, 2, 9), (64, 4, 4, 1), (256, 4, 1, 3)])
def test_one_long_lane(D, Hq, Hkv, nodes):
    # far more rows than one block would take: the rows are split and joined
    run_and_check(Case([(40001, nodes)], Hq, Hkv, D, 64, seed=D + nodes), heads=[0, Hq - 1])


def test_uneven_long_lanes():
    run_and_check(Case([(20000, 2), (5, 3), (9000, 1), (0, 1), (777, 8)], 8, 2, 128, 32, seed=3), heads=[0, 7])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_long_lanes_whose_last_units_are_short(D):
    # 72, 8, 24, 128 and 96 tree rows a kv head: full units, and ones of which most rows are missing
    run_and_check(Case([(9000, 9), (6500, 1), (0, 3), (7300, 16), (8100, 12)], 16, 2, D, 32, seed=D), heads=[0, 7, 15])


@pytest.mark.parametrize("nodes", [2, 9])
def test_more_lanes_than_a_block_has_threads(nodes):
    rng = np.random.RandomState(nodes)
    lanes = [(int(rng.randint(0, 1500 if b % 50 == 0 else 150)), int(rng.randint(0, nodes + 1))) for b in range(900)]
    run_and_check(Case(lanes, 8, 2, 64, 16, seed=nodes), heads=[0, 5], lanes=set(range(0, 900, 25)) | {899})


def test_nodes_that_see_nothing():
    c = Case([(0, 4), (0, 1), (200, 3), (0, 40)], 4, 2, 128, 16, seed=2)
    c.mask[1] = 0                         # of the first lane
    c.mask[4] = 0                         # the whole second lane
    c.mask[6] = 0                         # sees its lane's prefix alone
    c.mask[20:30] = 0
    got, lse = run_and_check(c)
    assert not got[1].any() and not got[4].any() and np.isneginf(lse[1]).all() and np.isneginf(lse[4]).all()
    assert np.isfinite(lse[6]).all() and np.isneginf(lse[20:30]).all()


def test_mask_bits_past_the_tree_do_nothing():
    c = Case([(30, 5), (31, 33)], 2, 1, 64, 16, seed=8)
    want, _ = run_and_check(c)
    c.mask[:5, 0] |= np.uint32(0xFFFFFFE0)
    c.mask[:5, 1] = 0xFFFFFFFF
    c.mask[5:, 1] |= np.uint32(0xFFFFFFFE)
    got, _ = c.gpu()
    assert np.array_equal(got, want)


@pytest.mark.parametrize("scale_byte,code", [(255, 0x00), (255, 0x35), (254, 0x7E), (0, 0x01)])
def test_rows_not_seen_do_nothing(scale_byte, code):
    # NaN vectors and the largest finite ones in the rows of sibling nodes
    c = Case([(100, 6), (0, 3)], 4, 2, 128, 16, seed=5)
    c.mask[:] = 0
    for i, m in enumerate([0b1, 0b11, 0b101, 0b1101, 0b10001, 0b100001]):
        c.mask[i] = m
    for i in range(3):
        c.mask[6 + i] = 1 << i
    # nodes 1 and 4 of the first lane are seen by themselves alone; nobody sees node 1 once its own bit is off
    c.mask[1] = 0b1
    c.mask[4] = 0b1
    for i in (1, 4):
        page, at = c.row(0, 100 + i)
        for codes, scales in (c.pool[:2], c.pool[2:]):
            codes[page, :, at] = code
            scales[page, :, at] = scale_byte
    run_and_check(c)


def test_rows_past_the_lane_do_nothing():
    # what lies behind a lane's rows on its last page, and on pages it does not have, is arbitrary bytes
    c = Case([(37, 2), (128, 1), (0, 1), (250, 5)], 4, 2, 128, 64, seed=6)
    for b, (p, n) in enumerate(c.lanes):
        for j in range(p + n, -(-(p + n) // c.page) * c.page):
            page, at = c.row(b, j)
            for codes, scales in (c.pool[:2], c.pool[2:]):
                codes[page, :, at] = 0x7F
                scales[page, :, at] = 255
    for page in c.spare:
        for codes, scales in (c.pool[:2], c.pool[2:]):
            codes[page], scales[page] = 0xFF, 255
    run_and_check(c)


def test_a_nan_vector_that_is_seen():
    # a NaN key or value reaches exactly the nodes and heads that see it
    c = Case([(130, 3), (9, 2)], 4, 2, 128, 16, seed=7)
    c.mask[:3, 0] = [0b001, 0b011, 0b101]
    for which, (b, j, h) in ((0, (0, 131, 1)), (2, (0, 132, 0)), (2, (1, 4, 1))):
        page, at = c.row(b, j)
        c.pool[which][page, h, at] = 0
        c.pool[which + 1][page, h, at] = 255
    k, v = ref.values(*c.pool[:2]), ref.values(*c.pool[2:])
    assert np.isnan(k).any() and np.isnan(v).any()
    got, lse = c.gpu()
    nan = np.isnan(got).all(-1)
    assert np.array_equal(nan, np.isnan(got).any(-1))
    want = np.zeros((5, 4), bool)
    want[1, 2:] = True                    # node 1 of lane 0 sees itself: NaN key in kv head 1
    want[2, :2] = True                    # node 2 sees itself: NaN value in kv head 0
    want[3:, 2:] = True                   # lane 1: a NaN value in the prefix, kv head 1
    assert np.array_equal(nan, want)
    fine = [(n, h) for n in range(5) for h in range(4) if not want[n, h]]
    assert all(np.isfinite(got[n, h]).all() for n, h in fine)
    assert moe.moe_device_status() == (moe.MOE_OK, 0)


@pytest.mark.parametrize("gain", [1e-3, 30.0, 1000.0])
def test_score_magnitudes(gain):
    # nearly uniform and nearly one-hot weights
    run_and_check(Case([(700, 5), (3, 2)], 8, 2, 128, 32, seed=9, q_gain=gain))


def test_queries_of_very_different_size():
    c = Case([(300, 8)], 8, 2, 128, 16, seed=10)
    gain = torch.from_numpy(np.exp2(np.linspace(-30, 6, 64)).reshape(8, 8, 1))
    c.q = (c.q.cpu().double() * gain).bfloat16().cuda()
    c.q_host = c.q.cpu().double().numpy()
    run_and_check(c)


def test_value_rows_of_very_different_size():
    c = Case([(600, 4)], 4, 2, 128, 16, seed=11)
    c.pool[3][:] = c.rng.randint(40, 200, c.pool[3].shape)
    run_and_check(c)


def test_a_peak_before_a_long_flat_tail():
    # one row with weight 2^14 times each of 30000 others, at the very first row: the tail keeps its share
    c = Case([(30000, 1)], 1, 1, 128, 64, tree=False, seed=12)
    c.pool[0][:], c.pool[1][:] = 0x38, 127 - 8            # all keys: ones times 2^-8
    c.q = torch.ones_like(c.q)
    c.q_host = c.q.cpu().double().numpy()
    c.scale = float(14 * np.log(2.0) / 0.5)
    page, at = c.row(0, 0)
    c.pool[1][page, 0, at] = 127 - 7                      # twice as large: score higher by 14 ln 2
    run_and_check(c)


def test_offsets_past_32_bits():
    # codes of more than 2^32 bytes: the lane's pages lie at the far end of the pool
    H, page, D = 4, 64, 256
    pages = (1 << 32) // (H * page * D) + 64
    c = Case([(500, 3), (70, 2)], 8, H, D, page, seed=13)
    small = [torch.from_numpy(a).cuda() for a in c.pool]
    n = small[0].shape[0]
    big = [torch.empty((pages, *a.shape[1:]), dtype=torch.uint8, device="cuda") for a in small]
    for a, b in zip(small, big):
        b[-n:] = a
    cache = moe.KvCache(big[0], big[2], big[1], big[3])
    table = torch.from_numpy(np.where(c.table >= 0, c.table + pages - n, -1).astype(np.int32)).cuda()
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    out = torch.empty((c.N, 8, D), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(moe.moe_tree_attention_workspace_bytes(c.N, 8, H, D, 2), dtype=torch.uint8, device="cuda")
    moe.moe_tree_attention(c.q, cache, table, dev(c.kv_len), dev(c.cu), c.max_nodes, dev(c.mask.view(np.int32)), c.scale, out, ws)
    torch.cuda.synchronize()
    c.check(out.double().cpu().numpy())
    # the other calls at the same far rows
    x = torch.randn(3, H, D, device="cuda")
    slots = torch.arange(pages * page - 3, pages * page, device="cuda")
    moe.moe_kv_write(x, -x, slots, cache)
    k, v = torch.empty_like(x), torch.empty_like(x)
    far = torch.tensor([[pages - 1]], dtype=torch.int32, device="cuda")
    moe.moe_kv_read(cache, far, torch.tensor([page - 3], dtype=torch.int32, device="cuda"),
                    torch.tensor([0, 3], dtype=torch.int32, device="cuda"), k, v)
    torch.cuda.synchronize()
    want = ref.values(*ref.quantise(x.cpu().numpy()))
    assert np.array_equal(k.double().cpu().numpy(), want) and np.array_equal(v.double().cpu().numpy(), -want)
    assert moe.moe_device_status() == (moe.MOE_OK, 0)


def test_strided_queries_other_stream_and_the_same_bits_twice():
    c = Case([(3000, 5), (100, 3), (0, 1)], 8, 2, 128, 32, seed=14)
    wide = torch.randn(c.N, 3, 8, 128, device="cuda").bfloat16()
    wide[:, 1] = c.q
    side = torch.cuda.Stream()
    n = moe.moe_tree_attention_workspace_bytes(c.N, 8, 2, 128, 3)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    a, la = c.gpu(q=wide[:, 1], stream=side, workspace=ws)
    c.check(a, la)
    heads_first = c.q.transpose(0, 1).contiguous().transpose(0, 1)
    b, lb = c.gpu(q=heads_first, workspace=ws)
    assert np.array_equal(a, b) and np.array_equal(la, lb)
    no_lse, _ = c.gpu(lse=False)
    assert np.array_equal(a, no_lse)


def test_lanes_that_do_not_fit_their_table():
    c = Case([(100, 3), (200, 2), (50, 1)], 4, 2, 128, 16, seed=15)
    c.kv_len[0] = 2                                        # fewer rows than nodes
    c.kv_len[1] = c.table.shape[1] * 16 + 1                # more rows than the table holds
    got, lse = c.gpu()
    assert moe.moe_device_status() == (moe.MOE_EDEVICE, moe.MOE_DEV_BAD_PAGE)
    assert not got[:5].any() and np.isneginf(lse[:5]).all()
    c.check(got, lse, lanes=[2])


def test_a_page_outside_the_cache_is_reported():
    c = Case([(100, 1), (50, 1)], 4, 2, 128, 16, seed=16)
    c.table[0, 2] = 10_000
    c.table[0, 3] = -5
    got, lse = c.gpu()
    assert moe.moe_device_status() == (moe.MOE_EDEVICE, moe.MOE_DEV_BAD_PAGE)
    c.check(got, lse, lanes=[1])


def test_a_lane_with_more_nodes_than_said():
    c = Case([(40, 5), (20, 2)], 4, 2, 128, 16, tree=False, seed=17)
    c.max_nodes = 4
    got, lse = c.gpu()
    assert moe.moe_device_status() == (moe.MOE_EDEVICE, moe.MOE_DEV_BAD_PAGE)
    assert not got[:5].any() and np.isneginf(lse[:5]).all()
    c.check(got, lse, lanes=[1])
