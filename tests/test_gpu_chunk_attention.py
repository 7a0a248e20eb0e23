"""Attention of chunks over the paged 8-bit cache on the GPU, against the definition in 64 bits.

The cache's values are exact on both sides. Bounds, u = 2^-24:
  score   a query is held to 2^-17 of the largest of its row, to 2^-13 where smaller rows are handled with it; a sum of D
          products is off by D u of the sum of their sizes; the product with the scale, the difference to the reference and
          the exponential by 8 u of |score| + 8 u: together d, in the exponent
  weight  held to 2^-8 of itself (bf16): an output is off by (2^-8 + 2 d) of sum p |v|, by n / 16 u of that for n rows
          added up (sixteen to a step, cut off, not rounded), and by 2^-8 of itself for its own rounding
  lse     d, and 2^-21 of itself and of one for the sum, the logarithm and the product
"""
import numpy as np
import pytest
import torch

from tests import kv_reference as ref

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("resident_expert_routed_gb300")

U = 2.0 ** -24


class Chunks:
    """Lanes of given (prefix rows, new tokens) over a cache with random rows."""

    def __init__(self, lanes, Hq, Hkv, D, page, seed=0, gain=1.0, spare=2, scale=None):
        rng = self.rng = np.random.RandomState(seed)
        self.lanes, self.Hq, self.Hkv, self.D, self.page = lanes, Hq, Hkv, D, page
        total = [p + n for p, n in lanes]
        need = [-(-t // page) for t in total]
        pages = sum(need) + spare
        self.pool = []
        for _ in range(2):
            x = rng.randn(pages, Hkv, page, D).astype(np.float32) * np.exp(rng.randn(pages, Hkv, page, 1)).astype(np.float32)
            e = np.ceil(np.log2(np.abs(x).max(-1) / 448.0)).astype(int)
            t = torch.from_numpy(np.ldexp(x, -e[..., None])).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
            self.pool += [t, (e + 127).astype(np.uint8)]
        self.table = np.full((len(lanes), max(1, max(need))), -1, np.int32)
        ids = rng.permutation(pages)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        self.spare = ids[at:]
        self.kv_len = np.array(total, np.int32)
        self.cu = np.r_[0, np.cumsum([n for _, n in lanes])].astype(np.int32)
        self.N = int(self.cu[-1])
        self.q = torch.from_numpy(rng.randn(self.N, Hq, D) * gain).bfloat16().cuda()
        self.scale = D ** -0.5 if scale is None else scale

    def at(self, b, j):
        """(page, row) of row j of lane b, to reach into the pool."""
        return self.table[b, j // self.page], j % self.page

    def args(self, tail=0):
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        kc, ks, vc, vs = (dev(a) for a in self.pool)
        out = torch.full((self.N + tail, self.Hq, self.D), 9.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((self.N + tail, self.Hq), 9.0, device="cuda")
        n = moe.moe_chunk_attention_workspace_bytes(self.N + tail, self.Hq, self.Hkv, self.D, len(self.lanes))
        ws = torch.randint(0, 256, (n,), dtype=torch.uint8, device="cuda")
        return moe.KvCache(kc, vc, ks, vs), dev(self.table), dev(self.kv_len), dev(self.cu), out, lse, ws

    def gpu(self, stream=None, with_lse=True):
        cache, table, kv_len, cu, out, lse, ws = self.args()
        torch.cuda.synchronize()
        moe.moe_chunk_attention(self.q, cache, table, kv_len, cu, self.scale, out, ws, lse=lse if with_lse else None, stream=stream)
        torch.cuda.synchronize()
        return out, lse

    def values(self, i, b, h, n):
        codes, scales = (ref.lane_rows(x, self.table[b], n)[:, h] for x in self.pool[i:i + 2])
        return ref.values(codes, scales)

    def check(self, out, lse=None, heads=None, tokens=None, weight=2.0 ** -8):
        """weight: half a step of a weight's rounding; in two parts, half a step of what the first leaves, and twice the sums."""
        G = self.Hq // self.Hkv
        for b, (p, n) in enumerate(self.lanes):
            if not n:
                continue
            which = np.arange(n) if tokens is None or n <= tokens else np.unique(np.r_[0, n - 1, self.rng.randint(0, n, tokens)])
            rows = torch.from_numpy(self.cu[b] + which).cuda()
            for h in range(self.Hq) if heads is None else heads:
                k, v = self.values(0, b, h // G, p + n), self.values(2, b, h // G, p + n)
                q = self.q[rows, h].double().cpu().numpy()
                with np.errstate(all="ignore"):
                    sees = np.arange(p + n) <= p + which[:, None]
                    s = np.where(sees, np.where(sees, q @ k.T, 0.0) * self.scale, -np.inf) if np.isfinite(k).all() and np.isfinite(q).all() else \
                        np.where(sees, np.array([[np.dot(x, y) for y in k] for x in q]) * self.scale, -np.inf)
                    top = s.max(-1, keepdims=True)
                    w = np.exp(s - top)
                    total = w.sum(-1, keepdims=True)
                    w /= total
                    clean = np.where(np.isfinite(v), v, 0.0)
                    o = w @ clean
                    seen_nan = (sees @ (~np.isfinite(v)).astype(float)) > 0
                    o = np.where(seen_nan | np.isnan(o), np.nan, o)
                    mass = w @ np.abs(clean)
                    e = (top + np.log(total))[:, 0]
                    mags = np.abs(q) @ np.nan_to_num(np.abs(k)).T * self.scale
                    mags = np.where(sees, mags, 0.0).max(-1)
                    held = self.scale * 2.0 ** -13 * np.abs(q).max(-1) * np.nan_to_num(np.abs(k)).sum(-1).max()
                    d = held + (self.D + 8) * U * mags + 8 * U
                got = out[rows, h].double().cpu().numpy()
                assert np.array_equal(np.isnan(got), np.isnan(o)), (b, h)
                tol = 2.0 ** -8 * np.abs(o) + (weight + 2 * d[:, None] + (p + n) / 16 * U * (1 if weight == 2.0 ** -8 else 2)) * mass * (1 + 2.0 ** -6) + 1e-30
                off = np.abs(got - o)
                fine = ~np.isnan(o)
                assert (off[fine] <= tol[fine]).all(), (b, h, np.nanmax(off / tol))
                if lse is not None:
                    x = lse[rows, h].double().cpu().numpy()
                    assert np.array_equal(np.isnan(x), np.isnan(e))
                    ok = np.isfinite(e)
                    assert (np.abs(x - e)[ok] <= (d + 2.0 ** -21 * (1 + np.abs(e)))[ok]).all(), (b, h, np.abs(x - e)[ok].max())


def run_and_check(c, status=(0, 0), **kw):
    out, lse = c.gpu()
    assert moe.moe_device_status() == status
    c.check(out, lse, **kw)
    return out, lse


@pytest.mark.parametrize("D,page", [(64, 16), (128, 64), (256, 32)])
@pytest.mark.parametrize("n", [1, 2, 15, 31, 32, 33, 63, 64, 65, 127, 128, 129, 257, 513])
def test_prompts(n, D, page):
    run_and_check(Chunks([(0, n)], 4, 2, D, page, seed=n))


@pytest.mark.parametrize("D,page", [(64, 64), (128, 16), (256, 128)])
@pytest.mark.parametrize("prefix", [1, 63, 127, 128, 129, 1000])
@pytest.mark.parametrize("n", [1, 33, 130])
def test_prefixes(prefix, n, D, page):
    run_and_check(Chunks([(prefix, n)], 4, 1, D, page, seed=prefix + n))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (6, 2), (5, 1), (16, 1), (40, 8), (24, 1), (64, 8), (100, 1), (128, 1)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_head_layouts(Hq, Hkv, D):
    run_and_check(Chunks([(150, 40), (3, 1), (0, 70)], Hq, Hkv, D, 16, seed=Hq), heads=sorted({0, Hq // 2, Hq - 1}))


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256, 1024])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_pages(page, D):
    run_and_check(Chunks([(77, 200), (0, 130), (1030, 5)], 4, 2, D, page, seed=page))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_mixed_batches(D):
    lanes = [(300, 1), (0, 257), (0, 0), (4000, 1), (1, 1), (515, 77), (0, 1), (0, 0), (2000, 300), (127, 1), (128, 1), (129, 1)]
    run_and_check(Chunks(lanes, 8, 2, D, 32, seed=D), heads=[0, 3, 7], tokens=40)


def test_many_lanes():
    lanes = [((37 * i) % 400, (11 * i) % 7) for i in range(900)]
    run_and_check(Chunks(lanes, 2, 1, 64, 16, seed=4))


def test_one_token_in_each_of_4096_lanes():
    run_and_check(Chunks([(i % 50, 1) for i in range(4096)], 1, 1, 64, 16, seed=5))


def test_waiting_lanes_around_one_that_does_not():
    run_and_check(Chunks([(0, 0)] * 700 + [(90, 45)] + [(5, 0)] * 700, 4, 2, 64, 16, seed=6))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_long_prefix(D):
    """Cut between many blocks and joined; few rows and a full block of them."""
    run_and_check(Chunks([(40000, 3)], 4, 2, D, 64, seed=1), heads=[0, 3])
    run_and_check(Chunks([(30000, 140)], 4, 2, D, 128, seed=2), heads=[1, 2], tokens=30)


@pytest.mark.parametrize("D,page", [(64, 16), (128, 64), (256, 128)])
def test_units_of_one_row_tile_and_of_two_beside_one_another(D, page):
    """Several units a block, of one tile of cache rows and of more, odd and even numbers of them."""
    lanes = [((53 * i) % 700, (1, 70, 33, 140, 2, 129, 0, 64)[(3 * i + i // 8) % 8]) for i in range(150)]
    run_and_check(Chunks(lanes, 8, 2, D, page, seed=24), heads=[0, 7], tokens=4)


@pytest.mark.parametrize("lanes", [[(0, 1024)] * 3, [(0, 900)] * 4, [(0, 640)] * 5, [(0, 1024)] * 2])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_several_prompts(lanes, D):
    """Of five to eight tiles, more and fewer units than twice the SMs: cut and not cut."""
    run_and_check(Chunks(lanes, 32, 8, D, 128, seed=25), heads=[0, 13, 31], tokens=6)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lanes,Hq,Hkv", [([(5000, 1)] * 30, 2, 2), ([(9000, 1), (70, 3), (0, 2)], 32, 8), ([(300, 100)], 8, 2), ([(0, 1024)], 1, 1),
                                          ([(1500, 200)], 5, 1)])
def test_few_rows_hold_their_weights_in_two_parts(lanes, Hq, Hkv, D):
    run_and_check(Chunks(lanes, Hq, Hkv, D, 64, seed=26), weight=2.0 ** -16)


def test_a_whole_prompt():
    run_and_check(Chunks([(0, 3000)], 8, 2, 128, 64, seed=3), heads=[0, 5], tokens=200)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("gain", [2.0 ** -30, 0.02, 30.0])
def test_scores_small_and_large(D, gain):
    """Nearly equal weights, and a few that hold all: the running reference moves again and again."""
    run_and_check(Chunks([(700, 150)], 4, 2, D, 64, seed=7, gain=gain))


def test_scores_that_grow_along_the_lane():
    """Each tile's scores pass the reference of those before it."""
    c = Chunks([(1500, 120)], 2, 1, 128, 64, seed=8)
    c.q = c.q.abs() + 0.5
    for j in range(1620):
        page, row = c.at(0, j)
        c.pool[0][page, 0, row] &= 0x7F
        c.pool[1][page, 0, row] = 115 + j // 128
    run_and_check(c)
    for j in range(1620):
        page, row = c.at(0, j)
        c.pool[1][page, 0, row] = 115 + (1619 - j) // 128
    run_and_check(c)


def test_rows_of_queries_far_apart_in_size():
    c = Chunks([(300, 130)], 4, 2, 128, 64, seed=9)
    f = torch.exp2(torch.from_numpy(c.rng.randint(-60, 4, (130, 4, 1)).astype(np.float32))).cuda()
    c.q = (c.q.float() * f).bfloat16()
    c.q[5], c.q[77, 2] = 0.0, 0.0
    run_and_check(c)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_values_far_apart_in_size(D):
    c = Chunks([(500, 140)], 2, 1, D, 16, seed=10)
    c.pool[3][...] = (127 + c.rng.randint(-90, 90, c.pool[3].shape)).astype(np.uint8)
    out, lse = run_and_check(c)
    c.pool[3][...] = 27 + 2                                    # the smallest vectors, but for zeros
    run_and_check(c)


def test_zero_vectors_and_zero_queries():
    c = Chunks([(200, 70)], 4, 2, 64, 16, seed=11)
    c.pool[0][::2] = 0
    c.pool[1][::2] = 127
    c.pool[2][1::2] = 0
    c.pool[3][1::2] = 127
    c.q[10:20] = 0
    run_and_check(c)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_rows_that_nobody_sees_hold_anything(D):
    """NaN vectors, NaN codes, codes of any kind behind a lane's rows and in other lanes' pages."""
    c = Chunks([(100, 61), (0, 190), (30, 1)], 4, 2, D, 64, seed=12)
    want = c.gpu()
    for x in range(4):
        c.pool[x][c.spare] = 255
    for b, (p, n) in enumerate(c.lanes):
        for j in range(p + n, -(-(p + n) // 64) * 64):
            page, row = c.at(b, j)
            c.pool[0][page, :, row] = c.pool[2][page, :, row] = 0x7F if j % 2 else 0xFF
            c.pool[1][page, :, row] = c.pool[3][page, :, row] = 255 if j % 3 else 254
    got = c.gpu()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    c.check(*got)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_vector_that_is_not_finite_reaches_those_that_see_it_and_nobody_else(D):
    for side, at in ((1, 150), (3, 150), (1, 0), (3, 299)):
        c = Chunks([(120, 180)], 4, 2, D, 64, seed=13)
        want = c.gpu()[0]
        page, row = c.at(0, at)
        c.pool[side - 1][page, 1, row] = 0
        c.pool[side][page, 1, row] = 255
        out, lse = c.gpu()
        first = max(0, at - 120)
        assert torch.isnan(out[first:, 2:]).all()
        assert torch.equal(out[:first], want[:first]) and torch.equal(out[:, :2], want[:, :2])
        assert moe.moe_device_status() == (0, 0)


def test_queries_that_are_not_finite_stay_in_their_row():
    c = Chunks([(100, 90)], 4, 2, 128, 64, seed=14)
    want = c.gpu()[0]
    c.q[7, 1, 5], c.q[80, 3, 0] = float("nan"), float("inf")
    out, _ = c.gpu()
    bad = ~torch.isfinite(out).all(-1)
    assert bad.nonzero().tolist() == [[7, 1], [80, 3]]
    # the others share a factor with the largest of their block or have their own: equal up to the query's holding
    assert ((out - want).abs()[~bad].double() <= 2.0 ** -6 * want.abs().max().double()).all()


def test_rows_of_q_and_out_behind_the_last_lane_stay():
    c = Chunks([(40, 33), (0, 10)], 4, 2, 64, 16, seed=15)
    cache, table, kv_len, cu, out, lse, ws = c.args(tail=50)
    q = torch.cat([c.q, torch.full((50, 4, 64), float("nan"), dtype=torch.bfloat16, device="cuda")])
    moe.moe_chunk_attention(q, cache, table, kv_len, cu, c.scale, out, ws, lse=lse)
    assert moe.moe_device_status() == (0, 0)
    c.check(out, lse)
    assert (out[c.N:] == 9).all() and (lse[c.N:] == 9).all()


def test_strided_queries():
    c = Chunks([(100, 50)], 8, 2, 128, 64, seed=16)
    wide = torch.full((50, 12, 136), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 2:10, :128] = c.q
    want = c.gpu()[0]
    c.q = wide[:, 2:10, :128]
    assert torch.equal(c.gpu()[0], want)


def test_lanes_that_do_not_fit_get_zeros_and_are_told():
    c = Chunks([(100, 50), (20, 30), (60, 10)], 4, 2, 64, 16, seed=17)
    want = c.gpu()[0]
    for bad in (29, 16 * c.table.shape[1] + 1, -3, 2 ** 31 - 1):
        c.kv_len[1] = bad
        out, lse = c.gpu()
        assert moe.moe_device_status() == (moe.MOE_EDEVICE, moe.MOE_DEV_BAD_PAGE)
        assert (out[50:80] == 0).all() and torch.isneginf(lse[50:80]).all()
        assert torch.equal(out[:50], want[:50]) and torch.equal(out[80:], want[80:])


def test_bad_sums_of_tokens_lead_nowhere():
    c = Chunks([(100, 50), (20, 30), (60, 10)], 4, 2, 64, 16, seed=18)
    want = c.gpu()[0]
    for cu in ([0, 50, 2 ** 30, 90], [0, 50, -7, 90], [0, 50, 91, 90]):
        c.cu = np.array(cu, np.int32)
        out, _ = c.gpu()
        assert moe.moe_device_status() == (moe.MOE_EDEVICE, moe.MOE_DEV_BAD_PAGE)
        assert torch.equal(out[:50], want[:50])


def test_page_ids_outside_the_cache_are_told():
    c = Chunks([(100, 50)], 4, 2, 64, 16, seed=19)
    t = c.table.copy()
    for bad in (-1, 10 ** 6):
        c.table[0, 2] = bad
        c.gpu()
        assert moe.moe_device_status() == (moe.MOE_EDEVICE, moe.MOE_DEV_BAD_PAGE)
        c.table = t.copy()
    run_and_check(c)


def test_same_bits_again_and_without_lse():
    c = Chunks([(5000, 70), (0, 700), (9000, 1)], 8, 2, 128, 64, seed=20)
    a, l = c.gpu()
    for _ in range(3):
        b, m = c.gpu()
        assert torch.equal(a, b) and torch.equal(l, m)
    assert torch.equal(c.gpu(with_lse=False)[0], a)


def test_captured_replayed_and_two_at_once():
    """Two streams with a workspace each; a captured call whose inputs change between replays."""
    c, d = Chunks([(3000, 70), (0, 300)], 8, 2, 128, 64, seed=21), Chunks([(0, 500), (700, 1)], 4, 4, 64, 16, seed=22)
    want = [x.gpu()[0] for x in (c, d)]
    sets = [x.args() for x in (c, d)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for x, (cache, table, kv_len, cu, out, lse, ws), s in zip((c, d), sets, streams):
            moe.moe_chunk_attention(x.q, cache, table, kv_len, cu, x.scale, out, ws, lse=lse, stream=s)
    torch.cuda.synchronize()
    for w, s in zip(want, sets):
        assert torch.equal(s[4], w)
    cache, table, kv_len, cu, out, lse, ws = sets[0]
    graph = torch.cuda.CUDAGraph()
    q = c.q.clone()
    with torch.cuda.graph(graph):
        moe.moe_chunk_attention(q, cache, table, kv_len, cu, c.scale, out, ws, lse=lse)
    for lens in ([(3000, 70), (0, 300)], [(2950, 120), (50, 250)]):
        e = Chunks([(3000, 70), (0, 300)], 8, 2, 128, 64, seed=21)
        e.lanes, e.kv_len = lens, np.array([p + n for p, n in lens], np.int32)
        e.cu = np.r_[0, np.cumsum([n for _, n in lens])].astype(np.int32)
        kv_len.copy_(torch.from_numpy(e.kv_len))
        cu.copy_(torch.from_numpy(e.cu))
        graph.replay()
        torch.cuda.synchronize()
        e.check(out, lse, heads=[0, 7], tokens=40)
    assert moe.moe_device_status() == (0, 0)


def test_refusals():
    c = Chunks([(10, 5)], 4, 2, 64, 16)
    cache, table, kv_len, cu, out, lse, ws = c.args()
    good = dict(q=c.q, cache=cache, page_table=table, kv_len=kv_len, cu_tokens=cu, scale=c.scale, out=out, workspace=ws, lse=lse)
    for bad in (dict(q=c.q.float()), dict(q=c.q[..., ::2]), dict(q=c.q[0]), dict(page_table=table.long()), dict(kv_len=kv_len[:0]),
                dict(cu_tokens=cu[:1]), dict(out=out.float()), dict(out=out[:, :2]), dict(lse=lse.double()), dict(workspace=ws.cpu())):
        with pytest.raises(ValueError):
            moe.moe_chunk_attention(**(good | bad))
    with pytest.raises(moe.MoeError) as e:
        moe.moe_chunk_attention(**(good | dict(workspace=ws[:0])))
    assert e.value.status in (moe.MOE_ENOMEM, moe.MOE_EINVAL)
    moe.moe_chunk_attention(c.q[:0], cache, table, kv_len, cu, c.scale, out[:0], ws)
