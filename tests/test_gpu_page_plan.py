"""The plan of a batch of new tokens on the GPU against one lane after the other on the host: whole numbers, all equal."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("resident_expert_routed_gb300")


def host_plan(new, rows, held, table, free, n_free, page, T):
    """The header's rules, one lane after the other."""
    rows, held, table, free = rows.copy(), held.copy(), table.copy(), free.copy()
    refused = False
    for b, n in enumerate(new):
        if n < 0:
            for p in range(held[b]):
                free[n_free] = table[b, p]
                n_free += 1
            table[b, :held[b]] = -1
            rows[b] = held[b] = 0
    there, asked = n_free, 0
    kv_len, cu = np.zeros(len(new), np.int32), np.zeros(len(new) + 1, np.int64)
    positions, slots = np.zeros(T, np.int32), np.full(T, -1, np.int64)
    for b, n in enumerate(new):
        n = max(int(n), 0)
        cu[b + 1] = cu[b] + n
        pages = -(-(int(rows[b]) + n) // page)
        fits = pages <= table.shape[1] and cu[b + 1] <= T
        need = max(0, pages - held[b]) if fits and n else 0
        asked += need
        served = n == 0 or (fits and (need == 0 or asked <= there))
        refused |= not served
        if served:
            for _ in range(need):
                n_free -= 1
                table[b, held[b]] = free[n_free]
                held[b] += 1
            kv_len[b] = rows[b] + n
        for t in range(cu[b], min(T, cu[b + 1])):
            at = rows[b] + t - cu[b]
            positions[t] = at
            if served:
                slots[t] = table[b, at // page] * page + at % page
    return dict(rows=rows, held=held, table=table, free=free, n_free=np.array([n_free], np.int32), kv_len=kv_len,
                cu=np.minimum(cu, T).astype(np.int32), positions=positions, slots=slots), refused


class State:
    def __init__(self, lanes, width, n_pages, page, seed=0, most=None):
        rng = self.rng = np.random.RandomState(seed)
        self.page = page
        self.held = np.minimum(rng.randint(0, width + 1, lanes), most if most is not None else width).astype(np.int32)
        ids = rng.permutation(n_pages).astype(np.int32)
        self.table = np.full((lanes, width), -1, np.int32)
        at = 0
        for b in range(lanes):
            self.held[b] = min(self.held[b], n_pages - at)
            self.table[b, :self.held[b]] = ids[at:at + self.held[b]]
            at += self.held[b]
        self.free = np.full(n_pages, -7, np.int32)
        self.free[:n_pages - at] = ids[at:]
        self.n_free = n_pages - at
        # some lanes hold pages that their rows have not reached
        self.rows = np.array([rng.randint(0, h * page + 1) for h in self.held], np.int32)

    def gpu(self, new, T, stream=None):
        dev = lambda a: torch.from_numpy(np.array(a)).cuda()  # noqa: E731
        s = dict(rows=dev(self.rows), held=dev(self.held), table=dev(self.table), free=dev(self.free), n_free=dev(np.array([self.n_free], np.int32)))
        s |= dict(kv_len=torch.full((len(new),), 99, dtype=torch.int32, device="cuda"), cu=torch.full((len(new) + 1,), 99, dtype=torch.int32, device="cuda"),
                  positions=torch.full((T,), 99, dtype=torch.int32, device="cuda"), slots=torch.full((T,), 99, dtype=torch.int64, device="cuda"))
        s["new"] = dev(np.asarray(new, np.int32))
        torch.cuda.synchronize()
        self.call(s, stream)
        torch.cuda.synchronize()
        return s

    def call(self, s, stream=None):
        moe.moe_page_plan(s["new"], s["rows"], s["held"], s["table"], s["free"], s["n_free"], self.page, s["kv_len"], s["cu"], s["positions"],
                          s["slots"], stream=stream)

    def check(self, new, T):
        want, refused = host_plan(np.asarray(new), self.rows, self.held, self.table, self.free, self.n_free, self.page, T)
        s = self.gpu(new, T)
        for name, w in want.items():
            got = s[name].cpu().numpy()
            assert np.array_equal(got, w), (name, got, w)
        st = moe.moe_device_status()
        assert st == ((moe.MOE_EDEVICE, moe.MOE_DEV_NO_PAGES) if refused else (moe.MOE_OK, 0))
        return s, want


@pytest.mark.parametrize("lanes", [1, 2, 31, 33, 257, 1024, 1025, 4096])
@pytest.mark.parametrize("page", [16, 64, 1024])
def test_plans(lanes, page):
    s = State(lanes, 9, lanes * 9 + 3, page, seed=lanes + page, most=6)
    rng = s.rng
    new = rng.randint(0, 2 * page, lanes)
    new[rng.rand(lanes) < 0.2] = -1
    s.check(new, int(np.maximum(new, 0).sum()) + 5)


@pytest.mark.parametrize("lanes,n_pages,seed", [(7, 20, 0), (50, 60, 1), (300, 700, 2), (2000, 3000, 3)])
def test_pools_that_run_out(lanes, n_pages, seed):
    s = State(lanes, 8, n_pages, 16, seed=seed, most=n_pages // lanes)
    rng = s.rng
    new = rng.randint(0, 60, lanes)
    new[rng.rand(lanes) < 0.15] = -3
    s.check(new, int(np.maximum(new, 0).sum()))


@pytest.mark.parametrize("T", [0, 1, 40, 99])
def test_batches_too_small_and_tables_too_narrow(T):
    s = State(6, 3, 40, 16, seed=T, most=2)
    s.check([10, 48, 0, 30, 200, 12], T)


def test_the_largest_batch_and_one_long_lane():
    s = State(3, 8300, 9000, 16, seed=5, most=8)
    s.check([1, 131072, 0], 131080)


def test_nothing_new_and_nothing_held():
    s = State(5, 4, 10, 32, seed=1, most=0)
    s.check([0, 0, 0, 0, 0], 8)
    s.check([-1, -1, -1, -1, -1], 8)
    s.check([-1, 1, -1, 0, 33], 40)


def test_calling_again_gives_the_same_and_pages_go_round():
    """A serving loop against the host's: plan, move the rows on, plan again, with lanes that end and begin."""
    s = State(12, 20, 120, 16, seed=9, most=4)
    T = 400
    for step in range(12):
        new = s.rng.randint(0, 40, 12)
        new[s.rng.rand(12) < 0.25] = -1
        got, want = s.check(new, T)
        s.call(got)
        torch.cuda.synchronize()
        moe.moe_device_status()
        for name in ("rows", "held", "table", "n_free", "kv_len", "cu", "positions", "slots"):
            assert np.array_equal(got[name].cpu().numpy(), want[name]), name
        ids = np.concatenate([want["table"][want["table"] >= 0], want["free"][:want["n_free"][0]]])
        assert sorted(ids) == list(range(120))
        s.held, s.table, s.free, s.n_free = want["held"], want["table"], want["free"], int(want["n_free"][0])
        s.rows = np.where(want["kv_len"] > 0, want["kv_len"], want["rows"]).astype(np.int32)


def test_bad_states_are_refused_and_told():
    s = State(4, 4, 20, 16, seed=2, most=2)
    s.rows[1], s.held[2] = -5, 9
    got = s.gpu([3, 3, 3, 3], 12)
    assert moe.moe_device_status() == (moe.MOE_EDEVICE, moe.MOE_DEV_BAD_PAGE | moe.MOE_DEV_NO_PAGES)
    kv, slots = got["kv_len"].tolist(), got["slots"].tolist()
    assert kv[0] == s.rows[0] + 3 and kv[1] == 0 and kv[2] == 0 and kv[3] == s.rows[3] + 3
    assert slots[3:9] == [-1] * 6 and min(slots[:3] + slots[9:]) >= 0
    for n_free in (-2, 21):
        s = State(2, 4, 20, 16, seed=3, most=1)
        s.n_free = n_free
        s.gpu([1, 1], 2)
        assert moe.moe_device_status()[1] & moe.MOE_DEV_BAD_PAGE
    s = State(2, 4, 20, 16, seed=4, most=3)
    s.held[:], s.rows[:] = 2, 20
    s.table[0, :2] = [3, 25]                                  # an id outside the pool: its rows get no slot
    got = s.gpu([2, 2], 4)
    assert moe.moe_device_status()[1] == moe.MOE_DEV_BAD_PAGE and got["slots"].tolist()[:2] == [-1, -1]


def test_captured_on_a_side_stream():
    s = State(9, 6, 60, 16, seed=6, most=3)
    new = [4, 0, 20, 1, -1, 33, 2, 0, 16]
    want, _ = host_plan(np.asarray(new), s.rows, s.held, s.table, s.free, s.n_free, 16, 80)
    got = s.gpu(new, 80)
    start = {k: torch.from_numpy(np.array(v)).cuda() for k, v in dict(rows=s.rows, held=s.held, table=s.table, free=s.free, n_free=[s.n_free]).items()}
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        s.call(got)
    for _ in range(2):
        for k, v in start.items():
            got[k].copy_(v)
        got["slots"].fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        for name, w in want.items():
            assert np.array_equal(got[name].cpu().numpy(), w), name
    assert moe.moe_device_status() == (moe.MOE_OK, 0)
