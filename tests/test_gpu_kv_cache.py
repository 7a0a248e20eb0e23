"""The paged 8-bit key/value cache on the GPU (write, read, keep) against the 64-bit definition.

Quantising is a division by a power of two and one rounding, reading back an
exact product: codes, scales and values have to be equal, bit for bit.
"""
import numpy as np
import pytest
import torch

from tests import kv_reference as ref

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("resident_expert_routed_gb300")

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def pool(pages, H, page, D, seed=0):
    """A cache with rows in it, and its bytes on the host."""
    rng = np.random.RandomState(seed)
    host = []
    for _ in range(2):
        codes = rng.randint(0, 256, (pages, H, page, D)).astype(np.uint8)
        codes[(codes & 0x7F) == 0x7F] = 0x11
        host += [codes, rng.randint(110, 140, (pages, H, page)).astype(np.uint8)]
    kc, ks, vc, vs = host
    return moe.KvCache(*(torch.from_numpy(a.copy()).cuda() for a in (kc, vc, ks, vs))), (kc, vc, ks, vs)


def held(cache):
    torch.cuda.synchronize()
    return [t.cpu().numpy() for t in (cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales)]


def ok_status():
    assert moe.moe_device_status() == (moe.MOE_OK, 0)


def put(bytes_, x, slots, which):
    """The reference's write of x [T, H, D] into the host copy."""
    codes, scales = ref.quantise(x)
    page = bytes_[0].shape[2]
    for t, s in enumerate(slots):
        if s >= 0:
            bytes_[which][s // page, :, s % page] = codes[t]
            bytes_[2 + which][s // page, :, s % page] = scales[t]


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("T,H,page,D", [(1, 1, 16, 64), (3, 5, 16, 64), (33, 3, 64, 128), (7, 2, 32, 256), (130, 8, 128, 128), (1, 40, 1024, 256)])
def test_write_is_the_definition(T, H, page, D, dtype):
    cache, bytes_ = pool(-(-T // page) + 2, H, page, D)
    rng = np.random.RandomState(T * D)
    kv = torch.from_numpy(rng.randn(T, 2 * H * D) * np.exp(3 * rng.randn(T, 1))).to(TYPES[dtype]).cuda()
    k, v = kv[:, :H * D].view(T, H, D), kv[:, H * D:].view(T, H, D)
    slots = rng.permutation(cache.n_pages * page)[:T].astype(np.int64)
    if T > 2:
        slots[2] = -1
    moe.moe_kv_write(k, v, torch.from_numpy(slots).cuda(), cache)
    put(bytes_, k.double().cpu().numpy(), slots, 0)
    put(bytes_, v.double().cpu().numpy(), slots, 1)
    for got, want in zip(held(cache), bytes_):
        assert np.array_equal(got, want)                 # the rest of the cache as it was
    ok_status()


def test_write_of_hard_values():
    # ties between codes, the step from 448 to the next scale, zeros, subnormals, the largest and smallest vectors
    D, H = 64, 1
    rows = [np.zeros(D), np.full(D, 448.0), np.full(D, 448.0001), np.full(D, 2.0 ** -149), np.full(D, 2.0 ** 127),
            np.full(D, 1.6e38), np.linspace(-448, 448, D), np.r_[448.0, np.arange(1, D) * 2.0 ** -10],
            np.r_[448.0, (np.arange(1, D) + 0.5) * 2.0 ** -9], np.r_[256.0, 17 + np.arange(1, D) / 2.0],
            -np.r_[1.75, 1.0625 + np.arange(1, D) / 128.0], np.full(D, 2.0 ** -95), np.r_[1.0, np.full(D - 1, 2.0 ** -30)]]
    x = np.stack(rows).astype(np.float32)[:, None, :]
    T = len(rows)
    cache, bytes_ = pool(2, H, 16, D)
    moe.moe_kv_write(torch.from_numpy(x).cuda(), torch.from_numpy(-x).cuda(), torch.arange(T, device="cuda"), cache)
    put(bytes_, x, range(T), 0)
    put(bytes_, -x, range(T), 1)
    for got, want in zip(held(cache), bytes_):
        assert np.array_equal(got, want)
    ok_status()


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_write_of_a_vector_that_is_not_finite(bad, dtype):
    T, H, D = 5, 3, 128
    rng = np.random.RandomState(4)
    k, v = rng.randn(T, H, D), rng.randn(T, H, D)
    k[1, 2, 127] = bad
    v[4, 0, 0] = bad
    kt, vt = (torch.from_numpy(a).to(TYPES[dtype]).cuda() for a in (k, v))
    cache, bytes_ = pool(1, H, 16, D)
    moe.moe_kv_write(kt, vt, torch.arange(T, device="cuda"), cache)
    put(bytes_, kt.double().cpu().numpy(), range(T), 0)
    put(bytes_, vt.double().cpu().numpy(), range(T), 1)
    got = held(cache)
    for a, b in zip(got, bytes_):
        assert np.array_equal(a, b)
    assert got[2][0, 2, 1] == 255 and not got[0][0, 2, 1].any()
    assert moe.moe_device_status() == (moe.MOE_EDEVICE, moe.MOE_DEV_NAN_KV)


def test_write_skips_slots_outside_the_cache():
    cache, bytes_ = pool(2, 2, 16, 64)
    x = torch.randn(4, 2, 64, device="cuda")
    slots = [5, 32, -1, -7]
    moe.moe_kv_write(x, x, torch.tensor(slots, device="cuda"), cache)
    put(bytes_, x.double().cpu().numpy()[:1], slots[:1], 0)
    put(bytes_, x.double().cpu().numpy()[:1], slots[:1], 1)
    for got, want in zip(held(cache), bytes_):
        assert np.array_equal(got, want)
    assert moe.moe_device_status() == (moe.MOE_EDEVICE, moe.MOE_DEV_BAD_PAGE)


def test_write_with_other_strides():
    # heads before tokens, and a projection row with a gap between the heads
    H, D, T = 3, 64, 9
    k = torch.randn(H, T, D, device="cuda").transpose(0, 1)
    v = torch.randn(T, H, 2 * D, device="cuda")[:, :, D:]
    cache, bytes_ = pool(1, H, 16, D)
    moe.moe_kv_write(k, v, torch.arange(T, device="cuda"), cache)
    put(bytes_, k.double().cpu().numpy(), range(T), 0)
    put(bytes_, v.double().cpu().numpy(), range(T), 1)
    for got, want in zip(held(cache), bytes_):
        assert np.array_equal(got, want)


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("lens,H,page,D", [([1], 1, 16, 64), ([0, 17, 0, 1, 40], 3, 16, 64), ([129, 5], 8, 64, 128), ([31, 33], 2, 32, 256)])
def test_read_is_the_definition(lens, H, page, D, dtype):
    rng = np.random.RandomState(len(lens) + D)
    starts = [3 * i for i in range(len(lens))]
    need = [-(-(n + s) // page) for n, s in zip(lens, starts)]
    cache, (kc, vc, ks, vs) = pool(sum(need) + 1, H, page, D, seed=5)
    ids = rng.permutation(cache.n_pages).astype(np.int32)
    table = np.full((len(lens), max(need) + 1), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    cu = np.r_[0, np.cumsum(lens)].astype(np.int32)
    n = int(cu[-1])
    k, v = (torch.full((n, H, D), 7.0, dtype=TYPES[dtype], device="cuda") for _ in range(2))
    moe.moe_kv_read(cache, torch.from_numpy(table).cuda(), torch.tensor(starts, dtype=torch.int32, device="cuda"),
                    torch.from_numpy(cu).cuda(), k, v)
    torch.cuda.synchronize()
    for got, codes, scales in ((k, kc, ks), (v, vc, vs)):
        want = np.concatenate([ref.lane_rows(ref.values(codes, scales), table[b], starts[b] + m)[starts[b]:]
                               for b, m in enumerate(lens)])
        want = torch.from_numpy(want).to(TYPES[dtype]).double().numpy()      # one rounding, where fp16 needs it
        assert np.array_equal(got.double().cpu().numpy(), want)
    ok_status()


def test_read_of_nan_vectors_and_bad_pages():
    H, page, D = 2, 16, 64
    cache, _ = pool(3, H, page, D)
    x = torch.randn(16, H, D, device="cuda")
    x[3, 1, 5] = float("inf")
    moe.moe_kv_write(x, x, torch.arange(16, device="cuda"), cache)
    moe.moe_device_status()
    table = torch.tensor([[0, 3], [-1, 1]], dtype=torch.int32, device="cuda")       # page 3 is outside
    cu = torch.tensor([0, 20, 40], dtype=torch.int32, device="cuda")
    k, v = (torch.zeros((40, H, D), device="cuda") for _ in range(2))
    moe.moe_kv_read(cache, table, None, cu, k, v)
    torch.cuda.synchronize()
    for o in (k, v):
        nan = torch.isnan(o)
        assert nan[3, 1].all() and not nan[3, 0].any() and not nan[:3].any() and not nan[4:16].any()
        assert nan[16:36].all() and not nan[36:].any()
    assert moe.moe_device_status() == (moe.MOE_EDEVICE, moe.MOE_DEV_BAD_PAGE)


@pytest.mark.parametrize("lanes,nodes,H,page,D", [(1, 1, 1, 16, 64), (4, 8, 3, 16, 64), (3, 70, 2, 32, 128), (2, 200, 1, 16, 256), (9, 5, 8, 128, 128)])
def test_keep_moves_the_path(lanes, nodes, H, page, D):
    rng = np.random.RandomState(nodes)
    prefix = rng.randint(0, 40, lanes).astype(np.int32)
    need = [-(-(p + nodes) // page) for p in prefix]
    cache, bytes_ = pool(sum(need), H, page, D, seed=nodes)
    table = np.full((lanes, max(need)), -1, np.int32)
    ids = rng.permutation(sum(need))
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    keep = rng.randint(0, nodes + 1, lanes).astype(np.int32)
    keep[0] = nodes if lanes == 1 else max(1, nodes - 1)
    path = np.full((lanes, nodes), -1, np.int32)
    want = [a.copy() for a in bytes_]
    for b in range(lanes):
        path[b, :keep[b]] = np.sort(rng.permutation(nodes)[:keep[b]])
        for i in range(keep[b]):
            s, d = prefix[b] + path[b, i], prefix[b] + i
            for new, old in zip(want, bytes_):
                new[table[b, d // page], :, d % page] = old[table[b, s // page], :, s % page]
    dev = [torch.from_numpy(a).cuda() for a in (table, prefix, path, keep)]
    moe.moe_kv_keep(cache, *dev)
    for got, w in zip(held(cache), want):
        assert np.array_equal(got, w)
    ok_status()


@pytest.mark.parametrize("path,n", [([1, 1], 2), ([2, 0], 2), ([-1, 3], 2), ([0, 40], 2), ([0, 1], 3)])
def test_keep_leaves_a_lane_with_a_bad_path_alone(path, n):
    cache, bytes_ = pool(4, 2, 16, 64)
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
    want = [a.copy() for a in bytes_]
    for w, old in zip(want, bytes_):
        w[2, :, 3] = old[2, :, 4]                       # the other lane: row 3 + 1 to row 3
    dev = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    moe.moe_kv_keep(cache, table, dev([3, 3]), dev([path, [1, -1]]), dev([n, 1]))
    for got, w in zip(held(cache), want):
        assert np.array_equal(got, w)
    assert moe.moe_device_status() == (moe.MOE_EDEVICE, moe.MOE_DEV_BAD_PAGE)


def test_cache_calls_on_another_stream():
    H, page, D, T = 4, 16, 128, 50
    cache, bytes_ = pool(8, H, page, D)
    side = torch.cuda.Stream()
    x = torch.randn(T, H, D, device="cuda")
    torch.cuda.synchronize()
    out = [torch.empty((T, H, D), device="cuda") for _ in range(2)]
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(1, 8)
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    slots = torch.arange(T, device="cuda")
    torch.cuda.synchronize()
    moe.moe_kv_write(x, -x, slots, cache, stream=side)
    moe.moe_kv_read(cache, table, None, cu, *out, stream=side)
    side.synchronize()
    codes, scales = ref.quantise(x.cpu().numpy())
    assert np.array_equal(out[0].double().cpu().numpy(), ref.values(codes, scales))
    assert torch.equal(out[0], -out[1])
