"""Chunk attention with outputs of more than 2^31 values, and over a cache of more than 2^31 bytes, against 64 bits."""
import numpy as np
import pytest
import torch

from tests import kv_reference as ref

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("resident_expert_routed_gb300")


def test_a_lane_whose_outputs_pass_32_bits():
    """16,500 tokens, 1,024 query heads of 128 to eight kv heads: values 2^31 and on begin at token 16,384. All tokens have the
    same queries (a stride of 0)."""
    n, Hq, H, D, page = 16500, 1024, 8, 128, 128
    rng = np.random.RandomState(3)
    pages = -(-n // page)
    host = []
    for _ in range(2):
        codes, scales = ref.quantise(rng.randn(H, page, D))              # page p holds these rows, turned by p
        at = (np.arange(page)[None, :] + 7 * np.arange(pages)[:, None]) % page
        host += [codes[:, at].transpose(1, 0, 2, 3), scales[:, at].transpose(1, 0, 2)]
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    cache = moe.KvCache(dev(host[0]), dev(host[2]), dev(host[1]), dev(host[3]))
    table = np.arange(pages, dtype=np.int32)[None, :]
    q = torch.from_numpy(rng.randn(1, Hq, D)).bfloat16()
    out = torch.full((n, Hq, D), 9.0, dtype=torch.bfloat16, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = torch.empty(moe.moe_chunk_attention_workspace_bytes(n, Hq, H, D, 1), dtype=torch.uint8, device="cuda")
    moe.moe_chunk_attention(q.cuda().expand(n, Hq, D), cache, dev(table), i32(n), i32(0, n), D ** -0.5, out, ws)
    torch.cuda.synchronize()
    assert moe.moe_device_status() == (moe.MOE_OK, 0)
    assert not any((out[a:a + 500] == 9.0).all(-1).any().item() for a in range(0, n, 500))
    k, v = (ref.lane_rows(ref.values(*host[i:i + 2]), table[0], n) for i in (0, 2))
    for t in (0, 100, 8191, 16383, 16384, 16385, 16499):
        for h in (0, 127, 128, 511, 1023):
            o, _, mass = ref.attention(q[:, h].double().numpy(), k[:t + 1, h // 128], v[:t + 1, h // 128], np.ones((1, t + 1), bool), D ** -0.5)
            got = out[t, h].double().cpu().numpy()
            # the weights' and the output's roundings, 2^-8 each, queries held to 2^-13, steps cut off: n / 16 2^-24
            assert (np.abs(got - o[0]) <= 2.0 ** -8 * np.abs(o[0]) + (2.0 ** -7 + 2.0 ** -13) * mass[0]).all(), (t, h)


def test_a_cache_past_4_gigabytes():
    """Pages at both ends of a pool of 2^32 bytes a side."""
    H, D, page = 4, 256, 1024
    pages = (1 << 32) // (H * page * D) + 3
    codes = [torch.zeros((pages, H, page, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.full((pages, H, page), 127, dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache = moe.KvCache(codes[0], codes[1], scales[0], scales[1])
    rng = np.random.RandomState(5)
    n, ids = 1500, [pages - 1, 0]
    rows = rng.randn(2, n, H, D).astype(np.float32)
    at = np.arange(n)
    slots = torch.from_numpy(np.array(ids)[at // page] * page + at % page).cuda()
    k, v = (torch.from_numpy(x).cuda() for x in rows)
    moe.moe_kv_write(k, v, slots, cache)
    q = torch.from_numpy(rng.randn(30, H, D)).bfloat16().cuda()
    out = torch.empty((30, H, D), dtype=torch.bfloat16, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = torch.empty(moe.moe_chunk_attention_workspace_bytes(30, H, H, D, 1), dtype=torch.uint8, device="cuda")
    moe.moe_chunk_attention(q, cache, i32([ids]), i32([n]), i32([0, 30]), D ** -0.5, out, ws)
    assert moe.moe_device_status() == (moe.MOE_OK, 0)
    for h in range(H):
        kk, vv = (ref.values(*ref.quantise(x[:, h].astype(np.float64))) for x in rows)
        for t in (0, 29):
            p = n - 30 + t
            o, _, mass = ref.attention(q[t:t + 1, h].double().cpu().numpy(), kk[:p + 1], vv[:p + 1], np.ones((1, p + 1), bool), D ** -0.5)
            got = out[t, h].double().cpu().numpy()
            assert (np.abs(got - o[0]) <= 2.0 ** -8 * np.abs(o[0]) + (2.0 ** -7 + 2.0 ** -13) * mass[0]).all(), (t, h)
