"""Tree attention with outputs of more than 2^31 values in one lane, against the definition in 64 bits."""
import numpy as np
import pytest
import torch

from tests import kv_reference as ref

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("resident_expert_routed_gb300")


def test_a_lane_whose_outputs_pass_32_bits():
    """One chunk of 16,500 nodes and 1,024 query heads of 128: values 2^31 and on begin at node 16,384. All nodes have the
    same queries (a stride of 0), so each output is that of its heads over the rows up to its own."""
    n, Hq, D, page = 16500, 1024, 128, 128
    rng = np.random.RandomState(3)
    pages = -(-n // page)
    host = []
    for _ in range(2):
        codes, scales = ref.quantise(rng.randn(1, page, D))              # page p holds this one's rows, turned by p
        at = (np.arange(page)[None, :] + 7 * np.arange(pages)[:, None]) % page
        host += [codes[0][at][:, None], scales[0][at][:, None]]
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    cache = moe.KvCache(dev(host[0]), dev(host[2]), dev(host[1]), dev(host[3]))
    table = np.arange(pages, dtype=np.int32)[None, :]
    q = torch.from_numpy(rng.randn(1, Hq, D)).bfloat16()
    out = torch.full((n, Hq, D), 9.0, dtype=torch.bfloat16, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = torch.empty(moe.moe_tree_attention_workspace_bytes(n, Hq, 1, D, 1), dtype=torch.uint8, device="cuda")
    moe.moe_tree_attention(q.cuda().expand(n, Hq, D), cache, dev(table), i32(n), i32(0, n), n, None, D ** -0.5, out, ws)
    torch.cuda.synchronize()
    assert moe.moe_device_status() == (moe.MOE_OK, 0)
    assert not any((out[a:a + 500] == 9.0).all(-1).any().item() for a in range(0, n, 500))
    k, v = (ref.lane_rows(ref.values(*host[i:i + 2]), table[0], n)[:, 0] for i in (0, 2))
    for t in (0, 100, 8191, 16383, 16384, 16385, 16450, 16499):
        for h in (0, 15, 16, 511, 1023):
            o, _, mass = ref.attention(q[:, h].double().numpy(), k[:t + 1], v[:t + 1], np.ones((1, t + 1), bool), D ** -0.5)
            got = out[t, h].double().cpu().numpy()
            # the weights' and the output's roundings, 2^-8 each
            assert (np.abs(got - o[0]) <= 2.0 ** -8 * np.abs(o[0]) + 2.0 ** -8 * mass[0] + 1e-6).all(), (t, h)
