"""Scores of any finite size in chunk attention, against the definition in 64 bits."""
import numpy as np
import pytest
import torch

from tests.test_gpu_chunk_attention import Chunks

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("resident_expert_routed_gb300")

U = 2.0 ** -24


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("up", [40, 60])
def test_scores_far_below_zero(D, up):
    """All of a row's scores the same, -2^(60 + up): the weights are equal, whatever the scores' size."""
    c = Chunks([(300, 150), (200, 1), (0, 3)], 4, 2, D, 64, seed=3, scale=1.0)
    c.q.zero_()
    c.q[..., 0] = 2.0 ** 60
    c.pool[0][...], c.pool[1][...] = 0, 127 + up
    c.pool[0][..., 0] = 0xB8
    out, lse = c.gpu()
    assert moe.moe_device_status() == (moe.MOE_OK, 0)
    for b, (p, n) in enumerate(c.lanes):
        for h in range(4):
            v = c.values(2, b, h // 2, p + n)
            for t in sorted({0, n // 2, n - 1}):
                seen, at = p + t + 1, c.cu[b] + t
                mean, mass = v[:seen].mean(0), np.abs(v[:seen]).mean(0)
                x = out[at, h].double().cpu().numpy()
                # weights of 1: nothing is rounded but the sums (n / 16 u, twice) and the output
                assert (np.abs(x - mean) <= 2.0 ** -8 * np.abs(mean) + 2 * (seen / 16 + 8) * U * mass).all(), (b, t, h)
                assert abs(lse[at, h].item() / -2.0 ** (60 + up) - 1) <= 2.0 ** -21
