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


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("scale", [2.0 ** 20, 2.0 ** 60, 2.0 ** 100])
def test_scores_whose_roundings_are_large(D, scale):
    """Scores of 2^22 and far more, of any sign, single tokens and chunks: where the largest is well ahead (2^-9 of the sum of its
    products' sizes, thousands of times what fp32 sums and the queries' holding are off), its value is the output; no row is
    anything but a mean of values."""
    c = Chunks([(300, 150), (200, 1), (0, 3), (1000, 1)], 4, 2, D, 64, seed=4, scale=scale)
    out, lse = c.gpu()
    assert moe.moe_device_status() == (moe.MOE_OK, 0)
    clear = 0
    for b, (p, n) in enumerate(c.lanes):
        for h in range(4):
            k, v = c.values(0, b, h // 2, p + n), c.values(2, b, h // 2, p + n)
            q = c.q[c.cu[b]:c.cu[b] + n, h].double().cpu().numpy()
            x = out[c.cu[b]:c.cu[b] + n, h].double().cpu().numpy()
            e = lse[c.cu[b]:c.cu[b] + n, h].double().cpu().numpy()
            assert np.isfinite(x).all() and np.isfinite(e).all()
            for t in range(n):
                seen = p + t + 1
                s = k[:seen] @ q[t]
                size = (np.abs(k[:seen]) @ np.abs(q[t])).max()
                top = int(s.argmax())
                assert (np.abs(x[t]) <= np.abs(v[:seen]).max(0) * (1 + 2.0 ** -7)).all(), (b, t, h)
                assert abs(e[t] - s[top] * scale) <= 2.0 ** -9 * size * scale
                if seen == 1 or s[top] - np.delete(s, top).max() > 2.0 ** -9 * size:
                    clear += 1
                    assert (np.abs(x[t] - v[top]) <= 2.0 ** -7 * np.abs(v[top])).all(), (b, t, h)
    assert clear > 100
