"""How exactly chunk attention holds weights, scores and log sums, and that it does not depend on what else is in the call.

Weights that nearly cancel. A third of a lane's rows has score 0 (weight 1) and values -s, the others weight w and values s, where
w = (1 + 2^-8 - 2^-12) / 2 lies just below the middle of two bf16 numbers: rounded to bf16 it is 1/2, which is off by
2^-8 - 2^-12 of itself, in all rows the same way. The output is near 0, so its own rounding hides nothing: one bf16 part is off by
about 2^-9 of sum p |v| = 1, two parts by at most 2^-16. Beside that, u = 2^-24: the exponential and its argument (|score| < 1)
by 2^-20 together, n rows added up by 2 n / 16 u and their weights by n / 32 u.

Random rows, mean squares. The output's rounding is even within half a step h of the output: h^2 / 3. The weights' is, too, and
independent from row to row: half a step of a weight is 2^-8 / f of it, with f in [1, 2), whose 1 / f^2 is 3 / (8 ln 2) = 0.541 over
all sizes, so r^2 0.541 / 3 sum p^2 v^2 with r = 2^-8, or 2^-16 in two parts. A query element is exact down to 2^-7 of its row's
largest and held within 2^-15 of it below (2^-9 and 2^-17, and rows that share a factor are within 2^2 of one another in these
cases), so a score is off by a sum over the small elements, independent from row to row: e_j^2 = (scale 2^-15 |q|max)^2 / 3 times
their k_jd^2, and D / 32 products cut off at 2^-24 of the score's size. That makes sum p^2 v^2 e^2 of the output and sum p^2 e^2 of
the log sum, which has four roundings more, 2^-24 each of itself or of one. Over thousands of outputs the mean of
the squares is within a tenth of that. Scores are small here, so that many weights matter, and not one alone, which would be 1.
"""
import numpy as np
import pytest
import torch

from tests import kv_reference as ref
from tests.test_gpu_chunk_attention import Chunks

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("resident_expert_routed_gb300")

U = 2.0 ** -24
WEIGHT = 0.5 * (1 + 2.0 ** -8 - 2.0 ** -12)
SCALE = float(np.float32(-np.log(WEIGHT)))
FEW = 1024                                                     # (token, query head) rows of a lane that has two parts


def cancelling(lanes, Hq, Hkv, D, page):
    c = Chunks(lanes, Hq, Hkv, D, page, scale=SCALE)
    c.pool[0][...], c.pool[2][...] = 0, 0
    c.pool[1][...], c.pool[3][...] = 127, 127
    for b, (p, n) in enumerate(lanes):
        for j in range(p + n):
            at, row = c.at(b, j)
            other = j % 3 > 0
            if other:
                c.pool[0][at, :, row, 0] = 0xB8                # -1
            c.pool[2][at, :, row, 0::2] = 0x38 if other else 0xB8
            c.pool[2][at, :, row, 1::2] = 0xB8 if other else 0x38
    c.q.zero_()
    c.q[..., 0] = 1.0
    return c


def lane_errors(c, out, b):
    """(what the lane's outputs are off, what they may be off beside their weights) by token."""
    p, n = c.lanes[b]
    seen = p + 1 + np.arange(n)
    ones = -(-seen // 3)
    w = np.exp(-SCALE)
    o = ((seen - ones) * w - ones) / (ones + (seen - ones) * w)
    got = out[c.cu[b]:c.cu[b + 1]].double().cpu().numpy()
    sign = np.where(np.arange(c.D) % 2, -1.0, 1.0)
    off = np.abs(got - o[:, None, None] * sign).max((1, 2))
    return off, 2.0 ** -8 * np.abs(o) + 2.0 ** -20 + (2 / 16 + 1 / 32) * U * seen


def check_lanes(c, out):
    for b, (p, n) in enumerate(c.lanes):
        if n:
            off, other = lane_errors(c, out, b)
            weight = 2.0 ** -16 if n * c.Hq <= FEW else 2.0 ** -8
            assert (off <= weight + other).all(), (b, p, n, float((off - other).max()))


@pytest.mark.parametrize("D,page", [(64, 16), (128, 64), (256, 128)])
def test_a_lane_of_few_rows_holds_its_weights_whatever_is_beside_it(D, page):
    """Alone, in a batch of more than 1,024 rows, beside chunks: two parts each time."""
    lane = (2900, 1)
    for lanes in ([lane], [lane] + [(700 + 31 * i, 1) for i in range(39)], [(0, 300), lane, (5, 130), (64, 32), (128, 33), (1000, 2)]):
        c = cancelling(lanes, 32, 8, D, page)
        out, _ = c.gpu()
        assert moe.moe_device_status() == (moe.MOE_OK, 0)
        check_lanes(c, out)


@pytest.mark.parametrize("tail", [0, 1, 40])
def test_rows_of_q_behind_the_last_lane_do_not_change_a_lanes_weights(tail):
    """32 single tokens of 32 heads are 1,024 rows; q has some more."""
    c = cancelling([(400 + i, 1) for i in range(32)], 32, 8, 128, 64)
    cache, table, kv_len, cu, out, lse, ws = c.args(tail=tail)
    q = torch.cat([c.q, torch.ones((tail, 32, 128), dtype=torch.bfloat16, device="cuda")])
    moe.moe_chunk_attention(q, cache, table, kv_len, cu, c.scale, out, ws, lse=lse)
    assert moe.moe_device_status() == (moe.MOE_OK, 0)
    check_lanes(c, out)


@pytest.mark.parametrize("Hq,Hkv,n", [(1, 1, 1024), (1, 1, 1025), (4, 1, 256), (8, 8, 128), (8, 1, 129), (128, 1, 8), (96, 1, 10), (128, 8, 9)])
@pytest.mark.parametrize("D", [64, 256])
def test_lanes_at_the_bound(Hq, Hkv, n, D):
    """Of one row tile and of several, of up to 1,024 rows and more; beside single tokens."""
    c = cancelling([(700, n), (60, 1), (0, n)], Hq, Hkv, D, 32)
    out, _ = c.gpu()
    assert moe.moe_device_status() == (moe.MOE_OK, 0)
    check_lanes(c, out)


def half_step(x):
    """Half the distance of bf16 numbers at x."""
    return np.ldexp(1.0, np.frexp(np.abs(x) + 2.0 ** -120)[1] - 9)


@pytest.mark.parametrize("lanes,Hq,Hkv,D", [([(5000, 1)] * 30, 2, 2, 64), ([(700 + 9 * i, 1) for i in range(40)], 32, 8, 128), ([(3000, 4)] * 6, 16, 2, 256),
                                            ([(0, 513)], 16, 16, 64), ([(0, 300)], 32, 8, 128), ([(1500, 200)], 8, 2, 256), ([(9000, 130)], 16, 4, 128)])
def test_mean_squares(lanes, Hq, Hkv, D):
    c = Chunks(lanes, Hq, Hkv, D, 64, seed=D + Hq, gain=0.3)
    out, lse = c.gpu()
    assert moe.moe_device_status() == (moe.MOE_OK, 0)
    few = lanes[0][1] * Hq <= FEW
    r = 2.0 ** -16 if few else 2.0 ** -8
    got, may, sums, sums_may = [], [], [], []
    for b, (p, n) in enumerate(lanes):
        which = np.unique(np.r_[0, n - 1, c.rng.randint(0, n, 24)])
        rows = torch.from_numpy(c.cu[b] + which).cuda()
        for h in range(Hq):
            k, v = c.values(0, b, h // (Hq // Hkv), p + n), c.values(2, b, h // (Hq // Hkv), p + n)
            q = c.q[rows, h].double().cpu().numpy()
            s = np.where(np.arange(p + n) <= p + which[:, None], q @ k.T * c.scale, -np.inf)
            top = s.max(-1, keepdims=True)
            w = np.exp(s - top)
            total = w.sum(-1, keepdims=True)
            w /= total
            o, e = w @ v, (top + np.log(total))[:, 0]
            most = np.abs(q).max(-1, keepdims=True)
            score = (c.scale * 2.0 ** -15 * most) ** 2 / 3 * ((np.abs(q) < 2.0 ** -7 * most) @ (k * k).T) + (D / 32 * U * c.scale * (np.abs(q) @ np.abs(k).T)) ** 2
            got.append((out[rows, h].double().cpu().numpy() - o) ** 2)
            may.append(half_step(o) ** 2 / 3 + (w * w) @ (v * v) * 0.541 * r * r / 3 + (w * w * score) @ (v * v) + (2.0 ** -20 * (w @ np.abs(v))) ** 2)
            sums.append((lse[rows, h].double().cpu().numpy() - e) ** 2)
            sums_may.append((w * w * score).sum(-1) + (2.0 ** -22 * (1 + np.abs(e))) ** 2)
    got, may, sums, sums_may = (np.concatenate([x.ravel() for x in y]).mean() for y in (got, may, sums, sums_may))
    assert got <= 1.1 * may, got / may
    assert sums <= 1.1 * sums_may, sums / sums_may
