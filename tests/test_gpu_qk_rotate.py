"""Norms and rotation of queries and keys on the GPU against the definition in 64 bits.

Bounds (u = 2^-24). A norm: the sum of D squares is off by at most (D / 8 + 4) u of itself (eight terms a lane, then a
tree), root, division and the product with the weight a few u more, half of the sum's error counts: (D / 16 + 8) u. An
angle is exact to 2^-32 turns and rounded to fp32 (pi u at most), sine and cosine are off by 2 u more: 6 u of the pair's
length for each of the two products, 3 u for their sum. The output's rounding: half a step, eps / 2.
"""
import math

import numpy as np
import pytest
import torch

from resident_expert_routed_gb300.rotary import rotary_frequencies, rotary_turns

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("resident_expert_routed_gb300")

KINDS = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def definition(x, positions, f, weight, eps, interleaved, magnitude):
    """64 bits: values, and the length that roundings act on (the pair's, the value's outside)."""
    y = x.double()
    if weight is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * weight.double()
    n = 2 * len(f)
    angle = positions.double()[:, None, None] * torch.tensor(f, dtype=torch.float64, device=x.device)
    c, s = torch.cos(angle) * magnitude, torch.sin(angle) * magnitude
    out, size = y.clone(), y.abs()
    a, b = (y[..., 0:n:2], y[..., 1:n:2]) if interleaved else (y[..., :n // 2], y[..., n // 2:n])
    length = torch.sqrt(a * a + b * b) * abs(magnitude)
    ra, rb = a * c - b * s, b * c + a * s
    if interleaved:
        out[..., 0:n:2], out[..., 1:n:2] = ra, rb
        size[..., 0:n:2] = size[..., 1:n:2] = length
    else:
        out[..., :n // 2], out[..., n // 2:n] = ra, rb
        size[..., :n // 2] = size[..., n // 2:n] = length
    return out, size


def check(got, want, size, dtype, D, normed):
    u = 2.0 ** -24
    tol = (torch.finfo(dtype).eps / 2) * want.abs() * (1 + 2.0 ** -6) + size * u * (15 + (D / 16 + 8 if normed else 0))
    if dtype is torch.float16:
        tol = tol + 2.0 ** -25                                # half the step of its subnormals
    off = (got.double() - want).abs()
    assert (off <= tol).all(), ((off / tol).max().item(), off.max().item())


def run(T, Q, H, D, kind, turned, norm, interleaved, length=4096, seed=0, strided=True, in_place=False, magnitude=1.0, gain=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = KINDS[kind]
    qkv = (torch.randn((T, (Q + 2 * H) * D), generator=gen, device="cuda") * gain).to(dtype)
    q, k = qkv[:, :Q * D].view(T, Q, D), qkv[:, Q * D:(Q + H) * D].view(T, H, D)
    if not strided:
        q, k = q.contiguous(), k.contiguous()
    v = qkv[:, (Q + H) * D:].clone()
    pos = torch.randint(0, length, (T,), generator=gen, device="cuda").to(torch.int32)
    f = rotary_frequencies(turned)
    w = [1 + 0.3 * torch.randn(D, generator=gen, device="cuda") if norm else None for _ in range(2)]
    want = [definition(x, pos, f, wx, 1e-5, interleaved, magnitude) for x, wx in zip((q, k), w)]
    qo, ko = (q, k) if in_place else (torch.full((T, Q, D), 9.0, dtype=dtype, device="cuda"), torch.full((T, H, D), 9.0, dtype=dtype, device="cuda"))
    moe.moe_qk_rotate(q, k, pos, rotary_turns(f, device="cuda"), qo, ko, q_weight=w[0], k_weight=w[1], eps=1e-5, interleaved=interleaved, magnitude=magnitude)
    for got, (out, size) in zip((qo, ko), want):
        check(got, out, size, dtype, D, norm)
    if strided:
        assert torch.equal(qkv[:, (Q + H) * D:], v)           # the values beside them
    return qo, ko


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("D,turned", [(64, 64), (64, 16), (64, 48), (128, 128), (128, 32), (256, 256), (256, 64), (128, 112)])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
def test_layouts(kind, D, turned, norm, interleaved):
    run(13, 6, 2, D, kind, turned, norm, interleaved, seed=D + turned)


@pytest.mark.parametrize("T", [1, 2, 7, 64, 333, 2049])
@pytest.mark.parametrize("Q,H", [(1, 1), (5, 1), (32, 8), (7, 7), (64, 1)])
def test_sizes(T, Q, H):
    run(T, Q, H, 128, "bf16", 128, True, False, seed=T + Q)
    run(T, Q, H, 64, "bf16", 32, False, True, seed=T + Q)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_in_place_and_contiguous(interleaved, kind):
    run(50, 8, 2, 128, kind, 64, True, interleaved, in_place=True)
    run(50, 8, 2, 128, kind, 64, True, interleaved, strided=False)
    run(50, 8, 2, 64, kind, 64, True, interleaved, strided=False, in_place=True)


@pytest.mark.parametrize("length", [1, 1 << 20, (1 << 31) - 1])
def test_far_positions(length):
    """The definition's own angle, position * f in 64 bits, is off by 2^-53 of itself: 2^-22 at 2^31 radians."""
    run(40, 4, 2, 128, "fp32" if length < 1 << 30 else "bf16", 128, False, False, length=length)


def test_magnitude_and_size():
    run(20, 4, 4, 128, "fp32", 128, False, False, magnitude=1.37)
    run(20, 4, 4, 128, "fp32", 64, True, True, magnitude=-0.5, gain=1e6)
    run(20, 4, 4, 128, "bf16", 64, True, True, gain=1e-4)


def test_negative_positions_turn_back():
    x = torch.randn((9, 2, 64), device="cuda")
    pos = torch.arange(-4, 5, dtype=torch.int32, device="cuda")
    turns = rotary_turns(rotary_frequencies(64), device="cuda")
    y, z = torch.empty_like(x), torch.empty_like(x)
    moe.moe_qk_rotate(x, x, pos, turns, y, torch.empty_like(x))
    moe.moe_qk_rotate(y, y, -pos, turns, z, torch.empty_like(x))
    # 15 u a rotation, of a pair's length
    assert ((z - x).abs() <= 40 * 2.0 ** -24 * x.abs().max()).all()


def test_norms_alone_one_side_alone_and_no_tokens():
    x = torch.randn((5, 3, 64), device="cuda")
    w = torch.rand(64, device="cuda")
    pos, none = torch.zeros(5, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int64, device="cuda")
    out, empty = torch.empty_like(x), x[:, :0]
    moe.moe_qk_rotate(x, empty, pos, none, out, empty, q_weight=w)
    want = x.double() / torch.sqrt((x.double() ** 2).mean(-1, keepdim=True) + 1e-6) * w.double()
    assert ((out - want).abs() <= 20 * 2.0 ** -24 * want.abs()).all()
    kout = torch.empty_like(x)
    moe.moe_qk_rotate(empty, x, pos, none, empty, kout, k_weight=w)
    assert torch.equal(kout, out)
    moe.moe_qk_rotate(x[:0], x[:0], pos[:0], none, out[:0], out[:0])


def test_values_that_are_not_finite_stay_in_their_vector():
    x = torch.randn((4, 3, 64), device="cuda")
    x[1, 2, 5], x[2, 0, 63] = math.inf, math.nan
    out, kout = torch.empty_like(x), torch.empty_like(x)
    w = torch.ones(64, device="cuda")
    turns = rotary_turns(rotary_frequencies(64), device="cuda")
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    moe.moe_qk_rotate(x, x, pos, turns, out, kout, q_weight=w)
    bad = ~torch.isfinite(out).all(-1)
    assert bad.nonzero().tolist() == [[1, 2], [2, 0]]
    bad = ~torch.isfinite(kout)
    assert bad.nonzero().tolist() == [[1, 2, 5], [1, 2, 37], [2, 0, 31], [2, 0, 63]]


def test_captured_on_a_side_stream():
    x = torch.randn((33, 8, 128), device="cuda").bfloat16()
    pos = torch.arange(33, dtype=torch.int32, device="cuda")
    turns = rotary_turns(rotary_frequencies(128), device="cuda")
    out, want = torch.empty_like(x), torch.empty_like(x)
    k = x[:, :2]
    ko = torch.empty((33, 2, 128), dtype=torch.bfloat16, device="cuda")
    moe.moe_qk_rotate(x, k, pos, turns, want, ko)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        moe.moe_qk_rotate(x, k, pos, turns, out, ko)
    out.zero_()
    graph.replay()
    assert torch.equal(out, want)


def test_refusals():
    x = torch.randn((4, 2, 64), device="cuda")
    i, t = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(32, dtype=torch.int64, device="cuda")
    for bad in (dict(k_out=x.half()), dict(q_out=x[:, :1]), dict(positions=i.long()), dict(turns=t.int()), dict(q=x[..., ::2]),
                dict(q_weight=torch.ones(32, device="cuda")), dict(k_weight=torch.ones(64, device="cuda").bfloat16())):
        with pytest.raises(ValueError):
            moe.moe_qk_rotate(**(dict(q=x, k=x, positions=i, turns=t, q_out=x, k_out=x) | bad))
    with pytest.raises(moe.MoeError) as e:
        moe.moe_qk_rotate(x, x, i, t[:4], x, x)
    assert e.value.status == moe.MOE_EUNSUPPORTED
