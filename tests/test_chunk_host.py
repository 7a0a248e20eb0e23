"""Host checks of the plan, rotation and chunk attention calls (no GPU needed): bad arguments are refused before anything
is launched."""
import ctypes
import math

import pytest
import torch

import resident_expert_routed_gb300 as moe
from tests.test_kv_host import NULL, ODD, P, cache


def plan(n_new=P, rows=P, held=P, table=P, width=4, lanes=2, free=P, n_pages=8, n_free=P, page=16, kv_len=P, cu=P, pos=P, slots=P, T=4):
    return moe.load().moe_page_plan(n_new, rows, held, table, width, lanes, free, n_pages, n_free, page, kv_len, cu, pos, slots, T, NULL)


def rotate(q=P, k=P, dtype=moe.MOE_BF16, strides=(256, 64) * 4, T=4, Q=4, H=2, D=64, pos=P, turns=P, pairs=32, interleaved=0,
           magnitude=1.0, qw=NULL, kw=NULL, eps=1e-6, qo=P, ko=P):
    return moe.load().moe_qk_rotate(q, k, dtype, None if strides is None else moe._STRIDES.pack(*strides), T, Q, H, D, pos, turns, pairs,
                                    interleaved, magnitude, qw, kw, eps, qo, ko, NULL)


def attend(c=None, q=P, strides=(256, 64), n=4, heads=4, table=P, width=2, lanes=2, kv_len=P, cu=P, scale=0.1, out=P, lse=NULL, ws=P,
           ws_bytes=1 << 40):
    return moe.load().moe_chunk_attention(q, *strides, n, heads, cache() if c is None else c, table, width, lanes, kv_len, cu, scale,
                                          out, lse, ws, ws_bytes, NULL)


def test_plan_refusals():
    for name in ("n_new", "rows", "held", "table", "free", "n_free", "kv_len", "cu", "pos", "slots"):
        assert plan(**{name: NULL}) == moe.MOE_EINVAL, name
    for kw in (dict(lanes=0), dict(width=0), dict(n_pages=0), dict(T=-1), dict(page=0), dict(page=24)):
        assert plan(**kw) == moe.MOE_EINVAL, kw
    for kw in (dict(lanes=4097), dict(page=8), dict(page=2048), dict(T=(1 << 24) + 1), dict(width=(1 << 20) + 1), dict(n_pages=1 << 27)):
        assert plan(**kw) == moe.MOE_EUNSUPPORTED, kw


def test_rotate_refusals():
    for kw in (dict(q=NULL), dict(k=NULL), dict(qo=NULL), dict(ko=NULL), dict(pos=NULL), dict(turns=NULL), dict(strides=None), dict(q=ODD),
               dict(k=ODD), dict(qo=ODD), dict(ko=ODD), dict(qw=ODD), dict(kw=ODD), dict(dtype=3), dict(dtype=-1), dict(T=-1), dict(Q=-1),
               dict(Q=0, H=0), dict(pairs=-8), dict(pairs=40), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf),
               dict(magnitude=math.nan), dict(magnitude=math.inf)):
        assert rotate(**kw) == moe.MOE_EINVAL, kw
    for i in range(8):
        s = [256, 64] * 4
        s[i] += 4
        assert rotate(strides=s) == moe.MOE_EINVAL
        assert rotate(strides=[x + 2 if j == i else x for j, x in enumerate([256, 64] * 4)], dtype=moe.MOE_FP32) == moe.MOE_EINVAL
    for kw in (dict(D=96), dict(D=32), dict(D=512), dict(pairs=4), dict(pairs=12), dict(Q=65537), dict(T=1 << 30)):
        assert rotate(**kw) == moe.MOE_EUNSUPPORTED, kw
    assert rotate(T=0, q=NULL, k=NULL) == moe.MOE_OK


def test_attention_refusals():
    for kw in (dict(q=NULL), dict(q=ODD), dict(out=NULL), dict(out=ODD), dict(ws=NULL), dict(ws=ODD), dict(table=NULL), dict(kv_len=NULL),
               dict(cu=NULL), dict(n=-1), dict(heads=3), dict(heads=0), dict(lanes=0), dict(width=0), dict(strides=(256, 60)),
               dict(strides=(250, 64)), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert attend(**kw) == moe.MOE_EINVAL, kw
    for kw in (dict(lanes=4097), dict(heads=1026), dict(heads=260), dict(n=(1 << 24) + 1)):
        assert attend(**kw) == moe.MOE_EUNSUPPORTED, kw
    assert attend(c=cache(head_dim=96)) == moe.MOE_EUNSUPPORTED and attend(c=cache(page_size=24)) == moe.MOE_EINVAL
    assert attend(ws_bytes=0) == moe.MOE_ENOMEM
    need = moe.moe_chunk_attention_workspace_bytes(4, 4, 2, 64, 2)
    assert need > 0 and attend(ws_bytes=need - 1) == moe.MOE_ENOMEM
    assert moe.moe_chunk_attention_workspace_bytes(0, 4, 2, 64, 2) == 0
    assert attend(n=0, q=NULL, out=NULL, ws=NULL) == moe.MOE_OK


def test_binding_refuses_host_tensors_and_other_shapes():
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        moe.moe_page_plan(i, i, i, torch.zeros((4, 2), dtype=torch.int32), i, i[:1], 16, i, torch.zeros(5, dtype=torch.int32), i, i.long())
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        moe.moe_qk_rotate(x, x, i, torch.zeros(32, dtype=torch.int64), x, x)
    with pytest.raises(ValueError):
        moe.moe_qk_rotate(x.int(), x, i, torch.zeros(32, dtype=torch.int64), x, x)
