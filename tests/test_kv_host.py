"""Host checks of the key/value cache and tree attention calls (no GPU needed): bad arguments are refused before
anything is launched."""
import ctypes

import numpy as np
import pytest
import torch

import resident_expert_routed_gb300 as moe
from tests import kv_reference as ref

NULL = None
P = ctypes.c_void_p(0x1000)             # never dereferenced: every case below fails a host check first
ODD = ctypes.c_void_p(0x1008)


def cache(**kw):
    f = dict(k_codes=0x1000, v_codes=0x2000, k_scales=0x3000, v_scales=0x4000, n_pages=4, n_kv_heads=2, page_size=16, head_dim=64)
    f.update(kw)
    return ctypes.byref(moe.MoeKvCache(*f.values()))


def write(c=None, k=P, v=P, dtype=moe.MOE_BF16, strides=(128, 64, 128, 64), slots=P, T=4):
    return moe.load().moe_kv_write(k, v, dtype, *strides, slots, T, cache() if c is None else c, NULL)


def read(c=None, table=P, width=2, lanes=2, cu=P, n=4, dtype=moe.MOE_BF16, k=P, v=P):
    return moe.load().moe_kv_read(cache() if c is None else c, table, width, lanes, NULL, cu, n, dtype, k, v, NULL)


def keep(c=None, table=P, width=2, lanes=2, prefix=P, path=P, path_width=4, n_keep=P):
    return moe.load().moe_kv_keep(cache() if c is None else c, table, width, lanes, prefix, path, path_width, n_keep, NULL)


def attend(c=None, q=P, strides=(256, 64), n=4, heads=4, table=P, width=2, lanes=2, kv_len=P, cu=P, max_nodes=2, mask=NULL,
           words=0, scale=0.1, out=P, lse=NULL, ws=P, ws_bytes=1 << 40):
    return moe.load().moe_tree_attention(q, *strides, n, heads, cache() if c is None else c, table, width, lanes, kv_len, cu,
                                         max_nodes, mask, words, ctypes.c_float(scale), out, lse, ws, ws_bytes, NULL)


CALLS = (write, read, keep, attend)


def test_struct_layout_matches_header():
    assert ctypes.sizeof(moe.MoeKvCache) == 4 * 8 + 4 * 4
    assert moe.MoeKvCache.n_pages.offset == 32 and moe.MoeKvCache.head_dim.offset == 44


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("kw,status", [
    (dict(k_codes=None), moe.MOE_EINVAL), (dict(v_scales=None), moe.MOE_EINVAL),
    (dict(v_codes=0x2008), moe.MOE_EINVAL), (dict(k_scales=0x3001), moe.MOE_EINVAL),
    (dict(n_pages=0), moe.MOE_EINVAL), (dict(n_kv_heads=0), moe.MOE_EINVAL), (dict(page_size=24), moe.MOE_EINVAL),
    (dict(page_size=0), moe.MOE_EINVAL),
    (dict(page_size=8), moe.MOE_EUNSUPPORTED), (dict(page_size=2048), moe.MOE_EUNSUPPORTED),
    (dict(head_dim=96), moe.MOE_EUNSUPPORTED), (dict(head_dim=512), moe.MOE_EUNSUPPORTED),
    (dict(n_kv_heads=1025), moe.MOE_EUNSUPPORTED), (dict(n_pages=1 << 26, n_kv_heads=2, page_size=16), moe.MOE_EUNSUPPORTED),
])
def test_every_call_checks_the_cache(call, kw, status):
    assert call(c=cache(**kw)) == status


def test_write_refusals():
    for kw in (dict(k=NULL), dict(v=NULL), dict(slots=NULL), dict(k=ODD), dict(v=ODD), dict(dtype=3), dict(dtype=-1), dict(T=-1),
               dict(strides=(128, 64, 124, 64)), dict(strides=(128, 60, 128, 64)), dict(dtype=moe.MOE_FP32, strides=(126, 64, 128, 64))):
        assert write(**kw) == moe.MOE_EINVAL, kw
    assert write(T=(1 << 26) + 1) == moe.MOE_EUNSUPPORTED
    assert write(T=0, k=NULL, v=NULL, slots=NULL) == moe.MOE_OK


def test_read_refusals():
    for kw in (dict(table=NULL), dict(cu=NULL), dict(k=NULL), dict(v=ODD), dict(dtype=7), dict(n=-1), dict(lanes=0), dict(width=0)):
        assert read(**kw) == moe.MOE_EINVAL, kw
    assert read(lanes=65537) == moe.MOE_EUNSUPPORTED and read(n=(1 << 26) + 1) == moe.MOE_EUNSUPPORTED
    assert read(n=0, table=NULL, k=NULL) == moe.MOE_OK


def test_keep_refusals():
    for kw in (dict(table=NULL), dict(prefix=NULL), dict(path=NULL), dict(n_keep=NULL), dict(lanes=-1), dict(width=0), dict(path_width=0)):
        assert keep(**kw) == moe.MOE_EINVAL, kw
    assert keep(lanes=65537) == moe.MOE_EUNSUPPORTED and keep(path_width=4097) == moe.MOE_EUNSUPPORTED
    assert keep(lanes=0, path=NULL) == moe.MOE_OK


def test_attention_refusals():
    for kw in (dict(q=NULL), dict(q=ODD), dict(out=NULL), dict(out=ODD), dict(ws=NULL), dict(ws=ODD), dict(table=NULL), dict(kv_len=NULL),
               dict(cu=NULL), dict(n=-1), dict(heads=3), dict(heads=0), dict(lanes=0), dict(width=0), dict(max_nodes=0),
               dict(strides=(256, 60)), dict(strides=(250, 64)), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(mask=P, words=0), dict(mask=P, words=1, max_nodes=33)):
        assert attend(**kw) == moe.MOE_EINVAL, kw
    for kw in (dict(lanes=4097), dict(heads=1026), dict(max_nodes=65537), dict(mask=P, words=2049)):
        assert attend(**kw) == moe.MOE_EUNSUPPORTED, kw
    assert attend(ws_bytes=0) == moe.MOE_ENOMEM
    need = moe.moe_tree_attention_workspace_bytes(4, 4, 2, 64, 2)
    assert need > 0 and attend(ws_bytes=need - 1) == moe.MOE_ENOMEM
    assert moe.moe_tree_attention_workspace_bytes(0, 4, 2, 64, 2) == 0
    assert attend(n=0, q=NULL, out=NULL, ws=NULL) == moe.MOE_OK


def test_binding_refuses_host_tensors_and_other_shapes():
    codes, scales = torch.zeros((4, 2, 16, 64), dtype=torch.uint8), torch.zeros((4, 2, 16), dtype=torch.uint8)
    with pytest.raises(ValueError):
        moe.KvCache(codes, codes, scales, scales)                          # host memory
    with pytest.raises(ValueError):
        moe.KvCache(codes, codes[:3], scales, scales)
    with pytest.raises(ValueError):
        moe.KvCache(codes, codes, scales, scales.int())
    with pytest.raises(ValueError):
        moe.KvCache(codes.int(), codes.int(), scales, scales)


def test_reference_rounding_pins():
    # the reference's own e4m3: pinned values, ties to even, and every code maps to itself
    assert ref.E4M3[0x38] == 1.0 and ref.E4M3[0x7E] == 448.0 and ref.E4M3[0x01] == 2.0 ** -9 and ref.E4M3[0xC0] == -2.0
    fine = [c for c in range(256) if (c & 0x7F) != 0x7F]
    assert list(ref.round_e4m3(ref.E4M3[fine])) == fine
    assert list(ref.round_e4m3(np.array([1.0625, 1.1875, 2.0 ** -10, 3 * 2.0 ** -10, -17.0]))) == [0x38, 0x3A, 0x00, 0x02, 0xD8]
    codes, scales = ref.quantise(np.array([[448.0, 1.0], [449.0, 1.0], [0.0, 0.0], [np.inf, 1.0]]))
    assert list(scales) == [127, 128, 127, 255] and codes[0, 0] == 0x7E and codes[3, 1] == 0
