"""Argument checks and sizes of the page-selection entry points (no GPU needed;
the addresses are never read)."""
import ctypes

import pytest

from mla_paged_kv_03_b200 import binding as B


def keys(**o):
    a = dict(kc=16, nb=8, bt=16, mp=4, sl=16, b=2, tail=4, keys=16, scales=16)
    a.update(o)
    return B.lib().mla_page_keys_update(*a.values(), None)


def decode(**o):
    a = dict(q=16, kc=16, nb=8, keys=16, scales=16, bt=16, mp=4, sl=16, b=2, s_q=1, h_q=16, h_kv=1,
             d_v=512, topk=2, scale=0.04, causal=1, parts=4, ws=256, wsb=1 << 30, pages=16, out=16,
             lse=16)
    a.update(o)
    return B.lib().mla_page_sparse_decode(*a.values(), None)


@pytest.mark.parametrize("over", [
    dict(kc=None), dict(bt=None), dict(sl=None), dict(keys=None), dict(scales=None), dict(kc=8),
    dict(keys=8), dict(bt=2), dict(sl=2), dict(scales=2), dict(nb=0), dict(mp=0), dict(tail=0),
    dict(tail=-1), dict(b=-1), dict(b=65536), dict(nb=1 << 25), dict(mp=1 << 25)])
def test_key_update_refuses(over):
    assert keys(**over) == B.MLA_ERR_INVALID_ARG
    assert B.lib().mla_last_error().decode() != ""


@pytest.mark.parametrize("over,code", [(dict(h_kv=2), B.MLA_ERR_UNSUPPORTED)] + [
    (o, B.MLA_ERR_INVALID_ARG) for o in (
        dict(q=None), dict(kc=None), dict(keys=None), dict(scales=None), dict(bt=None),
        dict(sl=None), dict(ws=None), dict(out=None), dict(lse=None), dict(q=8), dict(kc=8),
        dict(keys=8), dict(scales=2), dict(pages=2), dict(bt=2), dict(sl=2), dict(ws=128),
        dict(out=8), dict(lse=2), dict(nb=0), dict(mp=0), dict(b=-1), dict(s_q=0), dict(h_q=0),
        dict(d_v=256), dict(topk=0), dict(scale=0.0), dict(scale=float("nan")), dict(parts=0),
        dict(parts=1 << 20), dict(wsb=100), dict(b=8193), dict(b=1 << 20, s_q=1 << 12))])
def test_decode_refuses(over, code):
    assert decode(**over) == code
    assert B.lib().mla_last_error().decode() != ""


def test_empty_batches_are_no_ops():
    assert keys(b=0) == B.MLA_OK
    assert decode(b=0) == B.MLA_OK


def test_workspace_size():
    n = ctypes.c_size_t()
    size = B.lib().mla_page_sparse_workspace_size
    assert size(3, 2, 16, 512, 1000, 8, 74, ctypes.byref(n)) == 0
    assert n.value >= 6 * 1000 * 4 + 6 * 8 * 4
    small = n.value
    assert size(3, 2, 16, 512, 1000, 2000, 74, ctypes.byref(n)) == 0
    assert n.value >= small
    for bad in [(-1, 1, 1, 512, 1, 1, 1), (1, 0, 1, 512, 1, 1, 1), (1, 1, 0, 512, 1, 1, 1),
                (1, 1, 1, 500, 1, 1, 1), (1, 1, 1, 512, 0, 1, 1), (1, 1, 1, 512, 1, 0, 1),
                (1, 1, 1, 512, 1, 1, 0), (8193, 1, 1, 512, 1, 1, 1)]:
        assert size(*bad, ctypes.byref(n)) == B.MLA_ERR_INVALID_ARG
    assert size(1, 1, 1, 512, 1, 1, 1, None) == B.MLA_ERR_INVALID_ARG
