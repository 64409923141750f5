"""Argument checks and sizes of the shared-prefix entry points (no GPU needed;
the addresses are never read)."""
import ctypes

import pytest

from mla_paged_kv_03_b200 import binding as B


def call(**o):
    a = dict(q=16, kc=16, nb=8, pt=16, plen=100, bt=16, mp=4, sl=16, b=2, s_q=1, h_q=16, h_kv=1,
             d_v=512, scale=0.04, causal=1, meta=16, ns=16, parts=4, ws=16, wsb=1 << 30, out=16,
             lse=16)
    a.update(o)
    return B.lib().mla_shared_prefix_decode_fwd(*a.values(), None)


@pytest.mark.parametrize("over,code", [
    (dict(h_kv=2), B.MLA_ERR_UNSUPPORTED), (dict(d_v=576), B.MLA_ERR_UNSUPPORTED)] + [
    (o, B.MLA_ERR_INVALID_ARG) for o in (
        dict(q=None), dict(kc=None), dict(pt=None), dict(bt=None), dict(sl=None), dict(meta=None),
        dict(ns=None), dict(ws=None), dict(out=None), dict(lse=None), dict(q=8), dict(kc=8),
        dict(ws=8), dict(out=8), dict(pt=2), dict(plen=-1), dict(mp=0), dict(nb=0), dict(b=-1),
        dict(s_q=0), dict(h_q=0), dict(scale=0.0), dict(scale=float("inf")), dict(parts=0),
        dict(parts=5000), dict(wsb=1000), dict(plen=2 ** 31 - 1, mp=100), dict(b=9000),
        dict(b=4000, h_q=200), dict(b=1 << 20, s_q=1 << 10, h_q=16))])
def test_bad_arguments_are_refused(over, code):
    assert call(**over) == code
    assert B.lib().mla_last_error().decode() != ""


def test_empty_batch_and_absent_prefix():
    assert call(b=0) == B.MLA_OK
    assert call(b=0, plen=0, pt=None) == B.MLA_OK


def test_plan_checks_and_sizes():
    L = B.lib()
    m, s, w = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    # 5 sequences of 150 rows: 6 groups over the prefix, 2 per sequence over own tokens
    assert L.mla_shared_prefix_metadata_size(5, 150, 64, 74, ctypes.byref(m), ctypes.byref(s)) == 0
    assert m.value == 74 * 32 and s.value == (6 + 10 + 1) * 4
    assert L.mla_shared_prefix_metadata_size(5, 150, 0, 74, ctypes.byref(m), ctypes.byref(s)) == 0
    assert s.value == (10 + 1) * 4
    assert L.mla_shared_prefix_workspace_size(5, 150, 64, 74, ctypes.byref(w)) == 0
    assert w.value >= (16 + 74) * 128 * 513 * 4
    bad = [(None, 2, 16, 1, 10, 4, 16, 16), (16, -1, 16, 1, 10, 4, 16, 16),
           (16, 2, 0, 1, 10, 4, 16, 16), (16, 2, 16, 1, -1, 4, 16, 16),
           (16, 2, 16, 1, 10, 0, 16, 16), (16, 2, 16, 1, 10, 4, None, 16),
           (16, 2, 16, 1, 10, 4, 16, None), (2, 2, 16, 1, 10, 4, 16, 16),
           (16, 8192, 128, 1, 10, 4, 16, 16)]
    for args in bad:
        assert L.mla_shared_prefix_get_metadata(*args, None) == B.MLA_ERR_INVALID_ARG
    assert L.mla_shared_prefix_get_metadata(16, 2, 16, 2, 10, 4, 16, 16, None) == \
        B.MLA_ERR_UNSUPPORTED
