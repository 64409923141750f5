"""Argument checks of mla_cache_append: refused before anything is launched (no
GPU needed; the addresses are never read)."""
import pytest

from mla_paged_kv_03_b200 import binding as B


def call(**o):
    a = dict(kv=16, stride=576, d=576, slots=16, pos=16, gain=16, eps=1e-6, base=1e4, n=4,
             cache=16, num_slots=128, row_bytes=1152, rows=16)
    a.update(o)
    return B.lib().mla_cache_append(a["kv"], a["stride"], a["d"], a["slots"], a["pos"], a["gain"],
                                    a["eps"], a["base"], a["n"], a["cache"], a["num_slots"],
                                    a["row_bytes"], a["rows"], None)


@pytest.mark.parametrize("over", [
    dict(kv=None), dict(slots=None), dict(cache=None), dict(kv=8), dict(cache=24), dict(rows=8),
    dict(slots=2), dict(pos=2), dict(gain=2), dict(d=512), dict(row_bytes=528),
    dict(row_bytes=512), dict(row_bytes=0), dict(stride=568), dict(stride=580), dict(stride=-576),
    dict(stride=1 << 32), dict(n=-1), dict(num_slots=0), dict(num_slots=1 << 31), dict(eps=-1.0),
    dict(eps=float("nan")), dict(base=0.0), dict(base=float("inf")),
    dict(d=576, row_bytes=288), dict(d=512, row_bytes=656),
])
def test_bad_arguments_are_refused(over):
    assert call(**over) == B.MLA_ERR_INVALID_ARG
    assert B.lib().mla_last_error().decode() != ""


def test_no_tokens_is_a_no_op():
    assert call(n=0) == B.MLA_OK
    assert call(n=0, d=512, stride=512, row_bytes=288) == B.MLA_OK
