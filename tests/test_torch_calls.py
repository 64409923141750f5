"""Argument checks of the cache-side calls that need no GPU: CPU tensors, other
objects and wrong counts are refused with a Python error."""
import subprocess
import sys

import pytest
import torch

from mla_paged_kv_03_b200 import binding as B
from mla_paged_kv_03_b200 import build

BF16 = torch.bfloat16


def append_args(**o):
    a = dict(kv=torch.zeros((4, 576), dtype=BF16), slots=torch.zeros(4, dtype=torch.int32),
             kcache=torch.zeros((2, 64, 1, 576), dtype=BF16))
    return a | o


def test_cpu_tensors_are_refused():
    cache = torch.zeros((2, 64, 1, 576), dtype=BF16)
    q = torch.zeros((1, 1, 16, 576), dtype=BF16)
    i32 = torch.zeros((1, 2), dtype=torch.int32)
    sl = torch.zeros(1, dtype=torch.int32)
    keys, scales = torch.zeros((2, 576), dtype=torch.int8), torch.zeros(2)
    with pytest.raises(ValueError, match="kv must be CUDA"):
        B.mla_cache_append(**append_args())
    with pytest.raises(ValueError, match="kcache"):
        B.mla_page_keys_update(cache, i32, sl, keys, scales)
    with pytest.raises(ValueError, match="q must be CUDA"):
        B.mla_page_sparse_decode(q, cache, keys, scales, i32, sl, 2)
    with pytest.raises(ValueError, match="q must be CUDA"):
        B.mla_shared_prefix_decode_fwd(q, cache, sl, 64, i32, sl, i32, sl, 4)


@pytest.mark.parametrize("over", [
    dict(kv=None), dict(kv=[1, 2]), dict(kcache=None), dict(kcache="cache"),
    dict(kcache=torch.zeros((2, 64, 512), dtype=BF16)),
    dict(kcache=torch.zeros((2, 64, 600), dtype=torch.uint8)),
    dict(kcache=torch.zeros((), dtype=BF16)),
    dict(kv=torch.zeros((4, 512), dtype=BF16)), dict(kv=torch.zeros((4, 576)))])
def test_other_objects_and_shapes_are_refused(over):
    with pytest.raises(ValueError):
        B.mla_cache_append(**append_args(**over))


def test_counts_of_arguments():
    for f in (B.calls().cache_append, B.calls().page_keys_update, B.calls().page_sparse_decode,
              B.calls().shared_prefix_decode):
        with pytest.raises(TypeError):
            f()
        with pytest.raises(TypeError):
            f(*[None] * 30)


# Tensors that name a CUDA device without having any memory: the call gets as far as the
# device, where torch throws.  A process of its own, which used to end with a fault there.
AT_THE_DEVICE = """
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
from mla_paged_kv_03_b200 import binding as B
B.calls()
with FakeTensorMode():
    cuda = dict(device="cuda:63")
    args = (torch.empty((2, 64, 1, 576), dtype=torch.bfloat16, **cuda),
            torch.empty((1, 2), dtype=torch.int32, **cuda),
            torch.empty(1, dtype=torch.int32, **cuda),
            torch.empty((2, 576), dtype=torch.int8, **cuda), torch.empty(2, **cuda))
for _ in range(2):
    try:
        B.mla_page_keys_update(*args)
    except Exception as e:
        print("raised", type(e).__name__)
"""


def test_an_error_of_the_device_is_an_exception():
    r = subprocess.run([sys.executable, "-c", AT_THE_DEVICE], capture_output=True, text=True)
    assert r.returncode == 0, (r.returncode, r.stderr[-2000:])
    assert r.stdout.split().count("raised") == 2


def test_a_module_built_with_another_torch_is_built_anew_and_not_used(monkeypatch, tmp_path):
    assert B.calls().BUILT_WITH == build.calls_key()
    monkeypatch.setattr(build, "calls_key", lambda: "torch 0.0.0, cpython-00")
    monkeypatch.setattr(B, "_calls", None)
    with pytest.raises(ImportError, match="torch 0.0.0"):
        B.calls()
    # the build takes the file for stale although it is newer than its sources
    monkeypatch.setattr(build, "CALLS", str(tmp_path / "_torch_calls.so"))
    monkeypatch.setattr(build, "CALLS_BUILT_WITH", str(tmp_path / "_torch_calls.built_with"))
    for f, text in ((build.CALLS, "old"), (build.CALLS_BUILT_WITH, "torch 1.0, cpython-00")):
        with open(f, "w") as out:
            out.write(text)
    compiled = []
    monkeypatch.setattr(build.subprocess, "run", lambda cmd, **kw: compiled.append(cmd) or
                        build.subprocess.CompletedProcess(cmd, 0, "", ""))
    build.build_calls()
    assert len(compiled) == 1 and '-DMLA_BUILT_WITH="torch 0.0.0, cpython-00"' in compiled[0]
    build.build_calls()
    assert len(compiled) == 1
