"""Build libmla_b200.so (nvcc, sm_100a) and _torch_calls.so (the extension module
that takes the cache-side calls from Python to it) in-tree.

    python -m mla_paged_kv_03_b200.build [--force]

The build fails if ptxas reports more than SPILL_LIMIT bytes of register
spill stores in any kernel (the reference project's setup fails on any spill
[FlashMLA (AI Wiki), "Requirements and build"]; a few bytes in the fused and
sparse variants' rarely taken paths are tolerated here and reported).
"""
import os
import re
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmla_b200.so")
SOURCES = [os.path.join(CSRC, "mla_api.cu")]
DEPS = SOURCES + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))] + \
    [os.path.join(ROOT, "include", "mla.h")]

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
SPILL_LIMIT = 64  # bytes of spill stores tolerated per kernel
FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "--expt-relaxed-constexpr",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-Xptxas", "-v",
    "-shared",
]


CALLS = os.path.join(HERE, "_torch_calls.so")
CALLS_DEPS = [os.path.join(CSRC, "torch_calls.cpp"), os.path.join(ROOT, "include", "mla.h")]
CALLS_BUILT_WITH = os.path.join(HERE, "_torch_calls.built_with")  # calls_key() of CALLS


def calls_key() -> str:
    """The torch and Python whose ABI _torch_calls.so is compiled against."""
    import torch
    return f"torch {torch.__version__}, {sysconfig.get_config_var('SOABI')}"


def _stale(target=LIB, deps=DEPS):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build_calls(force: bool = False) -> str:
    """Compile _torch_calls.so against the installed torch and libmla_b200.so."""
    import torch
    key = calls_key()
    if not force and not _stale(CALLS, CALLS_DEPS) and os.path.exists(CALLS_BUILT_WITH):
        with open(CALLS_BUILT_WITH) as f:
            if f.read() == key:
                return CALLS
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(NVCC))
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC",
           "-fvisibility=hidden", "-Wall", "-Wno-unknown-pragmas",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DMLA_BUILT_WITH="{key}"',
           "-isystem", os.path.join(base, "include"),
           "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"),
           "-isystem", sysconfig.get_paths()["include"], "-o", CALLS, CALLS_DEPS[0],
           "-L", os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
           "-L", HERE, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("building _torch_calls.so failed")
    with open(CALLS_BUILT_WITH, "w") as f:
        f.write(key)
    return CALLS


def build(force: bool = False, verbose: bool = False, out: str = None, defines=()) -> str:
    """Compile libmla_b200.so (or `out`, with extra -D `defines`)."""
    target = out or LIB
    if not force and not defines and out is None and not _stale():
        build_calls()
        return LIB
    cmd = [NVCC] + FLAGS + [f"-D{d}" for d in defines] + \
        ["-I", os.path.join(ROOT, "include"), "-o", target] + SOURCES + ["-lcudart"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    log = r.stdout + r.stderr
    if r.returncode != 0:
        sys.stderr.write(log)
        raise RuntimeError("nvcc failed building libmla_b200.so")
    spills = [l for l in log.splitlines()
              if (m := re.search(r"(\d+) bytes spill stores", l)) and int(m.group(1)) > SPILL_LIMIT]
    if spills:
        if os.path.exists(target):
            os.remove(target)
        sys.stderr.write(log)
        raise RuntimeError("register spill in libmla_b200 kernels:\n" + "\n".join(spills))
    if verbose:
        sys.stderr.write(log)
    if out is None:
        with open(os.path.join(HERE, "ptxas_report.txt"), "w") as f:
            f.write(log)
        build_calls(force)
    return target


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
