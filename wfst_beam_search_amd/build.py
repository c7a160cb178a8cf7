"""Build the decoder library (HIP for gfx950 + the C ABI) in-tree with hipcc."""

from __future__ import annotations

import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libwfst_mi355x.so")
SOURCES = [os.path.join(HERE, "csrc", name) for name in (
    "wfst_layer_f32.hip", "wfst_layer_bf16.hip", "wfst_layer_f16.hip", "wfst_kernels.hip", "wfst_tokens.hip",
    "wfst_sample.hip", "wfst_noalloc.hip", "wfst_api.cpp", "wfst_layer.hip", "wfst_adapters.hip", "wfst_norm.hip",
    "wfst_score_api.cpp")]          # (the longest to compile first)

FLAGS = [
    "-O3", "-std=c++17", "--offload-arch=gfx950", "-fPIC",
    # every fp32 operation is rounded on its own: no contraction into FMA
    "-ffp-contract=off",
    # no packed fp32 instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
    # the kernels' few argument dwords (a Work pointer, step, pass) arrive in
    # SGPRs with the dispatch
    "-mllvm", "-amdgpu-kernarg-preload-count=16",
]


# machine probes (random gathers, dependent chains, atomics, launch floor) for
# bench.py --probe: a library of their own, not part of the decoder
PROBE_LIB = os.path.join(HERE, "libwfst_probe.so")
PROBE_SOURCES = [os.path.join(HERE, "csrc", "wfst_probe.hip")]


def _run(cmd, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.check_call(cmd)


def _jobs() -> int:
    """Compilers at once: MAX_JOBS where it is a number, at most 4."""
    given = os.environ.get("MAX_JOBS", "").strip()
    return max(1, min(4, int(given))) if given.isdigit() else 4


def _compile(out: str, sources, verbose: bool) -> None:
    """Each source to an object of its own, several at once, then one shared library."""
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    with tempfile.TemporaryDirectory(prefix="wfst_build_") as tmpdir:
        objs = [os.path.join(tmpdir, f"{i}.o") for i in range(len(sources))]
        with ThreadPoolExecutor(_jobs()) as pool:
            list(pool.map(lambda so: _run([hipcc, *FLAGS, "-I", os.path.join(ROOT, "include"), "-I",
                                           os.path.join(HERE, "csrc"), "-c", "-o", so[1], so[0]], verbose),
                          zip(sources, objs)))
        tmp = out + f".tmp{os.getpid()}"
        _run([hipcc, "--offload-arch=gfx950", "-fPIC", "-shared", "-o", tmp, *objs], verbose)
        os.replace(tmp, out)


def build(verbose: bool = False) -> str:
    _compile(LIB, SOURCES, verbose)
    _compile(PROBE_LIB, PROBE_SOURCES, verbose)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
