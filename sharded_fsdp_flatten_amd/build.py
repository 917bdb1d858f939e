"""Build libfsdpflat.so (the C-ABI library) in-tree with hipcc for gfx950, and
libfsdpprobe.so (hardware floor probes the benchmark times beside the library;
not part of the data path).

    python -m sharded_fsdp_flatten_amd.build

Flags that matter for results:
  -ffp-contract=off        every float operation rounds on its own (no FMA),
                           matching the CPU oracle's operation order;
  -Xclang -target-feature -Xclang -packed-fp32-ops
                           no packed-fp32 instructions are generated;
  no -ffast-math / -fgpu-flush-denormals-to-zero: IEEE division, square root
                           and subnormals.
A flag that matters for speed only:
  -mllvm -amdgpu-kernarg-preload-count=16
                           the first 16 dwords of a kernel's scalar arguments
                           arrive preloaded in scalar registers (the copy engine,
                           AdamW and the sums of squares pass what a workgroup
                           needs first that way), so a short-lived workgroup
                           issues its loads without waiting for a scalar load.
"""
from __future__ import annotations

import concurrent.futures
import os
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_NAME = "libfsdpflat.so"
LIB_PATH = os.path.join(HERE, LIB_NAME)

SOURCES = ["norm_backward_bf16.hip", "norm_backward_f32.hip", "norm_backward_bf16_nt.hip",
           "norm_backward_f32_nt.hip", "layer.hip", "kernels.hip", "rotary.hip", "logprob.hip",
           "adam_tensors.hip", "plan.cpp", "fsdp_abi.cpp"]
PROBE_LIB_PATH = os.path.join(HERE, "libfsdpprobe.so")
PROBE_SOURCES = ["probes.hip"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-ffp-contract=off",
    "-fno-fast-math",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-mllvm", "-amdgpu-kernarg-preload-count=16",
    "-Wall",
    "-Wno-unused-command-line-argument",
    "-fvisibility=hidden",
]


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    proc = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if proc.returncode != 0:
        sys.stderr.write(proc.stdout)
        raise RuntimeError("hipcc failed: %s" % " ".join(cmd[-3:]))


def _link(sources, path, verbose):
    """Compile the sources side by side and link them into the shared library at `path`."""
    tmp = path + ".tmp%d" % os.getpid()
    with tempfile.TemporaryDirectory() as d:
        objects = [os.path.join(d, s + ".o") for s in sources]
        compile_one = lambda so: _run([HIPCC, *FLAGS, "-I", INCLUDE, "-I", CSRC, "-c",  # noqa: E731
                                       os.path.join(CSRC, so[0]), "-o", so[1]], verbose)
        with concurrent.futures.ThreadPoolExecutor(max_workers=8) as pool:
            list(pool.map(compile_one, zip(sources, objects)))
        _run([HIPCC, *FLAGS, "-shared", *objects, "-o", tmp], verbose)
    os.replace(tmp, path)


def build(verbose: bool = False) -> str:
    _link(SOURCES, LIB_PATH, verbose)
    _link(PROBE_SOURCES, PROBE_LIB_PATH, verbose)
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose=True))
