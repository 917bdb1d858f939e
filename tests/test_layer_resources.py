"""Registers of the layer operators' kernels as they were compiled: the norms' backward pass launches as
many workgroups as the device holds at once, which needs what its rule counts on (no GPU needed: the
numbers are in the library's own kernel descriptions)."""
import os
import re
import shutil
import struct
import subprocess

import pytest

from sharded_fsdp_flatten_amd import binding as B

LLVM = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin")


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """{demangled name: {"vgprs", "spills", "threads"}} of every kernel in the library."""
    if not os.path.exists(B.LIB_PATH):
        from sharded_fsdp_flatten_amd import build
        build.build()
    readelf = os.path.join(LLVM, "llvm-readelf")
    filt = shutil.which("c++filt") or os.path.join(LLVM, "llvm-cxxfilt")
    if not os.path.exists(readelf) or not os.path.exists(filt):
        pytest.skip("no llvm-readelf or c++filt here")
    with open(B.LIB_PATH, "rb") as f:
        lib = f.read()
    magic, at, out = b"__CLANG_OFFLOAD_BUNDLE__", 0, {}
    d = tmp_path_factory.mktemp("objects")
    while (at := lib.find(magic, at)) >= 0:
        # a bundle: magic, number of entries, then offset, size and target of each
        p = at + len(magic)
        n, = struct.unpack_from("<Q", lib, p)
        p += 8
        for _ in range(n if n < 16 else 0):
            offset, size, name = struct.unpack_from("<QQQ", lib, p)
            target = lib[p + 24:p + 24 + name]
            p += 24 + name
            if target.endswith(b"gfx950") and size:
                path = d / ("%d.o" % len(os.listdir(d)))
                path.write_bytes(lib[at + offset:at + offset + size])
                text = subprocess.run([readelf, "--notes", str(path)], stdout=subprocess.PIPE, text=True, check=True).stdout
                for k in text.split("\n  - ")[1:]:
                    v = dict(re.findall(r"\.(name|vgpr_count|vgpr_spill_count|max_flat_workgroup_size):\s+(\S+)", k))
                    if "vgpr_count" in v:
                        out[v["name"]] = dict(vgprs=int(v["vgpr_count"]), spills=int(v["vgpr_spill_count"]),
                                              threads=int(v["max_flat_workgroup_size"]))
        at += len(magic)
    plain = subprocess.run([filt], input="\n".join(out), stdout=subprocess.PIPE, text=True, check=True).stdout.split("\n")
    return dict(zip(plain, out.values()))


def backward(kernels):
    """(type, source, residual, threads of a row, its vectors, description) of the norms' backward kernels."""
    for name, k in kernels.items():
        m = re.search(r"norm_bwd_kernel<([a-z ]+), (\d), (\w+), \w+, (\d+), (\d), \w+>", name)
        if m:
            t, src, res, threads, vectors = m.groups()
            yield t, int(src), res == "true", int(threads), int(vectors), k


def test_norm_backward_workgroups_are_all_resident(kernels):
    """A SIMD has 512 registers a lane: two workgroups of 8 waves a CU need 128 at most, one of 8 waves
    256, one of 16 waves 128.  Only a row's three vectors with a residual gradient, in fp32 or from a
    checkpoint, are launched one workgroup a CU."""
    seen = 0
    for t, src, res, threads, vectors, k in backward(kernels):
        one = threads <= 512 and vectors == 3 and res and (t == "float" or src)
        assert k["threads"] == max(threads, 512)
        assert k["vgprs"] <= (256 if one else 128), (t, src, res, threads, vectors, k)
        seen += 1
    assert seen == 2 * 3 * 2 * 2 * 12 * 2   # types, sources, residual, load policies, shapes, whole or not


def test_only_the_longest_rows_spill(kernels):
    for name, k in kernels.items():
        m = re.search(r"norm_bwd_kernel<.*, 1024, [34], \w+>", name)
        assert m or k["spills"] == 0, (name, k)
