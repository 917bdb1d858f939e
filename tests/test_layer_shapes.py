"""The widths that the norms' GPU tests run reach every shape that the kernels are made for, with rows that
are whole vectors and rows that end inside one (mapped here, without a GPU)."""
import os
import re

import pytest

from conftest import ROOT
from test_gpu_layer_norms import WIDTHS, threads_of_a_row

CSRC = os.path.join(ROOT, "sharded_fsdp_flatten_amd", "csrc")


def made_for(name):
    """(threads, vectors) of every FSDP_SHAPE in a source file"""
    with open(os.path.join(CSRC, name)) as f:
        return {(int(a), int(b)) for a, b in re.findall(r"FSDP_SHAPE\((\d+), (\d+)\)", f.read())}


def forward(cols):
    nv = -(-cols // 8)
    if nv <= 256:
        return 64, -(-nv // 64)
    return (256, -(-nv // 256)) if nv <= 1536 else (512, 4)


@pytest.mark.parametrize("name,shape,vector", [("layer.hip", forward, 8), ("norm_backward.h", threads_of_a_row, 4)])
def test_every_shape_is_tested(name, shape, vector):
    want = made_for(name)
    assert len(want) >= 10
    for whole in (True, False):
        assert {shape(c) for c in WIDTHS if (c % vector == 0) == whole} == want, (name, whole)
    assert {shape(c) for c in range(8, 16385)} == want
