"""The layer operators where a call's size changes how it runs: loads past the cache, and inputs that go in
several launches.  What the kernels give there is compared with the same rows in small calls, bit for bit,
or with torch on the GPU where that is exact."""
import gc

import pytest
import torch

import layer_ref as R
import sharded_fsdp_flatten_amd as F
from gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _free():
    F.load()
    yield
    gc.collect()
    torch.cuda.empty_cache()


def rand(seed, rows, cols, scale=1.0, pad=0, dtype=torch.bfloat16):
    g = torch.Generator(device=dev()).manual_seed(seed)
    t = torch.empty(rows, cols + pad, dtype=dtype, device=dev())
    return t.normal_(0, scale, generator=g)[:, :cols]


@pytest.mark.parametrize("source", ["tensor", "e4m3", "int8"])
@pytest.mark.parametrize("kind", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("cols,pad", [(8192, 0), (8195, 5), (8195, 4)])
def test_act_backward_past_the_cache(cols, pad, kind, source):
    """400 MB a call: non-temporal loads where the rows start on 16-byte boundaries, also of a width that
    ends inside a vector; parts of 1000 rows take the cached loads."""
    rows, part = 8193, 1000
    x, dy = rand(1, rows, cols, 3.0, pad), rand(2, rows, cols, 1.0, pad)
    src = x
    if source != "tensor":
        src = F.Ckpt.empty(rows, cols, source, device=dev())
        F.fsdp_ckpt_pack(x, src)
    dx, y = torch.empty_like(x), torch.empty_like(x)
    db = torch.empty(cols, device=dev())
    ws = torch.empty(F.fsdp_act_workspace(rows, cols), device=dev())
    F.fsdp_act_backward(dy, src, dx, db, ws, kind=kind, y=y)
    total, size = torch.zeros(cols, device=dev(), dtype=torch.float64), torch.zeros(cols, device=dev(), dtype=torch.float64)
    for at in range(0, rows, part):
        n = min(part, rows - at)
        few = x[at:at + n] if source == "tensor" else F.Ckpt(src.codes[at:at + n], src.scales[at:at + n], source)
        dx2, y2, db2 = torch.empty_like(dx[at:at + n]), torch.empty_like(y[at:at + n]), torch.empty_like(db)
        F.fsdp_act_backward(dy[at:at + n], few, dx2, db2, ws, kind=kind, y=y2)
        assert torch.equal(dx2, dx[at:at + n]) and torch.equal(y2, y[at:at + n])
        total += db2.double()
        size += dx2.double().abs().sum(0)
    # both sums are in binary32; dx was rounded to bf16 behind them, which makes its size 2^-8 less at most
    assert bool(((db.double() - total).abs() <= 2 * rows * R.U * size * (1 + 2 ** -7)).all())
