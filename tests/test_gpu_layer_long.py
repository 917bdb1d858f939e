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


# ---------------------------------------------------------------------------
# the norms past the cache
# ---------------------------------------------------------------------------
def aligned(cols, dtype):
    """columns to add so that rows start on 16-byte boundaries"""
    return -cols % (8 if dtype == torch.bfloat16 else 4)


def parameters(cols, dtype):
    return rand(5, 1, cols, 0.3, dtype=dtype)[0].add_(1), rand(6, 1, cols, dtype=dtype)[0]


@pytest.mark.parametrize("cols", [520, 1280, 1600, 2504, 4096, 10240, 12288, 14336])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_forward_past_the_cache(cols, residual):
    """Non-temporal loads, with a residual and its sum and without, and a checkpoint: the same rows in
    parts of a call that loads through the cache."""
    rows, part = (210 << 20) // (4 * cols) + 7, 777
    x, w = rand(1, rows, cols), parameters(cols, torch.bfloat16)
    r = rand(2, rows, cols) if residual else None
    q = F.Ckpt.empty(rows, cols, "int8", device=dev())
    y, s = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(rows, device=dev()), torch.empty(rows, device=dev())
    F.fsdp_norm_forward(x, *w, y, mean, rstd, kind="layer", residual=r, sum=s if residual else None, ckpt=q)
    for at in (0, part, rows // 2, rows - part):
        cut = slice(at, at + part)
        p = F.Ckpt.empty(part, cols, "int8", device=dev())
        y2, s2 = torch.empty_like(x[cut]), torch.empty_like(x[cut])
        mean2, rstd2 = torch.empty(part, device=dev()), torch.empty(part, device=dev())
        F.fsdp_norm_forward(x[cut], *w, y2, mean2, rstd2, kind="layer", residual=r[cut] if residual else None,
                            sum=s2 if residual else None, ckpt=p)
        for a, b in ((y2, y), (mean2, mean), (rstd2, rstd), (p.codes, q.codes), (p.scales, q.scales)):
            assert torch.equal(a, b[cut])
        assert not residual or torch.equal(s2, s[cut])


@pytest.mark.parametrize("source", ["tensor", "e4m3", "int8"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", [200, 700, 1021, 1280, 1600, 2501, 4096, 5120, 8192, 10243, 14336, 16381])
def test_norm_backward_past_the_cache(cols, dtype, source):
    """The same of the backward pass, with and without a residual gradient (also one whose rows are off the
    16-byte boundaries) and the output again; weight and bias gradients against sums in 64 bits."""
    e, part = dtype.itemsize, 777
    rows = (210 << 20) // (3 * e * cols) + 7
    pad = aligned(cols, dtype)
    x, dy = rand(1, rows, cols, 1.0, pad, dtype), rand(2, rows, cols, 0.1, pad, dtype)
    w, b = parameters(cols, dtype)
    mean, rstd = rand(7, 1, rows, 0.1, dtype=torch.float32)[0], rand(8, 1, rows, 0.1, dtype=torch.float32)[0].add_(1)
    src, held = x, x
    if source != "tensor":
        src = F.Ckpt.empty(rows, cols, source, device=dev())
        F.fsdp_ckpt_pack(x, src)
        held = torch.empty_like(x)
        F.fsdp_ckpt_unpack(src, held)
    ws = torch.empty(F.fsdp_norm_workspace(rows, cols), device=dev())
    for kind, extra, again in (("layer", None, True), ("rms", pad, False), ("layer", pad + 1, True)):
        res = None if extra is None else rand(3, rows, cols, 0.1, extra, dtype)
        dx, y = torch.empty_like(x), torch.empty_like(x) if again else None
        dw, db = torch.empty(cols, device=dev()), torch.empty(cols, device=dev())
        F.fsdp_norm_backward(dy, src, w, mean, rstd, dx, dw, db, ws, kind=kind, dres=res, y=y, bias=b if again else None)
        for at in (0, rows // 2, rows - part):
            cut = slice(at, at + part)
            few = x[cut] if source == "tensor" else F.Ckpt(src.codes[cut], src.scales[cut], source)
            dx2, y2, dw2 = torch.empty_like(x[cut]), torch.empty_like(x[cut]), torch.empty(cols, device=dev())
            F.fsdp_norm_backward(dy[cut], few, w, mean[cut], rstd[cut], dx2, dw2, dw2.clone(), ws, kind=kind,
                                 dres=None if res is None else res[cut], y=y2 if again else None, bias=b if again else None)
            assert torch.equal(dx2, dx[cut]) and (not again or torch.equal(y2, y[cut]))
        m = mean[:, None].double() if kind == "layer" else 0.0
        terms = (held.double() - m) * rstd[:, None].double() * dy.double()
        # one rounding for each term added, and four of each term
        assert bool(((dw.double() - terms.sum(0)).abs() <= (rows + 4) * R.U * terms.abs().sum(0)).all())
        assert bool(((db.double() - dy.double().sum(0)).abs() <= rows * R.U * dy.double().abs().sum(0)).all())


# ---------------------------------------------------------------------------
# inputs that take several launches
# ---------------------------------------------------------------------------
def whole(seed, rows, cols, low, high, dtype=torch.bfloat16):
    g = torch.Generator(device=dev()).manual_seed(seed)
    return torch.randint(low, high, (rows, cols), device=dev(), generator=g, dtype=torch.int8).to(dtype)


@pytest.mark.parametrize("cols", [3, 8])
def test_norms_of_more_rows_than_a_launch(cols):
    """2^22 rows a launch of the forward pass, and of the backward pass's means where a row is shorter than
    a vector: the last rows, which lie on both sides of the cut, and others against small calls, column sums of
    whole numbers."""
    rows, part = (1 << 22) + 5, 300
    x, r, dy = whole(1, rows, cols, -3, 4), whole(2, rows, cols, -3, 4), whole(3, rows, cols, -1, 2)
    w, b = parameters(cols, torch.float32)
    q = F.Ckpt.empty(rows, cols, "int8", device=dev())
    y, s, dx = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(rows, device=dev()), torch.empty(rows, device=dev())
    F.fsdp_norm_forward(x, w, b, y, mean, rstd, kind="layer", residual=r, sum=s, ckpt=q)
    assert torch.equal(s, x + r)
    back = torch.empty_like(x)
    F.fsdp_ckpt_unpack(q, back)
    assert torch.equal(back, s)
    ws = torch.empty(F.fsdp_norm_workspace(rows, cols), device=dev())
    ones, zeros = torch.ones(rows, device=dev()), torch.zeros(rows, device=dev())
    dw, db, again = torch.empty(cols, device=dev()), torch.empty(cols, device=dev()), torch.empty_like(x)
    F.fsdp_norm_backward(dy, q, w, mean, rstd, dx, dw, db, ws, kind="layer", dres=r, y=again, bias=b)
    for at in (0, rows // 2, rows - part):
        cut = slice(at, at + part)
        p = F.Ckpt(q.codes[cut], q.scales[cut], "int8")
        y2, dx2, again2, dw2 = torch.empty_like(x[cut]), torch.empty_like(x[cut]), torch.empty_like(x[cut]), dw.clone()
        mean2, rstd2 = torch.empty(part, device=dev()), torch.empty(part, device=dev())
        F.fsdp_norm_forward(x[cut], w, b, y2, mean2, rstd2, kind="layer", residual=r[cut])
        F.fsdp_norm_backward(dy[cut], p, w, mean2, rstd2, dx2, dw2, dw2.clone(), ws, kind="layer", dres=r[cut], y=again2, bias=b)
        for u, v in ((y2, y), (mean2, mean), (rstd2, rstd), (dx2, dx), (again2, again)):
            assert torch.equal(u, v[cut])
    # dy adds up to less than 2^24 on the way: exact; and so does dy (s - 0) 1
    assert torch.equal(db.double(), dy.double().sum(0))
    F.fsdp_norm_backward(dy, s, w, zeros, ones, dx, dw, db, ws, kind="layer")
    assert torch.equal(dw.double(), (dy.double() * s.double()).sum(0)) and torch.equal(db.double(), dy.double().sum(0))


def test_act_forward_and_checkpoints_of_more_rows_than_a_launch():
    """One column: 2^28 rows a launch, 2^30 where only a checkpoint is written or read."""
    rows = (1 << 30) + 5
    x = whole(1, rows, 1, -3, 4)
    q = F.Ckpt.empty(rows, 1, "int8", device=dev())
    back = torch.empty_like(x)
    F.fsdp_ckpt_pack(x, q)
    F.fsdp_ckpt_unpack(q, back)
    assert torch.equal(back, x)
    n = (1 << 28) + 5
    y, p = torch.empty_like(x[:n]), F.Ckpt(q.codes[:n].zero_(), q.scales[:n].zero_(), "int8")
    F.fsdp_act_forward(x[-n:], y, kind="relu", ckpt=p)
    assert torch.equal(y, x[-n:].clamp(min=0))
    F.fsdp_ckpt_unpack(p, back[:n])
    assert torch.equal(back[:n], x[-n:])


@pytest.mark.parametrize("source", ["tensor", "int8"])
def test_act_backward_of_more_rows_than_a_launch(source):
    """One column: 2^29 rows a launch, whose partial sums follow those of the launch before."""
    rows = (1 << 29) + 300
    x, dy = whole(1, rows, 1, -3, 4), whole(2, rows, 1, -1, 2)
    src = x
    if source != "tensor":
        src = F.Ckpt.empty(rows, 1, source, device=dev())
        F.fsdp_ckpt_pack(x, src)
    dx, y = torch.empty_like(x), torch.empty_like(x)
    base = torch.full((F.fsdp_act_workspace(rows, 1) + 64,), 7.0, device=dev())
    db = torch.full((65,), 7.0, device=dev())
    F.fsdp_act_backward(dy, src, dx, db[:1], base[:-64], kind="relu", y=y)
    want = dy * (x > 0)
    assert torch.equal(dx, want) and torch.equal(y, x.clamp(min=0))
    # whole numbers of small sums: exact in any order
    assert float(db[0]) == float(want.double().sum())
    assert bool((db[1:] == 7).all() and (base[-64:] == 7).all())
