"""The layer operators on the GPU against a plain 64-bit reference (layer_ref.py): 8-bit
checkpoints bit for bit, the norms and activations within the rounding errors that their binary32
arithmetic can make (bounds computed from the inputs), at sizes where rows end inside a vector or a
group, start at any element, are very short, very long, or none at all."""
import gc

import numpy as np
import pytest
import torch

import layer_ref as R
import sharded_fsdp_flatten_amd as F
from gpu_util import dev

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def _free():
    F.load()
    yield
    gc.collect()
    torch.cuda.empty_cache()


def f64(t):
    return t.detach().double().cpu().numpy()


class Guarded:
    """A rows x cols matrix inside a larger allocation: rows `pitch` apart from element `start`
    on, everything around them holding a pattern that must stay."""

    def __init__(self, rows, cols, dtype, pitch=None, start=0):
        pitch = cols if pitch is None else pitch
        self.base = torch.full((start + max(rows, 1) * pitch + 64,), 7, dtype=dtype, device=dev())
        self.t = self.base.as_strided((rows, cols), (pitch, 1), start)

    def around_is_untouched(self):
        b = self.base.clone()
        b.as_strided(self.t.shape, self.t.stride(), self.t.storage_offset()).fill_(7)
        return bool((b == 7).all())


def guarded(value, pitch=None, start=0):
    g = Guarded(value.shape[0], value.shape[1], value.dtype, pitch, start)
    g.t.copy_(value)
    return g


def close(got, want, bound, what):
    got = f64(got)
    bad = ~((np.abs(got - want) <= bound) | (np.isnan(got) & np.isnan(want)) | (got == want))
    assert not bad.any(), "%s: %d of %d beyond the bound; first at %s: got %r want %r bound %r" % (
        what, bad.sum(), bad.size, np.argwhere(bad)[0], got[bad][0], np.asarray(want)[bad][0],
        np.broadcast_to(bound, got.shape)[bad][0])


def normal(seed, *shape, scale=1.0):
    g = torch.Generator(device="cpu").manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale)


# ---------------------------------------------------------------------------
# checkpoints
# ---------------------------------------------------------------------------
SHAPES = [(1, 1), (1, 7), (2, 8), (3, 31), (5, 32), (4, 33), (65, 64), (9, 257), (33, 1280),
          (7, 2051), (3, 5003), (2, 12288), (1, 70001)]


def spread(seed, rows, cols, t):
    """values over many binades, with zeros"""
    x = normal(seed, rows, cols) * torch.exp(4 * normal(seed + 1, rows, cols))
    x[torch.rand(rows, cols, generator=torch.Generator().manual_seed(seed + 2)) < 0.1] = 0
    return x.to(t).to(dev())


def check_ckpt(x, fmt, pitch=0, start=0):
    rows, cols = x.shape
    groups = -(-cols // 32)
    codes = Guarded(rows, cols, torch.uint8, cols + pitch, start)
    scales = Guarded(rows, groups, torch.uint8, groups + pitch, start)
    q = F.Ckpt(codes.t, scales.t, fmt)
    F.fsdp_ckpt_pack(x, q)
    want, byte = R.ckpt(f64(x), fmt)
    got_byte = scales.t.cpu().numpy()
    assert np.array_equal(got_byte, byte)
    finite = byte != 255
    held = R.code_values(fmt)[codes.t.cpu().numpy()]
    each = np.repeat(byte.astype(float), 32, 1)[:, :cols]
    with np.errstate(over="ignore", invalid="ignore"):
        value = np.where(np.repeat(finite, 32, 1)[:, :cols], held * 2.0 ** (each - 127), np.nan)
    assert np.array_equal(value, want, equal_nan=True)
    for t in ("bf16", "f32"):
        back = Guarded(rows, cols, T[t], cols + pitch, start)
        F.fsdp_ckpt_unpack(q, back.t)
        with np.errstate(over="ignore"):
            as_t = want.astype(np.float32).astype(float)
        assert np.array_equal(f64(back.t), as_t, equal_nan=True), t
        assert back.around_is_untouched()
    assert codes.around_is_untouched() and scales.around_is_untouched()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_ckpt_bits(rows, cols, t, fmt):
    check_ckpt(spread(rows * 131 + cols, rows, cols, T[t]), fmt)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_ckpt_pitches_and_starts(t, fmt):
    x = guarded(spread(5, 37, 195, T[t]), 203, 3)
    check_ckpt(x.t, fmt, pitch=5, start=1)
    assert x.around_is_untouched()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_ckpt_borders_and_special_values(t, fmt):
    """Largest magnitudes at and next to the scale's borders, ties between codes, signed zeros,
    subnormals, the type's largest value, and groups with an infinity or a NaN."""
    rows = []
    for top in (463.0, 464.0, 465.0, 466.0, 448.0, 256.0, 511.0, 127.0, 127.25, 127.5, 127.75, 64.0, 1.0):
        for k in (0, -100, 100, -126, -133):
            r = np.zeros(64)
            r[:32] = np.arange(32) * 0.5 * (1 if top > 16 else 1 / 64)
            r[5] = -top
            r[32:] = np.linspace(-top, top, 32)
            rows.append(r * 2.0 ** k)
    for k in range(-10, 1):                      # ties of e4m3, all its subnormals among them
        r = np.zeros(64)
        r[0] = 448
        r[1:64] = np.arange(1, 64) * 2.0 ** k
        rows.append(r)
    big = float(torch.finfo(T[t]).max)
    tiny = float(torch.finfo(T[t]).tiny)
    for v in (big, 1.75 * 2.0 ** 127, 2.0 ** 127, tiny, tiny / 2, tiny / 64, -0.0, 0.0):
        rows.append(np.full(64, v))
    for v in (np.inf, -np.inf, np.nan):
        r = np.linspace(-1, 1, 64)
        r[40] = v
        rows.append(r)
    with np.errstate(over="ignore"):
        x = torch.from_numpy(np.array(rows)).float().to(T[t])
    assert not torch.isinf(x[:-3]).any()
    check_ckpt(x.to(dev()), fmt)


def test_ckpt_of_nothing():
    for rows, cols in ((0, 5), (3, 0), (0, 0)):
        x = torch.empty(rows, cols, device=dev())
        q = F.Ckpt.empty(rows, cols, "int8", device=dev())
        F.fsdp_ckpt_pack(x, q)
        F.fsdp_ckpt_unpack(q, x)
    torch.cuda.synchronize()


def test_ckpt_more_than_4_gib_of_codes():
    """Offsets past 32 bits: the last rows of 2^22 + 3 rows of 1056 columns."""
    rows, cols = (1 << 22) + 3, 1056
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device=dev())
    x[:2] = normal(1, 2, cols).to(dev())
    tail = normal(2, 700, cols).bfloat16().to(dev())
    x[2:-700] = 1.5
    x[-700:] = tail
    q = F.Ckpt.empty(rows, cols, "e4m3", device=dev())
    back = torch.empty_like(x)
    F.fsdp_ckpt_pack(x, q)
    F.fsdp_ckpt_unpack(q, back)
    want, byte = R.ckpt(f64(tail), "e4m3")
    assert np.array_equal(f64(back[-700:]), want)
    assert np.array_equal(q.scales[-700:].cpu().numpy(), byte)
    assert bool((back[2:-700] == 1.5).all())


# ---------------------------------------------------------------------------
# norms
# ---------------------------------------------------------------------------
EPS = 1e-5


def norm_inputs(seed, rows, cols, t, pt, bias=True):
    x = (normal(seed, rows, cols) * torch.exp(0.5 * normal(seed + 1, rows, 1)) + normal(seed + 2, 1, cols)).to(T[t]).to(dev())
    w = (1 + 0.3 * normal(seed + 3, cols)).to(T[pt]).to(dev())
    b = normal(seed + 4, cols).to(T[pt]).to(dev()) if bias else None
    return x, w, b


def stats(rows):
    return torch.full((rows,), 7.0, device=dev()), torch.full((rows,), 7.0, device=dev())


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("t,pt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("rows,cols", SHAPES + [(1, 1024), (130, 512), (6, 1536), (5, 4100), (3, 8192), (2, 16385), (3, 33000)])
def test_norm_forward(rows, cols, t, pt, kind):
    x, w, b = norm_inputs(rows + cols, rows, cols, t, pt, bias=kind == "layer")
    y = Guarded(rows, cols, T[t])
    mean, rstd = stats(rows)
    F.fsdp_norm_forward(x, w, b, y.t, mean if kind == "layer" else None, rstd, kind=kind, eps=EPS)
    r = R.norm(f64(x), f64(w), None if b is None else f64(b), kind, EPS, t)
    close(rstd, r["rstd"], r["erstd"], "rstd")
    if kind == "layer":
        close(mean, r["mean"], r["emean"], "mean")
    close(y.t, r["y"], r["ey"], "y")
    assert y.around_is_untouched()


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,pad", [(37, 195, 5), (19, 1280, 0), (9, 2500, 1), (5, 5003, 3), (2, 66000, 7)])
def test_norm_forward_residual_ckpt_and_pitches(rows, cols, pad, t, kind):
    x, w, b = norm_inputs(rows * 7 + cols, rows, cols, t, t)
    res = normal(9, rows, cols).to(T[t]).to(dev())
    xs, rs = guarded(x, cols + pad, 1), guarded(res, cols + 2 * pad, 2)
    y, s = Guarded(rows, cols, T[t], cols + pad, 3), Guarded(rows, cols, T[t], cols + 3 * pad, 1)
    mean, rstd = stats(rows)
    q = F.Ckpt.empty(rows, cols, "e4m3" if kind == "layer" else "int8", device=dev())
    F.fsdp_norm_forward(xs.t, w, b, y.t, mean, rstd, kind=kind, eps=EPS, residual=rs.t, sum=s.t, ckpt=q)
    want_sum = (x.float() + res.float()).to(T[t])
    assert torch.equal(s.t, want_sum)
    r = R.norm(f64(want_sum), f64(w), f64(b), kind, EPS, t)
    close(y.t, r["y"], r["ey"], "y")
    close(rstd, r["rstd"], r["erstd"], "rstd")
    for g in (xs, rs, y, s):
        assert g.around_is_untouched()
    back = torch.empty_like(want_sum)
    F.fsdp_ckpt_unpack(q, back)
    assert np.array_equal(f64(back), R.ckpt(f64(want_sum), q.format)[0])
    # the sum need not be stored
    y2 = torch.empty_like(x)
    F.fsdp_norm_forward(x, w, b, y2, mean, rstd, kind=kind, eps=EPS, residual=res)
    assert torch.equal(y2, y.t)


def test_norm_forward_large_mean():
    """Rows whose mean is far above their spread: the variance is that of the differences."""
    x = (1000 + normal(3, 8, 1280)).to(dev())
    w = torch.ones(1280, device=dev())
    mean, rstd = stats(8)
    y = torch.empty_like(x)
    F.fsdp_norm_forward(x, w, None, y, mean, rstd, kind="layer", eps=EPS)
    r = R.norm(f64(x), f64(w), None, "layer", EPS, "f32")
    close(rstd, r["rstd"], r["erstd"], "rstd")
    close(y, r["y"], r["ey"], "y")


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_rows_are_their_own(kind):
    """A row of NaN or infinities, and rows of zeros, leave the other rows as they are."""
    x, w, b = norm_inputs(4, 6, 1280, "bf16", "bf16")
    ref = torch.empty_like(x)
    mean, rstd = stats(6)
    F.fsdp_norm_forward(x, w, b, ref, mean, rstd, kind=kind, eps=EPS)
    x2 = x.clone()
    x2[1] = float("nan")
    x2[3, 77] = float("inf")
    x2[4] = 0
    y = torch.empty_like(x)
    F.fsdp_norm_forward(x2, w, b, y, mean, rstd, kind=kind, eps=EPS)
    for i in (0, 2, 5):
        assert torch.equal(y[i], ref[i])
    assert torch.isnan(y[1]).all() and torch.isnan(y[3, 77])
    assert torch.equal(y[4], b)


def run_backward(dy, src, w, mean, rstd, kind, t, gt="f32", dres=None, b=None, again=False,
                 dw0=None, db0=None, pad=0):
    rows, cols = dy.shape
    dx = Guarded(rows, cols, T[t], cols + pad, pad)
    y = Guarded(rows, cols, T[t], cols + pad, pad) if again else None
    dw = torch.full((cols,), 7.0, dtype=T[gt], device=dev()) if dw0 is None else dw0.clone()
    db = torch.full((cols,), 7.0, dtype=T[gt], device=dev()) if db0 is None else db0.clone()
    ws = Guarded(1, max(1, F.fsdp_norm_workspace(rows, cols)), torch.float32)
    F.fsdp_norm_backward(dy, src, w, mean, rstd, dx.t, dw, db, ws.t[0], kind=kind, dres=dres,
                         y=y.t if again else None, bias=b, accumulate=dw0 is not None)
    assert dx.around_is_untouched() and (not again or y.around_is_untouched()) and ws.around_is_untouched()
    return dx.t, dw, db, y.t if again else None


def given_stats(x, kind):
    x64 = x.double()
    m = x64.mean(1) if kind == "layer" else torch.zeros(x.shape[0], device=dev(), dtype=torch.float64)
    return m.float(), ((x64 - m[:, None]).square().mean(1) + EPS).rsqrt().float()


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("t,pt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("rows,cols", SHAPES + [(1, 1024), (300, 512), (6, 1536), (257, 96), (40, 4100), (3, 8192),
                                                (700, 3), (5, 16385), (3, 33000)])
def test_norm_backward(rows, cols, t, pt, kind):
    x, w, b = norm_inputs(rows + cols, rows, cols, t, pt)
    dy = normal(50, rows, cols, scale=0.1).to(T[t]).to(dev())
    mean, rstd = given_stats(x, kind)
    dx, dw, db, _ = run_backward(dy, x, w, mean, rstd, kind, t)
    r = R.norm_grads(f64(dy), f64(x), f64(w), None, f64(mean), f64(rstd), kind, t)
    close(dx, r["dx"], r["edx"], "dx")
    close(dw, r["dw"], r["edw"], "dw")
    close(db, r["db"], r["edb"], "db")


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,pad", [(41, 195, 5), (70, 1280, 0), (9, 2500, 1), (5, 5003, 3), (6, 12288, 8), (2, 66000, 7)])
def test_norm_backward_from_ckpt(rows, cols, pad, t, fmt, kind):
    """From the checkpoint, with the residual stream's gradient, the output again, and sums added
    to bf16 or fp32 gradients."""
    x, w, b = norm_inputs(rows + cols, rows, cols, t, t)
    dy = guarded(normal(50, rows, cols, scale=0.1).to(T[t]).to(dev()), cols + pad, 1)
    dres = guarded(normal(51, rows, cols, scale=0.1).to(T[t]).to(dev()), cols + 2 * pad, 3)
    mean, rstd = given_stats(x, kind)
    q = F.Ckpt.empty(rows, cols, fmt, device=dev())
    F.fsdp_ckpt_pack(x, q)
    held = R.ckpt(f64(x), fmt)[0]
    gt = t
    dw0, db0 = (normal(60 + i, cols).to(T[gt]).to(dev()) for i in (0, 1))
    dx, dw, db, y = run_backward(dy.t, q, w, mean, rstd, kind, t, gt, dres.t, b, True, dw0, db0, pad)
    r = R.norm_grads(f64(dy.t), held, f64(w), f64(b), f64(mean), f64(rstd), kind, t, f64(dres.t))
    close(dx, r["dx"], r["edx"], "dx")
    close(y, r["y"], r["ey"], "y")
    for got, start, want, e, what in ((dw, dw0, r["dw"], r["edw"], "dw"), (db, db0, r["db"], r["edb"], "db")):
        total = f64(start) + want
        e = e + R.U * np.abs(total)
        close(got, total, e + (np.abs(total) + e) * R.HALF[gt], what)
    assert dy.around_is_untouched() and dres.around_is_untouched()


@pytest.mark.parametrize("rows,cols", [(20000, 40), (9001, 1280), (2049, 5000)])
def test_norm_backward_column_sums_miss_no_row(rows, cols):
    """Small whole numbers: dy's column sums are exact in fp32, so db is exact; x = mean +- 1 and
    rstd = 1 make xh whole, and dw exact too."""
    g = torch.Generator().manual_seed(rows)
    dy = torch.randint(-4, 5, (rows, cols), generator=g).bfloat16().to(dev())
    x = torch.randint(-3, 4, (rows, cols), generator=g).bfloat16().to(dev())
    w = torch.ones(cols, device=dev())
    mean, rstd = torch.zeros(rows, device=dev()), torch.ones(rows, device=dev())
    _, dw, db, _ = run_backward(dy, x, w, mean, rstd, "layer", "bf16")
    assert torch.equal(db.double(), dy.double().sum(0))
    assert torch.equal(dw.double(), (dy.double() * x.double()).sum(0))


def test_norm_backward_either_gradient_alone_and_none():
    x, w, _ = norm_inputs(1, 50, 1280, "bf16", "bf16")
    dy = normal(2, 50, 1280).bfloat16().to(dev())
    mean, rstd = given_stats(x, "layer")
    dx, dw, db, _ = run_backward(dy, x, w, mean, rstd, "layer", "bf16")
    ws = torch.empty(F.fsdp_norm_workspace(50, 1280), device=dev())
    for want_w, want_b in ((True, False), (False, True), (False, False)):
        dx2, dw2, db2 = torch.empty_like(dx), torch.full_like(dw, 7), torch.full_like(db, 7)
        F.fsdp_norm_backward(dy, x, w, mean, rstd, dx2, dw2 if want_w else None,
                             db2 if want_b else None, ws, kind="layer")
        assert torch.equal(dx2, dx)
        assert torch.equal(dw2, dw if want_w else torch.full_like(dw, 7))
        assert torch.equal(db2, db if want_b else torch.full_like(db, 7))


def test_norm_of_no_rows():
    """No rows: nothing is touched, the gradients are sums of nothing."""
    w, b = torch.ones(100, device=dev()), torch.zeros(100, device=dev())
    e, z = torch.empty(0, 100, device=dev()), torch.empty(0, device=dev())
    F.fsdp_norm_forward(e, w, b, e.clone(), z, z.clone(), kind="layer")
    dw, db = torch.full((100,), 7.0, device=dev()), torch.full((100,), 7.0, device=dev())
    F.fsdp_norm_backward(e, e, w, z, z, e.clone(), dw, db, None, kind="layer", accumulate=True)
    assert bool((dw == 7).all() and (db == 7).all())
    F.fsdp_norm_backward(e, e, w, z, z, e.clone(), dw, db, None, kind="layer")
    assert bool((dw == 0).all() and (db == 0).all())
    F.fsdp_act_backward(e, e, e.clone(), db.fill_(7), None, kind="gelu")
    assert bool((db == 0).all())
    n = torch.empty(3, 0, device=dev())
    v = torch.empty(0, device=dev())
    F.fsdp_norm_forward(n, v, None, n.clone(), torch.ones(3, device=dev()), torch.ones(3, device=dev()), kind="layer")
    F.fsdp_act_forward(n, n.clone(), kind="relu")
    torch.cuda.synchronize()


def test_norm_gradients_against_differences():
    """Central differences of sum(r * y) in 64 bits along random directions of x, w and b."""
    rows, cols = 6, 160
    for kind in ("layer", "rms"):
        x, w, b = norm_inputs(12, rows, cols, "f32", "f32")
        r = normal(13, rows, cols).to(dev())
        y = torch.empty_like(x)
        mean, rstd = stats(rows)
        F.fsdp_norm_forward(x, w, b, y, mean, rstd, kind=kind, eps=EPS)
        dx, dw, db, _ = run_backward(r, x, w, mean, rstd, kind, "f32")

        def loss(xx, ww, bb):
            return (f64(r) * R.norm(xx, ww, bb, kind, EPS, "f32")["y"]).sum()

        h = 1e-4
        X, W, Bb = f64(x), f64(w), f64(b)
        for i in range(4):
            vx, vw, vb = (normal(70 + 3 * i + j, *s).double().numpy() for j, s in enumerate(((rows, cols), (cols,), (cols,))))
            for got, lo, hi, v in ((dx, (X - h * vx, W, Bb), (X + h * vx, W, Bb), vx),
                                   (dw, (X, W - h * vw, Bb), (X, W + h * vw, Bb), vw),
                                   (db, (X, W, Bb - h * vb), (X, W, Bb + h * vb), vb)):
                want = (loss(*hi) - loss(*lo)) / (2 * h)
                size = np.abs(f64(got) * v).sum()
                # h^2 times third derivatives of order one, and fp32 gradients
                assert abs((f64(got) * v).sum() - want) <= (1e-6 + 64 * R.U) * size


@pytest.mark.parametrize("rows,cols,t", [(24577, 4096, "bf16"), (8193, 12288, "bf16"), (24001, 2500, "f32"), (49999, 4100, "bf16")])
def test_long_calls(rows, cols, t):
    """Past 192 MB the loads are non-temporal, and a long checkpoint takes several rows a lane:
    some rows at the start, the end and between against the reference, whole-number column sums
    exactly, and a checkpoint against the same rows packed a few at a time, bit for bit."""
    g = torch.Generator(device=dev()).manual_seed(rows)
    x = torch.randint(-3, 4, (rows, cols), device=dev(), generator=g).to(T[t])
    some = torch.cat([torch.arange(9), torch.randint(9, rows - 9, (14,), generator=torch.Generator().manual_seed(1)),
                      torch.arange(rows - 9, rows)]).to(dev())
    x[some] += normal(2, some.numel(), cols).to(T[t]).to(dev()).round(decimals=2)
    w, b = (normal(3 + i, cols).to(T[t]).to(dev()) for i in (0, 1))
    y, back = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = stats(rows)
    q, few = F.Ckpt.empty(rows, cols, "e4m3", device=dev()), F.Ckpt.empty(640, cols, "e4m3", device=dev())
    F.fsdp_norm_forward(x, w, b, y, mean, rstd, kind="layer", eps=EPS)
    r = R.norm(f64(x[some]), f64(w), f64(b), "layer", EPS, t)
    close(y[some], r["y"], r["ey"], "y")
    close(rstd[some], r["rstd"], r["erstd"], "rstd")
    F.fsdp_ckpt_pack(x, q)
    F.fsdp_ckpt_unpack(q, back)
    for at in (0, 640, rows - 640):
        F.fsdp_ckpt_pack(x[at:at + 640], few)
        assert torch.equal(few.codes, q.codes[at:at + 640]) and torch.equal(few.scales, q.scales[at:at + 640])
    assert np.array_equal(f64(back[some]), R.ckpt(f64(x[some]), "e4m3")[0])
    dy = torch.randint(-4, 5, (rows, cols), device=dev(), generator=g).to(T[t])
    mean.zero_(), rstd.fill_(1)
    dx = torch.empty_like(x)
    for src, held in ((x, x), (q, back)):
        dw, db = torch.empty(cols, device=dev()), torch.empty(cols, device=dev())
        ws = torch.empty(F.fsdp_norm_workspace(rows, cols), device=dev())
        F.fsdp_norm_backward(dy, src, w, mean, rstd, dx, dw, db, ws, kind="layer", y=y, bias=b, dres=x)
        assert torch.equal(db.double(), dy.double().sum(0))
        want = (dy.double() * held.double()).sum(0)
        bound = (rows + 4) * R.U * (dy.double() * held.double()).abs().sum(0)
        assert bool(((dw.double() - want).abs() <= bound).all())
        r = R.norm_grads(f64(dy[some]), f64(held[some]), f64(w), f64(b), f64(mean[some]), f64(rstd[some]), "layer", t, f64(x[some]))
        close(dx[some], r["dx"], r["edx"], "dx")
        close(y[some], r["y"], r["ey"], "y")
    dbias = torch.empty(cols, device=dev())
    wa = torch.empty(F.fsdp_act_workspace(rows, cols), device=dev())
    F.fsdp_act_forward(x, y, kind="relu")
    assert torch.equal(y, x.clamp(min=0))
    F.fsdp_act_backward(dy, x, dx, dbias, wa, kind="relu")
    assert torch.equal(dx, torch.where(x > 0, dy, torch.zeros_like(dy)))
    assert torch.equal(dbias.double(), dx.double().sum(0))


# ---------------------------------------------------------------------------
# activations
# ---------------------------------------------------------------------------
KINDS = ["relu", "gelu", "gelu_tanh", "silu"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_act_forward_and_backward(rows, cols, t, kind):
    x = (3 * normal(rows + cols, rows, cols)).to(T[t]).to(dev())
    dy = normal(8, rows, cols).to(T[t]).to(dev())
    y, dx = Guarded(rows, cols, T[t]), Guarded(rows, cols, T[t])
    F.fsdp_act_forward(x, y.t, kind=kind)
    f, d = R.act(f64(x), kind)
    ef, ed = R.act_bounds(f64(x), kind)
    close(y.t, f, ef + (np.abs(f) + ef) * R.HALF[t], "y")
    db = torch.full((cols,), 7.0, device=dev())
    ws = Guarded(1, F.fsdp_act_workspace(rows, cols), torch.float32)
    F.fsdp_act_backward(dy, x, dx.t, db, ws.t[0], kind=kind)
    g = f64(dy) * d
    eg = np.abs(f64(dy)) * ed + 2 * R.U * np.abs(g)
    close(dx.t, g, eg + (np.abs(g) + eg) * R.HALF[t], "dx")
    close(db, g.sum(0), eg.sum(0) + rows * R.U * np.abs(g).sum(0), "db")
    assert y.around_is_untouched() and dx.around_is_untouched() and ws.around_is_untouched()
    # without the bias's gradient no workspace is needed
    dx2 = torch.empty_like(x)
    F.fsdp_act_backward(dy, x, dx2, kind=kind)
    assert torch.equal(dx2, dx.t)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("t,gt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("rows,cols,pad", [(41, 195, 5), (70, 1280, 0), (9, 2500, 1)])
def test_act_backward_from_ckpt(rows, cols, pad, t, gt, fmt, kind):
    x = guarded((3 * normal(rows + cols, rows, cols)).to(T[t]).to(dev()), cols + pad, pad)
    dy = guarded(normal(8, rows, cols).to(T[t]).to(dev()), cols + 2 * pad, 1)
    y, dx, again = (Guarded(rows, cols, T[t], cols + pad, k) for k in (1, 2, 3))
    q = F.Ckpt.empty(rows, cols, fmt, device=dev())
    F.fsdp_act_forward(x.t, y.t, kind=kind, ckpt=q)
    held = R.ckpt(f64(x.t), fmt)[0]
    f, d = R.act(held, kind)
    ef, ed = R.act_bounds(held, kind)
    start = normal(4, cols).to(T[gt]).to(dev())
    db = start.clone()
    ws = torch.empty(F.fsdp_act_workspace(rows, cols), device=dev())
    F.fsdp_act_backward(dy.t, q, dx.t, db, ws, kind=kind, y=again.t, accumulate=True)
    g = f64(dy.t) * d
    eg = np.abs(f64(dy.t)) * ed + 2 * R.U * np.abs(g)
    close(dx.t, g, eg + (np.abs(g) + eg) * R.HALF[t], "dx")
    close(again.t, f, ef + (np.abs(f) + ef) * R.HALF[t], "y again")
    total = f64(start) + g.sum(0)
    e = eg.sum(0) + rows * R.U * np.abs(g).sum(0) + R.U * np.abs(total)
    close(db, total, e + (np.abs(total) + e) * R.HALF[gt], "db")
    for m in (x, dy, y, dx, again):
        assert m.around_is_untouched()


@pytest.mark.parametrize("kind", KINDS)
def test_act_far_values(kind):
    """Large arguments of either sign saturate: no NaN from an overflow inside the formulas."""
    h = torch.tensor([[0.0, -0.0, 1e-30, -1e-30, 6, -6, 12, -12, 40, -40, 1e4, -1e4, 1e13, -1e13, 3e38, -3e38]], device=dev())
    y, dx = torch.empty_like(h), torch.empty_like(h)
    F.fsdp_act_forward(h, y, kind=kind)
    F.fsdp_act_backward(torch.ones_like(h), h, dx, kind=kind)
    f, d = R.act(np.clip(f64(h), -60, 60), kind)
    f = np.where(f64(h) > 60, f64(h), f)
    ef, ed = R.act_bounds(np.clip(f64(h), -60, 60), kind)
    close(y, f, ef + np.abs(f) * 4 * R.U, "y")
    close(dx, d, ed + 4 * R.U, "dx")
    n = torch.full((1, 40), float("nan"), device=dev())
    F.fsdp_act_forward(n, y2 := torch.zeros_like(n), kind=kind)
    F.fsdp_act_backward(torch.ones_like(n), n, d2 := torch.zeros_like(n), kind=kind)
    assert torch.isnan(y2).all() and torch.isnan(d2).all()


def test_more_columns_than_one_column_sum_launch():
    rows, cols = 3, (1 << 26) + 41
    g = torch.Generator(device=dev()).manual_seed(5)
    x = torch.randint(-3, 4, (rows, cols), device=dev(), generator=g, dtype=torch.int8).to(torch.bfloat16)
    q = F.Ckpt.empty(rows, cols, "int8", device=dev())
    y, back = torch.empty_like(x), torch.empty_like(x)
    F.fsdp_act_forward(x, y, kind="relu", ckpt=q)
    F.fsdp_ckpt_unpack(q, back)
    assert torch.equal(back, x) and torch.equal(y, x.clamp(min=0))
    db = torch.full((cols + 64,), 7.0, device=dev())
    ws = torch.empty(F.fsdp_act_workspace(rows, cols), device=dev())
    F.fsdp_act_backward(x, q, y, db[:cols], ws, kind="relu")
    assert torch.equal(db[:cols], (x * (x > 0)).float().sum(0)) and bool((db[cols:] == 7).all())
    w = torch.ones(cols, dtype=torch.bfloat16, device=dev())
    mean, rstd = torch.zeros(rows, device=dev()), torch.ones(rows, device=dev())
    dw = torch.empty(cols, device=dev())
    ws = torch.empty(F.fsdp_norm_workspace(rows, cols), device=dev())
    F.fsdp_norm_backward(x, q, w, mean, rstd, y, dw, db[:cols], ws, kind="layer")
    assert torch.equal(dw, x.float().square().sum(0)) and torch.equal(db[:cols], x.float().sum(0))


# ---------------------------------------------------------------------------
# how they are called
# ---------------------------------------------------------------------------
def test_inputs_of_one_repeated_row_and_of_three_dimensions():
    """A broadcast gradient (row stride 0) is read as it stands; leading dimensions count as rows."""
    x, w, b = norm_inputs(3, 24, 320, "f32", "f32")
    row = normal(5, 320).to(dev())
    mean, rstd = given_stats(x, "layer")
    a = run_backward(row.expand(24, 320), x, w, mean, rstd, "layer", "f32")
    c = run_backward(row.expand(24, 320).contiguous(), x, w, mean, rstd, "layer", "f32")
    for u, v in zip(a[:3], c[:3]):
        assert torch.equal(u, v)
    y2, y3 = torch.empty_like(x), torch.empty(4, 6, 320, device=dev())
    F.fsdp_norm_forward(x, w, b, y2, mean, rstd, kind="layer")
    F.fsdp_norm_forward(x.view(4, 6, 320), w, b, y3, mean.view(4, 6), rstd.view(4, 6), kind="layer")
    assert torch.equal(y2, y3.view(24, 320))


def block_state(seed, tokens=520, d=640, t=torch.bfloat16):
    g = torch.Generator(device=dev()).manual_seed(seed)
    n = lambda *s, sc=1.0: (torch.randn(*s, device=dev(), generator=g) * sc)  # noqa: E731
    e = lambda *s, dt=t: torch.empty(*s, dtype=dt, device=dev())  # noqa: E731
    f = torch.float32
    return dict(x=n(tokens, d).to(t), res=n(tokens, d).to(t), w=(1 + n(d, sc=0.1)).to(t), b=n(d, sc=0.1).to(t),
                up=n(4 * d, d, sc=0.03).to(t), down=n(d, 4 * d, sc=0.02).to(t), bias=n(4 * d, sc=0.1).to(t),
                dout=n(tokens, d, sc=0.01).to(t), s=e(tokens, d), y=e(tokens, d), mean=e(tokens, dt=f),
                rstd=e(tokens, dt=f), qx=F.Ckpt.empty(tokens, d, "e4m3", device=dev()),
                qh=F.Ckpt.empty(tokens, 4 * d, "int8", device=dev()), a=e(tokens, 4 * d),
                dh=e(tokens, 4 * d), a2=e(tokens, 4 * d), y2=e(tokens, d), dx=e(tokens, d),
                dw=torch.zeros(d, device=dev()), db=torch.zeros(d, device=dev()), dbias=torch.zeros(4 * d, device=dev()),
                ws=e(F.fsdp_norm_workspace(tokens, d), dt=f), wa=e(F.fsdp_act_workspace(tokens, 4 * d), dt=f))


def block_step(st):
    """norm(x + res) -> up -> GELU -> down, and its backward pass from the two checkpoints."""
    F.fsdp_norm_forward(st["x"], st["w"], st["b"], st["y"], st["mean"], st["rstd"], kind="layer",
                        residual=st["res"], sum=st["s"], ckpt=st["qx"])
    h = torch.addmm(st["bias"], st["y"], st["up"].t())
    F.fsdp_act_forward(h, st["a"], kind="gelu_tanh", ckpt=st["qh"])
    out = st["a"] @ st["down"].t()
    da = st["dout"] @ st["down"]
    F.fsdp_act_backward(da, st["qh"], st["dh"], st["dbias"], st["wa"], kind="gelu_tanh", y=st["a2"], accumulate=True)
    dy = st["dh"] @ st["up"]
    F.fsdp_norm_backward(dy, st["qx"], st["w"], st["mean"], st["rstd"], st["dx"], st["dw"], st["db"], st["ws"],
                         kind="layer", dres=st["dout"], y=st["y2"], bias=st["b"], accumulate=True)
    ddown = st["dout"].t() @ st["a2"]
    dup = st["dh"].t() @ st["y2"]
    return out, ddown, dup


def test_block_step_gradients_from_checkpoints():
    """An MLP block's gradients against those of torch's autograd in 64 bits without checkpoints:
    what 8 bits cost (e4m3: at most 2^-4 of an element, so 2^-5 or so in the mean; integers less)
    and bf16 products add, and no more."""
    st = block_state(1)
    out, ddown, dup = block_step(st)
    p = {k: st[k].double().cpu().requires_grad_() for k in ("x", "w", "b", "up", "down", "bias")}
    s = p["x"] + st["res"].double().cpu()
    y = torch.nn.functional.layer_norm(s, (s.shape[1],), p["w"], p["b"], 1e-5)
    h = y @ p["up"].t() + p["bias"]
    o = torch.nn.functional.gelu(h, approximate="tanh") @ p["down"].t()
    # the block's output also reaches the residual stream, whose gradient is dout
    (o * st["dout"].double().cpu()).sum().backward()
    dx = p["x"].grad + st["dout"].double().cpu()
    for name, got, want, tol in (("out", out, o, 0.02), ("dx", st["dx"], dx, 0.02), ("dw", st["dw"], p["w"].grad, 0.05),
                                 ("db", st["db"], p["b"].grad, 0.03), ("dbias", st["dbias"], p["bias"].grad, 0.03),
                                 ("ddown", ddown, p["down"].grad, 0.03), ("dup", dup, p["up"].grad, 0.05)):
        err = float((got.double().cpu() - want).detach().norm() / want.detach().norm())
        assert err < tol, (name, err)


def test_block_step_replays_from_a_captured_graph():
    """Captured once, replayed among eager work; every replay equals the eager result bit for bit."""
    eager, graph = block_state(3), block_state(3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block_step(block_state(4))
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        block_step(graph)
    for rep in range(3):
        g.replay()
        block_step(eager)
        torch.cuda.synchronize()
        for k in ("s", "y", "a", "dh", "a2", "y2", "dx", "dw", "db", "dbias", "mean", "rstd"):
            assert torch.equal(eager[k], graph[k]), (rep, k)
        torch.randn(1 << 20, device=dev()).mul_(2.0).sum().item()


def test_same_call_same_bits_on_any_stream():
    x, w, b = norm_inputs(3, 3001, 1280, "bf16", "bf16")
    dy = normal(5, 3001, 1280).bfloat16().to(dev())
    mean, rstd = given_stats(x, "layer")
    first = run_backward(dy, x, w, mean, rstd, "layer", "bf16")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = torch.empty(F.fsdp_norm_workspace(3001, 1280), device=dev())
    dx, dw, db = torch.empty_like(x), torch.empty(1280, device=dev()), torch.empty(1280, device=dev())
    torch.cuda.synchronize()
    F.fsdp_norm_backward(dy, x, w, mean, rstd, dx, dw, db, ws, kind="layer", stream=s)
    s.synchronize()
    for u, v in zip(first[:3], (dx, dw, db)):
        assert torch.equal(u, v)


def test_gradients_go_through_the_unit():
    """dweight and dbias accumulate in the unit's unsharded fp32 gradient at the parameters'
    offsets, which the cast, the reduction and AdamW of the data path then take."""
    d, tokens = 320, 96
    shapes = [(d,), (d,), (4 * d, d), (4 * d,)]
    u = F.fsdp_unit_create(F.FSDP_FLAT, shapes, 4)
    acc = torch.zeros(u.L, device=dev())
    x, w, b = norm_inputs(3, tokens, d, "bf16", "bf16")
    h = normal(5, tokens, 4 * d).bfloat16().to(dev())
    dw = acc[u.offset(0):u.offset(0) + d]
    db = acc[u.offset(1):u.offset(1) + d]
    dbias = acc[u.offset(3):u.offset(3) + 4 * d]
    ws = torch.empty(max(F.fsdp_norm_workspace(tokens, d), F.fsdp_act_workspace(tokens, 4 * d)), device=dev())
    mean, rstd = given_stats(x, "layer")
    dx, dh = torch.empty_like(x), torch.empty_like(h)
    want = torch.zeros(u.L, dtype=torch.float64)
    ones = torch.ones(tokens, 4 * d, dtype=torch.bfloat16, device=dev())
    for step in range(3):
        dy = normal(20 + step, tokens, d).bfloat16().to(dev())
        F.fsdp_norm_backward(dy, x, w, mean, rstd, dx, dw, db, ws, kind="layer", accumulate=True)
        F.fsdp_act_backward(ones, h, dh, dbias, ws, kind="relu", accumulate=True)
        r = R.norm_grads(f64(dy), f64(x), f64(w), None, f64(mean), f64(rstd), "layer", "bf16")
        for i, v in ((0, r["dw"]), (1, r["db"]), (3, R.act(f64(h), "relu")[1].sum(0))):
            want[u.offset(i):u.offset(i) + v.size] += torch.from_numpy(v)
    err = (acc.double().cpu() - want).abs()
    assert float(err.max()) <= 1e-5 * float(want.abs().max())
    low = torch.empty(u.L, dtype=torch.bfloat16, device=dev())
    F.fsdp_cast_to_bf16(u, F.FSDP_ALL_RANKS, acc, low)
    grad = torch.empty(u.S, device=dev())
    F.fsdp_grad_reduce_shard(u, [low[1 * u.S:2 * u.S]] * 4, 1.0, 4.0, grad)
    assert torch.equal(grad, low[u.S:2 * u.S].float())


def test_the_binding_refuses_what_does_not_fit():
    """Shapes, dtypes, strides and devices are checked before the library is called."""
    x = torch.zeros(6, 40, device=dev())
    w, m = torch.zeros(40, device=dev()), torch.zeros(6, device=dev())
    q = F.Ckpt.empty(6, 40, "int8", device=dev())
    ok = lambda **k: F.fsdp_norm_forward(**{**dict(x=x, weight=w, bias=w, y=x.clone(), mean=m, rstd=m.clone()), **k})  # noqa: E731
    ok()
    for bad, kind in ((dict(y=x[:5]), ValueError), (dict(y=x.bfloat16()), TypeError), (dict(weight=w[:39]), ValueError),
                      (dict(y=torch.zeros(40, 6, device=dev()).t()), ValueError), (dict(y=x.cpu()), ValueError),
                      (dict(bias=w.bfloat16()), TypeError), (dict(weight=None), TypeError), (dict(mean=m[:3]), ValueError),
                      (dict(rstd=m.double()), TypeError), (dict(kind="batch"), ValueError), (dict(ckpt=q.codes), TypeError),
                      (dict(ckpt=F.Ckpt.empty(6, 39, "int8", device=dev())), ValueError), (dict(x=x.half()), TypeError),
                      (dict(sum=x.clone()), F.FsdpError), (dict(y=torch.zeros(40, device=dev()).expand(6, 40)), F.FsdpError),
                      (dict(eps=-1.0), F.FsdpError), (dict(mean=None), F.FsdpError)):
        with pytest.raises(kind):
            ok(**bad)
    ws = torch.zeros(F.fsdp_norm_workspace(6, 40), device=dev())
    bwd = lambda **k: F.fsdp_norm_backward(**{**dict(dy=x, x=q, weight=w, mean=m, rstd=m, dx=x.clone(), dweight=w.clone(), dbias=w.clone(), workspace=ws), **k})  # noqa: E731
    F.fsdp_ckpt_pack(x, q)
    bwd()
    for bad, kind in ((dict(workspace=ws[:-4]), F.FsdpError), (dict(workspace=None), F.FsdpError), (dict(dweight=w.double()), TypeError),
                      (dict(dbias=w.bfloat16()), TypeError), (dict(workspace=ws[1:]), F.FsdpError), (dict(x=None), TypeError)):
        with pytest.raises(kind):
            bwd(**bad)
    with pytest.raises(ValueError):
        F.fsdp_act_forward(x, x.clone(), kind="tanh")
    with pytest.raises(ValueError):
        F.Ckpt(q.codes, q.scales[:, :1], "int8")
    with pytest.raises(TypeError):
        F.Ckpt(q.codes.int(), q.scales, "int8")
    with pytest.raises(ValueError):
        F.Ckpt(q.codes, q.scales, "int4")


def test_two_streams_with_a_workspace_each():
    """Calls at the same time on two streams, each with its own workspace and outputs."""
    x, w, b = norm_inputs(3, 2000, 1280, "bf16", "bf16")
    mean, rstd = given_stats(x, "layer")
    dys = [normal(5 + i, 2000, 1280).bfloat16().to(dev()) for i in (0, 1)]
    alone = [run_backward(dy, x, w, mean, rstd, "layer", "bf16")[:3] for dy in dys]
    streams = [torch.cuda.Stream() for _ in dys]
    out = [(torch.empty_like(x), torch.empty(1280, device=dev()), torch.empty(1280, device=dev()),
            torch.empty(F.fsdp_norm_workspace(2000, 1280), device=dev())) for _ in dys]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, dy, (dx, dw, db, ws) in zip(streams, dys, out):
            F.fsdp_norm_backward(dy, x, w, mean, rstd, dx, dw, db, ws, kind="layer", stream=s)
    torch.cuda.synchronize()
    for want, got in zip(alone, out):
        for u, v in zip(want, got):
            assert torch.equal(u, v)
