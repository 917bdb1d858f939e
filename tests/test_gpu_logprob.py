"""Token log probabilities on the GPU against a plain 64-bit reference (train_ref.py) within bounds computed from
the inputs, and their gradients: short and long vocabularies, rows at any element, padded tokens, masked
logits and rows, infinities and NaN, ties among the alternatives, in place."""
import numpy as np
import pytest
import torch

import sharded_fsdp_flatten_amd as F
import train_ref as R
from gpu_util import dev

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f32": torch.float32}
FILL = 7.0
COLS = [1, 2, 7, 8, 9, 31, 63, 64, 65, 257, 511, 1000, 2048, 2049, 4097, 8200, 16385, 50257, 131073, 300001]


def f64(t):
    return t.detach().double().cpu().numpy()


class Matrix:
    def __init__(self, rows, cols, dtype, pitch=None, start=0):
        pitch = cols if pitch is None else pitch
        self.base = torch.full((start + max(rows, 1) * pitch + 64,), FILL, dtype=dtype, device=dev())
        self.view = ((rows, cols), (pitch, 1), start)
        self.t = self.base.as_strided(*self.view)

    def around_is_untouched(self):
        b = self.base.clone()
        b.as_strided(*self.view).fill_(FILL)
        return bool((b == FILL).all())


def logits(seed, rows, cols, dtype, spread=3.0, ignored=0.2):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, cols, generator=g) * spread).to(T[dtype])
    tok = torch.randint(0, cols, (rows,), generator=g)
    tok[torch.rand(rows, generator=g) < ignored] = -100
    return x, tok


def close(got, want, bound, what):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    with np.errstate(invalid="ignore"):
        bad = ~((np.abs(got - want) <= bound) | (np.isnan(got) & np.isnan(want)) | (got == want))
    assert not bad.any(), "%s: %d of %d beyond the bound; first at %s: got %r want %r bound %r" % (
        what, bad.sum(), bad.size, np.argwhere(bad)[0], got[bad][0], np.asarray(want)[bad][0], np.broadcast_to(bound, got.shape)[bad][0])


def guard(n, dtype=torch.float32):
    base = torch.full((n + 8,), FILL, dtype=dtype, device=dev())
    return base, base[4:4 + n]


def forward(m, tok, scale=1.0, top=0, entropy=True):
    """The call's outputs, all in guarded buffers."""
    rows, cols = m.t.shape
    bufs = {k: guard(rows) for k in ("logprob", "max", "logsum", "entropy")}
    bufs |= {"top_logprob": guard(rows * top), "top_token": guard(rows * top, torch.int64)}
    need = F.fsdp_logprob_workspace(rows, cols, top)
    ws, wv = guard((need + 3) // 4 * 4)
    ws.fill_(float("nan"))
    o = {k: v for k, (_, v) in bufs.items()}
    tops = dict(top_logprob=o["top_logprob"].view(rows, top), top_token=o["top_token"].view(rows, top)) if top else {}
    F.fsdp_logprob_forward(m.t, tok.to(dev()), o["logprob"], o["max"], o["logsum"], wv, scale=scale, entropy=o["entropy"] if entropy else None, **tops)
    for k, (b, v) in bufs.items():
        assert (b[:4] == FILL).all() and (b[4 + v.numel():] == FILL).all(), k
    assert ws[:4].isnan().all() and ws[4 + wv.numel():].isnan().all()
    assert m.around_is_untouched()
    return {**o, **tops}


def check_forward(x, tok, scale=1.0, top=0, pitch=None, start=0):
    m = Matrix(*x.shape, x.dtype, pitch, start)
    m.t.copy_(x)
    got = forward(m, tok, scale, top)
    want = R.logprob(f64(x), tok.numpy(), float(np.float32(scale)))
    close(got["max"], want["max"], 0.0, "max")
    close(got["logsum"], want["logsum"], want["elogsum"], "logsum")
    close(got["entropy"], want["entropy"], want["eentropy"], "entropy")
    close(got["logprob"], want["logprob"], want["elogprob"], "logprob")
    if top:
        cols = R.top(f64(x), top)
        assert np.array_equal(got["top_token"].cpu().numpy(), cols)
        r = np.arange(len(x))[:, None]
        close(got["top_logprob"], want["lp"][r, cols], want["elp"][r, cols], "top_logprob")
    again = forward(m, tok, scale, top)
    for k in got:
        assert torch.equal(got[k].nan_to_num(9), again[k].nan_to_num(9)), k
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", COLS)
def test_forward(cols, dtype):
    rows = 3 if cols > 100000 else 13
    x, tok = logits(cols, rows, cols, dtype)
    check_forward(x, tok, top=min(cols, 5))
    check_forward(x, tok, 0.7, 0, cols + 3, 1)


@pytest.mark.parametrize("top", [1, 2, 20, 33, 63, 64])
@pytest.mark.parametrize("cols", [64, 100, 777, 5003, 50257, 262144])
def test_top(cols, top):
    x, tok = logits(cols + top, 4, cols, "bf16")
    check_forward(x, tok, top=top)
    x, tok = logits(cols + top, 2, cols, "f32")
    check_forward(x, tok, 1.3, top, cols + 1, 3)


@pytest.mark.parametrize("dtype,cols", [("bf16", 70000), ("bf16", 4900), ("bf16", 33000), ("f32", 33000), ("f32", 4900), ("f32", 2000)])
def test_top_in_every_column(cols, dtype):
    """The largest logits at every place of the last vectors and around the ends of whole steps, rows at any
    element: none of them is lost where lanes part."""
    n = 128
    x = torch.zeros(n, cols)
    for r in range(n):
        x[r, cols - 1 - 9 * r % 1100] = 3.0
        x[r, r * 37 % cols] = 2.0
        x[r, (cols // 2 + r * 61) % cols] = 4.0
    check_forward(x.to(T[dtype]), torch.zeros(n, dtype=torch.int64), top=3, pitch=cols + 1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [64, 100, 2051, 50257, 200003])
def test_ties(cols, dtype):
    """Equal logits in every arrangement: lower columns come first."""
    j = torch.arange(cols)
    rows = [torch.zeros(cols), (j % 3).float(), (j // 100 % 2).float(), -(j // 7).float().clamp(max=50), (j // (cols // 4 + 1)).float(),
            torch.where(j % 2 == 0, 0.0, -0.0), torch.where(j % 512 < 8, 5.0, 0.0), torch.where(j % 4096 < 512, -1.0, 2.0)]
    x = torch.stack(rows).to(T[dtype])
    check_forward(x, torch.full((len(rows),), cols // 2), top=min(64, cols))


@pytest.mark.parametrize("cols", [100, 5000, 50257])
def test_sorted_rows(cols):
    """Every logit larger than all before it, and smaller."""
    x = torch.linspace(-5, 5, cols)
    check_forward(torch.stack([x, x.flip(0)]), torch.tensor([0, cols - 1]), top=64)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [9, 513, 50257, 140000])
def test_masks_infinities_and_nan(cols, dtype):
    """Rows with a few allowed tokens, one, none; masks of the type's lowest value; infinities and NaN."""
    inf, nan, low = float("inf"), float("nan"), torch.finfo(T[dtype]).min
    x, _ = logits(cols, 16, cols, dtype)
    x = x.float()
    a, b = cols // 3, cols - 1
    x[0, :a] = -inf
    x[1, a:] = -inf
    x[2] = -inf
    x[2, [a, b]] = torch.tensor([1.0, 2.0])
    x[3] = -inf
    x[3, b] = 3.0
    x[4] = -inf
    x[5, 1:] = low
    x[6] = low
    x[7, a] = inf
    x[8, b] = nan
    x[9] = nan
    x[10] = -inf
    x[10, 0] = nan
    x[11, [a, b]] = inf
    x[12] = -inf
    x[12, b] = inf
    x[13] = low
    x[13, a] = -low
    x[14, a] = -inf
    tok = torch.tensor([b, 0, a, b, 0, 0, b, a, 0, a, 0, 1, 0, a, a, -1])
    for top in (0, min(cols, 20)):
        check_forward(x.to(T[dtype]), tok, top=top)
    check_forward(x.to(T[dtype]), tok, 1.5, 3)
    check_forward(x.to(T[dtype]), torch.where(tok == 0, cols, tok), 0.5, 3)


def test_entropy_and_tokens_are_optional():
    x, tok = logits(5, 9, 1003, "bf16")
    m = Matrix(9, 1003, T["bf16"])
    m.t.copy_(x)
    full = forward(m, tok, top=4)
    less = forward(m, tok, top=4, entropy=False)
    for k in ("logprob", "max", "logsum", "top_logprob", "top_token"):
        assert torch.equal(full[k], less[k]), k
    mx, ls = torch.empty(9, device=dev()), torch.empty(9, device=dev())
    F.fsdp_logprob_forward(m.t, None, None, mx, ls)
    assert torch.equal(mx, full["max"]) and torch.equal(ls, full["logsum"])


def test_equal_rows_by_pitch_zero():
    x, _ = logits(5, 1, 777, "f32")
    t = x.to(dev()).expand(6, 777)
    o = [torch.empty(6, device=dev()) for _ in range(3)]
    F.fsdp_logprob_forward(t, torch.arange(6, device=dev()), *o)
    want = R.logprob(f64(x.expand(6, 777)), np.arange(6), 1.0)
    close(o[0], want["logprob"], want["elogprob"], "logprob")


# ---------------------------------------------------------------------------
# gradients
# ---------------------------------------------------------------------------
def check_backward(x, tok, dl, dh, scale=1.0, pitch=None, start=0, out_pitch=None, out_start=0, inplace=False, stats=None):
    rows, cols = x.shape
    t = "bf16" if x.dtype == torch.bfloat16 else "f32"
    m = Matrix(rows, cols, x.dtype, pitch, start)
    m.t.copy_(x)
    if stats is None:
        ref = R.logprob(f64(x), tok.numpy(), float(np.float32(scale)))
        stats = [torch.tensor(ref[k], dtype=torch.float32) for k in ("max", "logsum", "entropy")]
    d = [v.to(dev()) for v in stats]
    y = m if inplace else Matrix(rows, cols, x.dtype, out_pitch, out_start)
    F.fsdp_logprob_backward(m.t, None if dl is None else tok.to(dev()), None if dl is None else dl.to(dev()), d[0], d[1], y.t, scale=scale,
                            dentropy=None if dh is None else dh.to(dev()), entropy=None if dh is None else d[2])
    zero = np.zeros(rows)
    want, bound = R.logprob_grad(f64(x), tok.numpy(), zero if dl is None else f64(dl), zero if dh is None else f64(dh), f64(stats[0]),
                                 f64(stats[1]), f64(stats[2]), float(np.float32(scale)), t)
    close(y.t, want, bound, "dlogits")
    assert y.around_is_untouched() and m.around_is_untouched()
    if not inplace:
        assert torch.equal(m.t.cpu().nan_to_num(9), x.nan_to_num(9))
    return y.t


def grads(seed, rows):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(rows, generator=g) * 0.1, torch.randn(rows, generator=g) * 0.01


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", COLS)
def test_backward(cols, dtype):
    rows = 3 if cols > 100000 else 13
    x, tok = logits(cols, rows, cols, dtype)
    dl, dh = grads(cols, rows)
    check_backward(x, tok, dl, dh)
    check_backward(x, tok, dl, None, 1.3, cols + 3, 1, cols + 2, 5)
    check_backward(x, tok, None, dh, 0.7, cols + 8, 8, cols, 3)
    check_backward(x, tok, dl, dh, 0.7, cols + 5, 3, inplace=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_without_gradient_are_zero_and_not_read(dtype):
    """Padded tokens, gradients of 0 and rows without an allowed token give zeros even over NaN."""
    x, _ = logits(1, 6, 1234, dtype)
    x[:4] = float("nan")
    x[4] = -float("inf")
    tok = torch.tensor([-100, 1234, 5, 7, 9, 11])
    dl = torch.tensor([1.0, 2.0, 0.0, -0.0, 1.0, 1.0])
    y = check_backward(x, tok, dl, torch.zeros(6))
    assert (y[:5] == 0).all() and (y[5] != 0).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [9, 5000, 50257])
def test_backward_of_masks_infinities_and_nan(cols, dtype):
    inf, nan, low = float("inf"), float("nan"), torch.finfo(T[dtype]).min
    x, _ = logits(cols, 8, cols, dtype)
    x[0, : cols // 2] = -inf
    x[1] = -inf
    x[1, cols - 1] = 2.0
    x[2, 1:] = low
    x[3] = low
    x[4, cols // 2] = inf
    x[5, cols // 2] = nan
    x[6] = -inf
    tok = torch.tensor([cols - 1, cols - 1, 0, 3, 1, 1, 1, 1])
    dl, dh = grads(3, 8)
    m = Matrix(8, cols, x.dtype)
    m.t.copy_(x)
    o = forward(m, tok)
    stats = [o[k].cpu() for k in ("max", "logsum", "entropy")]
    y = check_backward(x, tok, dl, dh, stats=stats)
    assert y[4:6].isnan().all() and (y[6] == 0).all() and (y[0, : cols // 2] == 0).all()
    check_backward(x, tok, dl, None, stats=stats)


def test_gradient_against_differences():
    """Central differences of the forward pass's own outputs in fp32, step 2^-6: the truncation is at most
    h^2 / 6 times the third derivative (at most scale^3 for a log probability, 6 scale^3 (1 + H) for the
    entropy), the roundings 2^-20 of sums of a few units over 2 h."""
    rows, cols, h, scale = 4, 33, 2.0 ** -6, 1.25
    x, tok = logits(8, rows, cols, "f32", 1.0, 0.0)
    dl, dh = torch.tensor([1.0, -0.5, 2.0, 0.25]), torch.tensor([0.5, 1.0, -1.0, 0.0])
    m = Matrix(rows, cols, torch.float32)
    m.t.copy_(x)
    o = forward(m, tok, scale)
    y = torch.empty(rows, cols, device=dev())
    F.fsdp_logprob_backward(m.t, tok.to(dev()), dl.to(dev()), o["max"], o["logsum"], y, scale=scale, dentropy=dh.to(dev()), entropy=o["entropy"])
    for j in range(cols):
        f = []
        for s in (h, -h):
            m.t.copy_(x)
            m.t[:, j] += s
            o = forward(m, tok, scale)
            f.append(dl * o["logprob"].cpu() + dh * o["entropy"].cpu())
        diff = ((f[0] - f[1]) / (2 * h)).double().numpy()
        bound = (h * h / 6 * scale ** 3 * (dl.abs() + 6 * 5 * dh.abs()) + 2.0 ** -20 * 8 * (dl.abs() + dh.abs()) / h).numpy() + 1e-6
        assert (np.abs(diff - f64(y)[:, j]) <= bound).all(), j


def test_refusals():
    x = torch.zeros(4, 8, device=dev())
    tok = torch.zeros(4, dtype=torch.int64, device=dev())
    v = torch.zeros(4, device=dev())
    with pytest.raises(TypeError):
        F.fsdp_logprob_forward(x, tok.int(), v, v, v)
    with pytest.raises(ValueError, match="tokens"):
        F.fsdp_logprob_forward(x, tok[:3], v, v, v)
    with pytest.raises(F.FsdpError, match="together"):
        F.fsdp_logprob_forward(x, tok, None, v, v)
    with pytest.raises(F.FsdpError, match="top"):
        F.fsdp_logprob_forward(x, tok, v, v, v, top_logprob=torch.zeros(4, 9, device=dev()), top_token=torch.zeros(4, 9, dtype=torch.int64, device=dev()))
    with pytest.raises(TypeError):
        F.fsdp_logprob_forward(x, tok, v, v, v, top_logprob=torch.zeros(4, 2, device=dev()))
    with pytest.raises(F.FsdpError, match="dlogprob"):
        F.fsdp_logprob_backward(x, tok, None, v, v, x)
    with pytest.raises(TypeError):
        F.fsdp_logprob_backward(x, tok, v, v, v, x.bfloat16())


@pytest.mark.parametrize("rows,cols,dtype,top,start", [(2048, 50257, "f32", 20, 1), (2051, 50257, "bf16", 0, 3), (2050, 66001, "bf16", 64, 7),
                                                       (2048, 32768, "f32", 7, 0), (700, 5003, "bf16", 0, 1), (12000, 9001, "bf16", 0, 3),
                                                       (600, 16384, "bf16", 0, 0), (513, 4097, "bf16", 0, 7)])
def test_many_long_rows(rows, cols, dtype, top, start):
    """Rows that fill the chip; a few of them hold masks, infinities, NaN, one value throughout and rising values."""
    m = Matrix(rows, cols, T[dtype], cols + 2, start)
    g = torch.Generator(device=dev()).manual_seed(rows)
    m.t.copy_((torch.randn(rows, cols, generator=g, device=dev()) * 3).to(T[dtype]))
    low = torch.finfo(T[dtype]).min
    m.t[1] = 0.25
    m.t[2] = -float("inf")
    m.t[3] = low
    m.t[4, 70:] = -float("inf")
    m.t[5, 100] = float("nan")
    m.t[6, 9] = float("inf")
    m.t[7] = torch.arange(cols, device=dev()).to(T[dtype])
    m.t[8, :cols - 30] = low
    tok = torch.randint(-1, cols, (rows,))
    got = forward(m, tok, 1.0, top)
    some = [*range(12), rows // 2, rows - 2, rows - 1]
    x = f64(m.t[some])
    want = R.logprob(x, tok[some].numpy(), 1.0)
    for k in ("logsum", "entropy", "logprob"):
        close(got[k][some], want[k], want["e" + k], k)
    if top:
        order = R.top(x, top)
        assert np.array_equal(got["top_token"][some].cpu().numpy(), order)
        r = np.arange(len(some))[:, None]
        close(got["top_logprob"][some], want["lp"][r, order], want["elp"][r, order], "top_logprob")
    again = forward(m, tok, 1.0, top)
    for k in got:
        assert torch.equal(got[k].nan_to_num(9), again[k].nan_to_num(9)), k


@pytest.mark.parametrize("rows,cols,dtype,start,in_place", [(2051, 33001, "bf16", 5, False), (1500, 20003, "f32", 1, False), (2049, 40007, "bf16", 1, True)])
def test_gradient_of_many_long_rows(rows, cols, dtype, start, in_place):
    """Loads past the cache: rows at any element, what lies between the rows stays."""
    m = Matrix(rows, cols, T[dtype], cols + 3, start)
    g = torch.Generator(device=dev()).manual_seed(rows)
    m.t.copy_((torch.randn(rows, cols, generator=g, device=dev()) * 3).to(T[dtype]))
    tok = torch.randint(-1, cols, (rows,))
    some = [*range(20), rows // 2, rows - 1]
    tok[:4] = torch.tensor([0, cols - 1, 1, cols - 2])
    x = f64(m.t[some])
    o = forward(m, tok, 0.8, 0)
    dl, dh = torch.randn(rows, generator=torch.Generator().manual_seed(1)), torch.randn(rows, generator=torch.Generator().manual_seed(2))
    y = m if in_place else Matrix(rows, cols, T[dtype], cols + 6, start + 2)
    F.fsdp_logprob_backward(m.t, tok.to(dev()), dl.to(dev()), o["max"], o["logsum"], y.t, scale=0.8, dentropy=dh.to(dev()), entropy=o["entropy"])
    want, bound = R.logprob_grad(x, tok[some].numpy(), f64(dl[some]), f64(dh[some]), *(f64(o[k][some]) for k in ("max", "logsum", "entropy")),
                                 float(np.float32(0.8)), dtype)
    close(y.t[some], want, bound, "gradient")
    assert y.around_is_untouched() and m.around_is_untouched()
