"""Rotary positions on the GPU against a plain 64-bit reference (train_ref.py) within bounds computed from the
inputs: both layouts, parts of a head, odd heads, any order of the dimensions, packed matrices, in place, far
and negative positions, frequencies scaled for long contexts."""
import numpy as np
import pytest
import torch

import sharded_fsdp_flatten_amd as F
import train_ref as R
from gpu_util import dev

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f32": torch.float32}
FILL = 7.0


def normal(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def f64(t):
    return t.detach().double().cpu().numpy()


class Heads:
    """[B, T, H, D] inside a larger allocation, in some order of the dimensions, with gaps and a start, all
    around it holding a pattern that must stay."""

    def __init__(self, shape, dtype, order="bthd", gap=0, start=0):
        B, n, H, D = shape
        size = dict(b=B, t=n, h=H, d=D)
        pitch, step = {}, 1
        for k in reversed(order):
            pitch[k] = step
            step *= size[k]
            if k != "d" or gap:
                step += gap
        self.base = torch.full((start + step + 64,), FILL, dtype=dtype, device=dev())
        self.view = ((B, n, H, D), tuple(pitch[k] for k in "bthd"), start)
        self.t = self.base.as_strided(*self.view)

    def around_is_untouched(self):
        b = self.base.clone()
        b.as_strided(*self.view).fill_(FILL)
        return bool((b == FILL).all())


def check(shape, kv, rot, dtype, layout="half", order="bthd", gap=0, start=0, inplace=False, backward=False, scale=1.0, positions=None,
          first=0, freqs=None, seed=0):
    B, n, H, D = shape
    f = F.fsdp_rotary_freqs(rot, **(freqs or {}))
    x = {"q": normal(seed, B, n, H, D).to(T[dtype]), "k": normal(seed + 1, B, n, kv, D).to(T[dtype])}
    src, out = {}, {}
    for k, h in (("q", H), ("k", kv)):
        src[k] = Heads((B, n, h, D), T[dtype], order, gap, start)
        src[k].t.copy_(x[k])
        out[k] = src[k] if inplace else Heads((B, n, h, D), T[dtype], order, gap + 1, start)
    fn = F.fsdp_rotary_backward if backward else F.fsdp_rotary_forward
    kw = dict(k=src["k"].t, k_out=out["k"].t) if kv else {}
    fn(src["q"].t, out["q"].t, f.to(dev()), positions=None if positions is None else positions.to(dev()), start=first, layout=layout,
       scale=scale, **kw)
    pos = np.broadcast_to(first + np.arange(n), (B, n)) if positions is None else positions.numpy().reshape(B, n)
    for k in ("q", "k") if kv else ("q",):
        want, bound = R.rotary(f64(x[k]), f.numpy(), pos, layout, float(np.float32(scale)), -1 if backward else 1, dtype)
        got = f64(out[k].t)
        bad = np.abs(got - want) > bound
        assert not bad.any(), (k, bad.sum(), np.argwhere(bad)[0], got[bad][0], want[bad][0], bound[bad][0])
        assert np.array_equal(got[..., rot:], f64(x[k])[..., rot:])
        assert out[k].around_is_untouched() and src[k].around_is_untouched()
        if not inplace:
            assert torch.equal(src[k].t.cpu(), x[k])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,rot", [(2, 2), (3, 2), (7, 4), (8, 8), (16, 16), (17, 14), (33, 30), (64, 64), (64, 32), (80, 40), (96, 96), (128, 128),
                                   (128, 64), (256, 256), (255, 2), (1024, 1024), (1023, 1022)])
def test_head_sizes(D, rot, dtype, layout):
    check((2, 5, 3, D), 2, rot, dtype, layout, seed=D + rot)


@pytest.mark.parametrize("H,kv", [(1, 0), (1, 1), (2, 1), (5, 3), (8, 8), (31, 2), (40, 0), (96, 96), (130, 1), (200, 57)])
@pytest.mark.parametrize("n", [1, 2, 33])
def test_heads_and_tokens(H, kv, n):
    check((3, n, H, 64), kv, 64, "bf16", seed=H)
    check((1, n, H, 24), kv, 20, "f32", "interleaved", seed=H)


@pytest.mark.parametrize("order", ["bthd", "bhtd", "tbhd", "thbd", "hbtd"])
@pytest.mark.parametrize("gap,start", [(0, 0), (3, 1), (8, 5)])
@pytest.mark.parametrize("inplace", [False, True])
def test_orders_gaps_and_places(order, gap, start, inplace):
    for dtype in T:
        check((2, 7, 5, 40), 2, 36, dtype, "half", order, gap, start, inplace)
        check((2, 7, 5, 40), 2, 36, dtype, "interleaved", order, gap, start, inplace, backward=True)


def test_inside_a_packed_matrix():
    qkv = normal(1, 2, 9, 3 * 6 * 32).bfloat16().to(dev())
    before = qkv.clone()
    x = qkv.view(2, 9, 3, 6, 32)
    f = F.fsdp_rotary_freqs(32)
    F.fsdp_rotary_forward(x[:, :, 0], x[:, :, 0], f.to(dev()), k=x[:, :, 1], k_out=x[:, :, 1])
    pos = np.broadcast_to(np.arange(9), (2, 9))
    for i in (0, 1):
        want, bound = R.rotary(f64(before.view(2, 9, 3, 6, 32)[:, :, i]), f.numpy(), pos, "half", 1.0, 1, "bf16")
        assert (np.abs(f64(x[:, :, i]) - want) <= bound).all()
    assert torch.equal(x[:, :, 2], before.view(2, 9, 3, 6, 32)[:, :, 2])


@pytest.mark.parametrize("first", [0, 5, 4095, 1 << 20, (1 << 24) + 1, (1 << 30) - 40, -17])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_far_positions(first, dtype):
    check((1, 40, 2, 64), 2, 64, dtype, first=first)
    g = torch.Generator().manual_seed(3)
    check((2, 20, 2, 64), 0, 64, dtype, positions=first + torch.randint(0, 1000, (2, 20), generator=g))


@pytest.mark.parametrize("freqs", [dict(base=5e5), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
                                   dict(scaling="parts", factor=8.0, trained_len=4096)])
@pytest.mark.parametrize("scale", [1.0, 1.2079441, -0.5, 0.0])
def test_scaled(freqs, scale):
    check((1, 50, 3, 128), 1, 128, "f32", first=30000, freqs=freqs, scale=scale)
    check((1, 50, 3, 128), 1, 96, "bf16", "interleaved", first=30000, freqs=freqs, scale=scale, backward=True)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_backward_is_the_gradient(layout):
    """<dy, forward(x)> differs along dx by <backward(dy), dx>: the rotation is linear, so a difference of any
    length is exact but for roundings."""
    f = F.fsdp_rotary_freqs(24).to(dev())
    x, d, dy = (normal(s, 2, 6, 3, 30).to(dev()) for s in (1, 2, 3))
    y0, y1, g = (torch.empty_like(x) for _ in range(3))
    F.fsdp_rotary_forward(x, y0, f, layout=layout, scale=1.25, start=7)
    F.fsdp_rotary_forward(x + d, y1, f, layout=layout, scale=1.25, start=7)
    F.fsdp_rotary_backward(dy, g, f, layout=layout, scale=1.25, start=7)
    a, b = ((y1 - y0).double() * dy.double()).sum(), (g.double() * d.double()).sum()
    size = float(((y1.abs() + y0.abs()).double() * dy.abs().double()).sum() + (g.abs() * d.abs()).double().sum())
    assert abs(float(a - b)) <= 32 * 2.0 ** -24 * size


def test_special_values():
    """An infinity or a NaN stays in its own pair."""
    x = normal(5, 1, 4, 2, 16).to(dev())
    x[0, 1, 0, 3], x[0, 2, 1, 9] = float("inf"), float("nan")
    y = torch.empty_like(x)
    F.fsdp_rotary_forward(x, y, F.fsdp_rotary_freqs(16).to(dev()), start=3)
    bad = torch.zeros_like(x, dtype=torch.bool)
    for t, h, i in ((1, 0, 3), (2, 1, 1)):
        bad[0, t, h, i] = bad[0, t, h, i + 8] = True
    assert torch.equal(~y.isfinite(), bad)


def test_many_tokens_of_one_head():
    check((1, 5000, 1, 8), 0, 8, "bf16")
    check((3, 1111, 1, 16), 1, 6, "f32", "interleaved")


def test_refusals():
    x = torch.zeros(2, 3, 4, 8, device=dev())
    f = F.fsdp_rotary_freqs(8).to(dev())
    with pytest.raises(ValueError, match="shape"):
        F.fsdp_rotary_forward(x, x[:, :2], f)
    with pytest.raises(ValueError, match="next to each other"):
        F.fsdp_rotary_forward(x, x.transpose(2, 3).contiguous().transpose(2, 3), f)
    with pytest.raises(TypeError):
        F.fsdp_rotary_forward(x, x.bfloat16(), f)
    with pytest.raises(TypeError):
        F.fsdp_rotary_forward(x, x, f.float())
    with pytest.raises(ValueError, match="GPU"):
        F.fsdp_rotary_forward(x, x, f.cpu())
    with pytest.raises(TypeError):
        F.fsdp_rotary_forward(x, x, f, k=x)
    with pytest.raises(ValueError, match="positions"):
        F.fsdp_rotary_forward(x, x, f, positions=torch.zeros(5, dtype=torch.int64, device=dev()))
    with pytest.raises(F.FsdpError, match="RANGE"):
        F.fsdp_rotary_forward(x, x, F.fsdp_rotary_freqs(10).to(dev()))
    with pytest.raises(F.FsdpError, match="overlap"):
        F.fsdp_rotary_forward(x, x[:, :, :1].expand(2, 3, 4, 8), f)
