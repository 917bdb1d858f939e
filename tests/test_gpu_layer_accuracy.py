"""How far the activations are from their 64-bit values, point by point over the arguments that
matter.  The bounds count roundings: U = 2^-24 is half a step of binary32 relative to the value, the
hardware's 2^x and reciprocal are off by one step each."""
import numpy as np
import pytest
import torch
from scipy.special import ndtr

import layer_ref as R
import sharded_fsdp_flatten_amd as F
from gpu_util import dev

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f32": torch.float32}
TINY = 2.0 ** -126


def arguments(t, most):
    """Every bf16 number up to `most`, or as many binary32 numbers: evenly spaced, and over the binades
    down to 2^-100."""
    if t == "bf16":
        h = (torch.arange(1 << 16, dtype=torch.int32) << 16).view(torch.float32)
        h = h[torch.isfinite(h) & (h.abs() <= most)]
    else:
        g = torch.Generator().manual_seed(7)
        h = torch.linspace(-most, most, 400001)
        h = h + (2 * most / 400000) * (torch.rand(h.shape, generator=g) - 0.5)
        small = 2.0 ** (-100 * torch.rand(50000, generator=g))
        h = torch.cat([h.clamp(-most, most), small, -small])
    return h[None].to(T[t]).to(dev())


def both(kind, h, ckpt=None):
    """y from the forward pass, and again from the backward pass, and f' (dx for a gradient of ones)"""
    y, dx, again = torch.empty_like(h), torch.empty_like(h), torch.empty_like(h)
    F.fsdp_act_forward(h, y, kind=kind)
    F.fsdp_act_backward(torch.ones_like(h), h, dx, kind=kind, y=again)
    assert torch.equal(y, again)
    return y.double().cpu().numpy(), dx.double().cpu().numpy()


def inside(got, want, bound, h, what):
    bad = ~(np.abs(got - want) <= bound)
    i = int(np.argmax(np.abs(got - want) / np.maximum(bound, 1e-300)))
    assert not bad.any(), "%s: %d beyond the bound; worst at h = %r: got %r want %r bound %r" % (
        what, bad.sum(), h.flat[i], got.flat[i], want.flat[i], np.broadcast_to(bound, got.shape).flat[i])


@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_gelu_has_its_stated_bounds(t):
    """Phi(-|h|) = Q = e R: 1.0e-8 of the fit, the roundings of the polynomial's ten steps, of a + 3, its
    reciprocal and their product (times |dR/dq|), of h^2 log2(e)/2 and the exponential, and of the product
    add up to 0.96e-7 at most (at h = 0; 1.25e-7 with the rounding of 1 - Q) and to (6 + 4|h| + h^2) U of Q, which is 2.6, 7.3, 19, 90 and 177 U at
    |h| = 0.1, 1, 3, 8 and 13 where they are added up step by step.  f' adds h times the density (relative
    2.5 U + h^2 U): 1.57e-7 at most.  Where the exponential is below the smallest
    normal number it may be 0."""
    x = arguments(t, 13.0)
    y, d = both("gelu", x)
    h = x.double().cpu().numpy()
    phi = ndtr(h)
    want, slope = h * phi, phi + h * np.exp(-h * h / 2) / np.sqrt(2 * np.pi)
    e = np.abs(h) * 1.3e-7
    e = np.where(h < 0, np.minimum(e, (6 + 4 * np.abs(h) + h * h) * R.U * np.abs(want)), e) + R.U * np.abs(want)
    half = R.HALF[t] if t == "bf16" else 0    # binary32's own last rounding is counted above
    inside(y, want, e + (np.abs(want) + e) * half + 13 * TINY, h, "y")
    e = 1.6e-7 + R.U * np.abs(slope)
    inside(d, slope, e + (np.abs(slope) + e) * half, h, "f'")


def test_gelu_of_infinities_and_nan():
    """As the formula in torch's erf form gives them: inf, -inf x 0 and NaN, and large numbers as they are."""
    h = torch.tensor([[float("inf"), float("-inf"), float("nan"), 3e38, -3e38, 1e20, -1e20, 17.0, -17.0]], device=dev())
    y, d = torch.empty_like(h), torch.empty_like(h)
    F.fsdp_act_forward(h, y, kind="gelu")
    F.fsdp_act_backward(torch.ones_like(h), h, d, kind="gelu")
    y, d = y[0].tolist(), d[0].tolist()
    assert y[0] == float("inf") and np.isnan(y[1]) and np.isnan(y[2])
    assert y[3:] == [h[0, 3].item(), 0, h[0, 5].item(), 0, 17, 0] and d[3:] == [1, 0, 1, 0, 1, 0]


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["gelu_tanh", "silu"])
def test_logistic_activations(kind, t):
    """s = 1 / (1 + E), w = 1 - s = E s.  E = e^-z has the relative error rz U |z| of its argument (SiLU: the
    product with log2(e) and that constant, 2; GELU: two constants, h^2, a multiply-add and a product, 4) and
    2 U of the exponential; 1 + E, its reciprocal and a product add 4 U.  f' is s (1 + h w), or
    s + h s w p with p = 2a + 6ac h^2.  Where s is below the smallest normal number it may be 0."""
    x = arguments(t, 13.0)
    y, d = both(kind, x)
    h = x.double().cpu().numpy()
    a, c = np.sqrt(2 / np.pi), 0.044715
    z, rz = (h, 2) if kind == "silu" else (2 * a * (h + c * h ** 3), 4)
    with np.errstate(over="ignore"):
        s, w = 1 / (1 + np.exp(-z)), 1 / (1 + np.exp(z))
    U = R.U
    re = (rz * np.abs(z) + 2) * U
    es, ew = s * (w * re + 3 * U), w * (s * re + 4 * U)
    want = h * s
    ey = np.abs(h) * es + U * np.abs(want)
    if kind == "silu":
        k = 1 + h * w
        slope = s * k
        ed = np.abs(k) * es + s * (np.abs(h) * (ew + U * w) + U * np.abs(k)) + U * np.abs(slope)
    else:
        p = 2 * a + 6 * a * c * h * h
        slope = s + want * w * p
        ed = es + p * (w * ey + np.abs(want) * (ew + 5 * U * w)) + U * np.abs(slope)
    half = R.HALF[t] if t == "bf16" else 0
    inside(y, want, ey + (np.abs(want) + ey) * half + 1000 * TINY, h, "y")
    inside(d, slope, ed + (np.abs(slope) + ed) * half + 1000 * TINY, h, "f'")
