"""AdamW with 8-bit states on the GPU where values are small: an exp_avg_sq above 0 is held as the smallest code at
least, so that the next update stays about as large as fp32 states allow; subnormal exp_avg_sq; eps of 0, subnormal,
tiny and huge."""
import numpy as np
import pytest
import torch

import sharded_fsdp_flatten_amd as F
import train_ref as R
from gpu_util import dev
from test_gpu_adam_tensors import Case, f32

pytestmark = pytest.mark.gpu

nearest = R.write_state


def kept_state(x, r, which):
    """The reference's 8-bit state, where a v above 0 whose code would be 0 has the smallest one."""
    buf = nearest(x, r, which)
    if which == "v":
        n = len(x)
        finite = np.repeat(buf[R.scales_at(n):] != 255, 32)[:n]
        buf[:n] = np.where(finite & (x != 0) & (buf[:n] == 0), 1, buf[:n])
    return buf


@pytest.fixture(autouse=True)
def states_keep_v(monkeypatch):
    monkeypatch.setattr(R, "write_state", kept_state)


def smallest(buf, n, which):
    """The smallest code's value, element by element."""
    byte = buf[R.scales_at(n):R.state_bytes(n)].astype(float)
    return np.repeat(2.0 ** (byte - 127 - (9 if which == "m" else 17)), 32)[:n]


@pytest.mark.parametrize("size", [1e-12, 1e-7, 1e-6, 2e-6, 5e-6, 2e-5, 1e-3])
def test_updates_stay_as_large_as_in_32_bits(size):
    """One gradient of 1 beside 31 of `size` in every group, then none, as for the row of an embedding that is seen
    once.  What a rounding can do, element by element: up by an eighth, or a smallest code, of m; down by a ninth of v,
    by half where its code is below 8, and never below the smallest.  (With v rounded to 0 the second update is
    hundreds of times lr; with fp32 states it is 0.67.)"""
    n, lr, b1, b2 = 32 * 500, 0.5, 0.9, 0.999
    g = np.full(n, size, np.float32)
    g[::32] = 1.0
    g[1::2] *= -1
    p, grad = torch.zeros(n, device=dev()), torch.from_numpy(g).to(dev())
    m, v = (torch.zeros(F.fsdp_adam_state_bytes(n), dtype=torch.uint8, device=dev()) for _ in range(2))
    tensors = F.AdamTensors([p], [grad], [m], [v], states="8bit")
    most_m, least_v = np.zeros(n), np.zeros(n)
    for t in range(1, 5):
        before = f32(p).astype(float)
        F.fsdp_adam_tensors(tensors, dict(lr=lr, betas=(b1, b2), step=t), seed=11)
        got = np.abs(f32(p) - before)
        a = np.abs(g.astype(float)) if t == 1 else np.zeros(n)
        most_m, least_v = b1 * most_m + (1 - b1) * a, b2 * least_v + (1 - b2) * a * a
        most = lr * most_m / (1 - b1 ** t) / np.sqrt(least_v / (1 - b2 ** t))
        # binary32: a few roundings of the moments and of the update, and one of p
        assert (got <= most * (1 + 32 * R.U) + 2 * R.U * np.abs(f32(p))).all(), (t, (got / lr).max())
        assert most.max() < 10 * lr, t
        qm, qv = smallest(m.cpu().numpy(), n, "m"), smallest(v.cpu().numpy(), n, "v")
        most_m = most_m * 9 / 8 + qm
        least_v = np.maximum(np.where(least_v >= 8 * qv, 8 / 9, 0.5) * least_v, qv)
        assert (R.read_state(v.cpu().numpy(), n, "v") >= least_v * (1 - 32 * R.U)).all()
        grad.zero_()


@pytest.mark.parametrize("grad", ["f32", "bf16"])
@pytest.mark.parametrize("spread", [3.0, 7.0])
def test_gradients_of_many_sizes_in_a_group(spread, grad):
    """Steps with gradients up to e^(3 spread) apart in a group, half of them none, and whole steps without any."""
    sizes = [4000, 33, 1, 700]
    c = Case(sizes, "8bit", grad)
    rng = np.random.Generator(np.random.PCG64(int(spread)))
    for step in range(1, 9):
        for i, n in enumerate(sizes):
            g = np.exp(spread * rng.standard_normal(n)) * rng.choice([-1e-3, 0.0, 1e-3, 0.0], n) * (step % 3 != 0)
            c.g[i] = torch.from_numpy(g.astype(np.float32)).to(c.g[i].dtype)
            c.arena["g"].parts[i].copy_(c.g[i])
        cfg = dict(lr=1e-2, betas=(0.9, 0.999), weight_decay=0.1, step=step)
        F.fsdp_adam_tensors(c.list, cfg, seed=5)
        c.reference([cfg], seed=5)
        c.check()


def test_conversion_keeps_small_values():
    """From 32 bits the same rounding: what is above 0 stays above it."""
    n = 6400
    rng = np.random.Generator(np.random.PCG64(2))
    x = np.exp(8 * rng.standard_normal(n)).astype(np.float32)
    x[::7] = 0.0
    m, v = (torch.from_numpy(x).to(dev()) for _ in range(2))
    to = [torch.zeros(F.fsdp_adam_state_bytes(n), dtype=torch.uint8, device=dev()) for _ in range(2)]
    p = torch.zeros(n, device=dev())
    F.fsdp_adam_convert(F.AdamTensors(None, None, [m], [v]), F.AdamTensors([p], [p], [to[0]], [to[1]], states="8bit"), seed=3, step=2)
    r = R.random16(n, R.key(3, 2, 0))
    for got, which, u in zip(to, "mv", r):
        assert np.array_equal(got.cpu().numpy(), kept_state(x, u, which)), which
    assert np.array_equal(R.read_state(to[1].cpu().numpy(), n, "v") > 0, x > 0)


@pytest.mark.parametrize("grad", ["f32", "bf16"])
@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-40, 1e-30, 1e-20, 2.0 ** 95, 2.0 ** 100, 2.0 ** 127])
@pytest.mark.parametrize("size", [1e-22, 1e-20, 1e-19, 1e-17, 1.0])
def test_subnormal_squares_and_any_eps(size, eps, grad):
    """exp_avg_sq of 1e-45 to 1e-37 among others, where eps does not hide its root; eps whose reciprocal is
    subnormal or infinite."""
    c = Case([4000, 45], "8bit", grad, scale=size)
    for step in (1, 2):
        cfg = dict(lr=1e-2, betas=(0.9, 0.999), eps=eps, step=step)
        F.fsdp_adam_tensors(c.list, cfg, seed=step)
        c.reference([cfg], seed=step)
        c.check()


@pytest.mark.parametrize("size", [1e-21, 1e-20, 3e-19])
def test_a_first_step_of_tiny_gradients_without_eps(size):
    """From states of 0, as fsdp_adam_shard takes it: by about lr."""
    n = 100
    g = torch.full((n,), size, device=dev())
    p = torch.ones(n, device=dev())
    m, v = (torch.zeros(F.fsdp_adam_state_bytes(n), dtype=torch.uint8, device=dev()) for _ in range(2))
    F.fsdp_adam_tensors(F.AdamTensors([p], [g], [m], [v], states="8bit"), dict(lr=0.25, step=1, eps=0.0))
    q, qm, qv = torch.ones(n, device=dev()), torch.zeros(n, device=dev()), torch.zeros(n, device=dev())
    unit = F.fsdp_unit_create(F.FSDP_FLAT, [(n,)], 1)
    F.fsdp_adam_shard(unit, q, g, qm, qv, lr=0.25, betas=(0.9, 0.999), eps=0.0, weight_decay=0.0, step=1)
    # the update, within 14 x 2^-24 of itself, and both results' rounding
    assert float((p - q).abs().max()) <= (14 * 0.3 + 2) * R.U
    assert 0.2 < float(1 - q.max()) < 0.3
