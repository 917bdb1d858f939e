"""AdamW over many tensors on the GPU: with fp32 states bit for bit fsdp_adam_shard's step, with 8-bit states these
bit for bit as a plain reference has them (train_ref.py: binary32 steps, codes found in a table) and the
parameters within bounds; conversions; odd sizes, any
alignment, long lists, groups, clipping and skipped steps, infinities and NaN."""
import numpy as np
import pytest
import torch

import sharded_fsdp_flatten_amd as F
import train_ref as R
from gpu_util import assert_f32_bits, dev

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZES = [1, 2, 3, 4, 5, 31, 32, 33, 63, 64, 100, 255, 1000, 2047, 2048, 2049, 4100, 12345, 70001]
CFG = dict(lr=1e-2, betas=(0.9, 0.98), eps=1e-8, weight_decay=0.1, step=3)


class Arena:
    """Pieces of given sizes one after another in one buffer from element `start` on, `gap` apart, everything
    around them holding a pattern that must stay."""

    def __init__(self, sizes, dtype, start=0, gap=0):
        self.base = torch.full((start + sum(sizes) + gap * len(sizes) + 64,), 77, dtype=dtype, device=dev())
        self.parts, at = [], start
        for n in sizes:
            self.parts.append(self.base[at:at + n])
            at += n + gap

    def around_is_untouched(self):
        keep = self.base.clone()
        for p in self.parts:
            o = p.storage_offset()
            keep[o:o + p.numel()] = 77
        return bool((keep == 77).all())


def f32(t):
    return t.detach().float().cpu().numpy()


def same(got, want, what):
    """the same bits, any NaN for any NaN"""
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    fine = ~np.isnan(want)
    assert_f32_bits(got[fine], want[fine], what)


class Case:
    """Tensors of these sizes, their gradients and states, on both sides."""

    def __init__(self, sizes, states="f32", grad="f32", copy=True, start=0, gap=0, seed=0, scale=1e-3, groups=None):
        g = np.random.Generator(np.random.PCG64(seed))
        self.sizes, self.states = sizes, states
        normal = lambda n, s: (g.standard_normal(n) * s).astype(np.float32)  # noqa: E731
        self.p = [normal(n, 0.02) for n in sizes]
        self.g = [torch.from_numpy(normal(n, scale) * np.exp(normal(n, 1.0))).to(T[grad]) for n in sizes]
        self.m = [normal(n, scale / 5) for n in sizes]
        self.v = [normal(n, scale) ** 2 for n in sizes]
        self.arena = {k: Arena(sizes, torch.float32, start, gap) for k in ("p",)}
        self.arena["g"] = Arena(sizes, T[grad], start, gap)
        small = states == "8bit"
        for k in ("m", "v"):
            self.arena[k] = Arena([R.state_bytes(n) for n in sizes] if small else sizes, torch.uint8 if small else torch.float32, start, gap)
        if copy:
            self.arena["pb"] = Arena(sizes, torch.bfloat16, start, gap)
        for i, n in enumerate(sizes):
            self.arena["p"].parts[i].copy_(torch.from_numpy(self.p[i]))
            self.arena["g"].parts[i].copy_(self.g[i])
            for k, x in (("m", self.m), ("v", self.v)):
                if small:
                    r = R.random16(n, R.key(99, 1, i))
                    x[i] = R.write_state(x[i], r[0] if k == "m" else r[1], k)
                self.arena[k].parts[i].copy_(torch.from_numpy(x[i]))
        a = {k: x.parts for k, x in self.arena.items()}
        self.groups = groups or [0] * len(sizes)
        self.off = [np.zeros(n) for n in sizes]   # how far p may be from the reference's
        self.list = F.AdamTensors(a["p"], a["g"], a["m"], a["v"], states=states, groups=self.groups, param_bf16=a.get("pb"))

    def reference(self, cfgs, seed=0, gs=None):
        """The next step of the host's copies."""
        for i, n in enumerate(self.sizes):
            cfg = cfgs[self.groups[i]]
            g = f32(self.g[i])
            if self.states == "f32":
                self.p[i], self.m[i], self.v[i], _ = R.adam_f32(self.p[i], g, self.m[i], self.v[i], cfg, gs)
                continue
            m, v = (R.read_state(x[i], n, k).astype(np.float32) for k, x in (("m", self.m), ("v", self.v)))
            self.p[i], m, v, off = R.adam_f32(self.p[i], g, m, v, cfg, gs)
            self.off[i] = self.off[i] * abs(1 - cfg["lr"] * cfg.get("weight_decay", 0.0)) + off
            r = R.random16(n, R.key(seed, cfg["step"], i))
            self.m[i], self.v[i] = R.write_state(m, r[0], "m"), R.write_state(v, r[1], "v")

    def check(self):
        for i, n in enumerate(self.sizes):
            what = "tensor %d of %d elements: " % (i, n)
            p = f32(self.arena["p"].parts[i])
            if self.states == "f32":
                same(p, self.p[i], what + "p")
            else:
                assert np.array_equal(np.isnan(p), np.isnan(self.p[i])), what + "p"
                with np.errstate(invalid="ignore"):
                    bad = np.flatnonzero(~((np.abs(p.astype(float) - self.p[i]) <= self.off[i]) | (p == self.p[i]) | np.isnan(p)))
                assert not bad.size, what + "p %d: %r want %r" % (bad[0], p[bad[0]], self.p[i][bad[0]])
            for k, x in (("m", self.m), ("v", self.v)):
                got = self.arena[k].parts[i].cpu().numpy()
                if self.states == "f32":
                    same(got, x[i], what + k)
                    continue
                bad = np.flatnonzero(got[R.scales_at(n):] != x[i][R.scales_at(n):])
                assert not bad.size, what + "%s scale %d: %d want %d" % (k, bad[0], got[R.scales_at(n) + bad[0]], x[i][R.scales_at(n) + bad[0]])
                bad = np.flatnonzero(got[:n] != x[i][:n])
                assert not bad.size, what + "%s code %d: %d want %d" % (k, bad[0], got[bad[0]], x[i][bad[0]])
            if "pb" in self.arena:
                want = torch.from_numpy(p).bfloat16()
                assert torch.equal(self.arena["pb"].parts[i].cpu().nan_to_num(9), want.nan_to_num(9)), what + "copy"
            assert torch.equal(self.arena["g"].parts[i].cpu().nan_to_num(9), self.g[i].nan_to_num(9))
        for k, a in self.arena.items():
            if k in "mv" and self.states == "8bit":
                continue  # a state's own filling, checked below
            assert a.around_is_untouched(), k


@pytest.mark.parametrize("grad", ["f32", "bf16"])
@pytest.mark.parametrize("states", ["f32", "8bit"])
@pytest.mark.parametrize("start,gap", [(0, 0), (1, 3), (8, 16)])
def test_steps(states, grad, start, gap):
    c = Case(SIZES, states, grad, True, start, gap)
    for step in (1, 2, 50):
        cfg = dict(CFG, step=step)
        F.fsdp_adam_tensors(c.list, cfg, seed=5)
        c.reference([cfg], seed=5)
        c.check()


@pytest.mark.parametrize("states", ["f32", "8bit"])
def test_filling_between_codes_and_scales_stays(states):
    """The bytes that fill an 8-bit state's codes up to 16, and those behind its scales."""
    c = Case(SIZES, states, copy=False, start=3, gap=5)
    before = {k: c.arena[k].base.clone() for k in "mv"}
    F.fsdp_adam_tensors(c.list, CFG)
    for k in "mv":
        own = torch.zeros_like(before[k], dtype=torch.bool)
        for p, n in zip(c.arena[k].parts, SIZES):
            o = p.storage_offset()
            own[o:o + n] = True
            if states == "8bit":
                own[o + R.scales_at(n):o + R.state_bytes(n)] = True
        assert torch.equal(c.arena[k].base[~own], before[k][~own])


def test_like_the_single_shard():
    """fp32 states: the same bits as fsdp_adam_shard, tensor by tensor."""
    c = Case([1, 77, 4096, 50000], "f32", "f32", True)
    want = []
    for i, n in enumerate(c.sizes):
        u = F.fsdp_unit_create(F.FSDP_FLAT, [(n,)], 1)
        t = [c.arena[k].parts[i].clone() for k in ("p", "g", "m", "v")]
        pb = torch.empty(n, dtype=torch.bfloat16, device=dev())
        F.fsdp_adam_shard(u, *t, lr=CFG["lr"], betas=CFG["betas"], eps=CFG["eps"], weight_decay=CFG["weight_decay"], step=CFG["step"], param_bf16=pb)
        want.append((t[0], t[2], t[3], pb))
    F.fsdp_adam_tensors(c.list, CFG)
    for i, w in enumerate(want):
        for k, x in zip(("p", "m", "v", "pb"), w):
            assert torch.equal(c.arena[k].parts[i], x), (i, k)


@pytest.mark.parametrize("states", ["f32", "8bit"])
def test_many_tensors_and_groups(states):
    """More tensors than a launch's table holds, some without elements, of sixteen groups."""
    g = np.random.Generator(np.random.PCG64(1))
    sizes = [int(x) for x in g.integers(0, 300, 217)]
    groups = [int(x) for x in g.integers(0, 16, 217)]
    cfgs = [dict(lr=1e-3 * (i + 1), betas=(0.5 + 0.02 * i, 0.9 + 0.005 * i), eps=10.0 ** -(i % 9), weight_decay=0.01 * i, step=1 + 7 * i)
            for i in range(16)]
    c = Case(sizes, states, "bf16", True, groups=groups)
    for _ in range(2):
        F.fsdp_adam_tensors(c.list, cfgs, seed=123456789012345)
        c.reference(cfgs, seed=123456789012345)
    c.check()


@pytest.mark.parametrize("states", ["f32", "8bit"])
def test_clipping_and_skipping(states):
    c = Case([5, 3000, 64], states, "bf16")
    scale, skip = torch.tensor([0.37], device=dev()), torch.zeros(1, device=dev())
    F.fsdp_adam_tensors(c.list, CFG, grad_scale=scale, skip=skip, seed=1)
    c.reference([CFG], seed=1, gs=np.float32(0.37))
    c.check()
    for flag in (1.0, float("nan"), float("inf"), -2.0):
        skip.fill_(flag)
        F.fsdp_adam_tensors(c.list, CFG, grad_scale=scale, skip=skip, seed=1)
        c.check()


def test_some_tensors_have_a_copy():
    c = Case([100, 200, 300], "f32", copy=False)
    pb = [None, torch.empty(200, dtype=torch.bfloat16, device=dev()), None]
    a = {k: x.parts for k, x in c.arena.items()}
    F.fsdp_adam_tensors(F.AdamTensors(a["p"], a["g"], a["m"], a["v"], param_bf16=pb), CFG)
    c.reference([CFG])
    c.check()
    assert torch.equal(pb[1], a["p"][1].bfloat16())


def test_zero_state_is_a_first_step():
    n = 5000
    g = torch.randn(n, generator=torch.Generator().manual_seed(4)).to(dev())
    out = []
    for states in ("f32", "8bit"):
        p = torch.ones(n, device=dev())
        zero = torch.zeros(F.fsdp_adam_state_bytes(n), dtype=torch.uint8, device=dev()) if states == "8bit" else torch.zeros(n, device=dev())
        F.fsdp_adam_tensors(F.AdamTensors([p], [g], [zero], [zero.clone()], states=states), dict(lr=0.1, step=1))
        out.append(p)
    want, _, _, off = R.adam_f32(np.ones(n, np.float32), f32(g), np.zeros(n, np.float32), np.zeros(n, np.float32), dict(lr=0.1, step=1))
    assert_f32_bits(f32(out[0]), want)
    assert (np.abs(f32(out[1]).astype(float) - want) <= off).all()


@pytest.mark.parametrize("grad", ["f32", "bf16"])
@pytest.mark.parametrize("size", [1e-38, 1e-30, 1e-12, 1.0, 1e15, 1e19, 1e30])
def test_sizes_of_gradients(size, grad):
    """Gradients whose squares vanish, overflow, and lie anywhere between."""
    c = Case([4000], "8bit", grad, scale=size)
    for step in (1, 2):
        cfg = dict(CFG, step=step)
        F.fsdp_adam_tensors(c.list, cfg, seed=step)
        c.reference([cfg], seed=step)
        c.check()


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("states", ["f32", "8bit"])
def test_infinities_and_nan(states, bad):
    """They stay in their element, and in 8-bit states in their group, which reads as NaN from then on."""
    c = Case([300], states, "f32")
    for i in (0, 40, 299):
        c.g[0][i] = bad
    c.arena["g"].parts[0].copy_(c.g[0])
    for step in (1, 2):
        cfg = dict(CFG, step=step)
        F.fsdp_adam_tensors(c.list, cfg)
        c.reference([cfg])
        c.check()
    got = ~c.arena["p"].parts[0].isfinite().cpu()
    want = torch.zeros(300, dtype=torch.bool)
    if states == "8bit":
        want[:64] = want[288:] = True
    else:
        want[[0, 40, 299]] = True
    assert torch.equal(got, want)


def test_rounding_at_random_has_the_right_mean():
    """The state after one step from 0 of many equal gradients: codes on both sides of the exact value in the
    odds of its place (5 standard deviations of the mean, fixed seed; 2^-17 of a step is the random numbers'
    own coarseness)."""
    n = 1 << 16
    for x in (0.7317, 1.0, 3.3e-5):
        p, g = torch.zeros(n, device=dev()), torch.full((n,), x, device=dev())
        m, v = (torch.zeros(F.fsdp_adam_state_bytes(n), dtype=torch.uint8, device=dev()) for _ in range(2))
        F.fsdp_adam_tensors(F.AdamTensors([p], [g], [m], [v], states="8bit"), dict(lr=0.0, step=1), seed=3)
        x = float(g[0])
        for buf, which, exact in ((m, "m", np.float32(0.1) * np.float32(x)), (v, "v", np.float32(1 - 0.999) * (np.float32(x) * np.float32(x)))):
            got = R.read_state(buf.cpu().numpy(), n, which)
            lo, hi = got.min(), got.max()
            assert lo <= exact <= hi and hi - lo <= exact / 8
            step = max(hi - lo, exact / 16)
            assert abs(got.mean() - exact) <= step * (5 * 0.5 / n ** 0.5 + 2.0 ** -16)


# ---------------------------------------------------------------------------
# conversion
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("to", ["f32", "bf16"])
@pytest.mark.parametrize("start", [0, 1])
def test_convert(to, start):
    c = Case(SIZES + [0, 7] * 30, "8bit", start=start)
    sizes = c.sizes
    out = {k: Arena(sizes, T[to], start) for k in "mv"}
    values = F.AdamTensors(None, None, out["m"].parts, out["v"].parts, states=to)
    F.fsdp_adam_convert(c.list, values)
    for i, n in enumerate(sizes):
        for k, x in (("m", c.m), ("v", c.v)):
            assert np.array_equal(out[k].parts[i].double().cpu().numpy(), R.read_state(x[i], n, k)), (i, k)
    assert out["m"].around_is_untouched() and out["v"].around_is_untouched()
    # values that are codes come back as they were, whatever the seed; -0 stands for a negative code of 0
    back = Case(sizes, "8bit", start=start, seed=1)
    F.fsdp_adam_convert(values, back.list, seed=9, step=4)
    for i, n in enumerate(sizes):
        for k, x in (("m", c.m), ("v", c.v)):
            got = back.arena[k].parts[i].cpu().numpy()
            assert np.array_equal(R.read_state(got, n, k), R.read_state(x[i], n, k)), (i, k)


def test_convert_rounds_as_a_step_does():
    c = Case([1000, 333], "f32")
    q = Case([1000, 333], "8bit", seed=2)
    F.fsdp_adam_convert(c.list, q.list, seed=77, step=12)
    for i, n in enumerate(c.sizes):
        r = R.random16(n, R.key(77, 12, i))
        for k, x, u in (("m", c.m, r[0]), ("v", c.v, r[1])):
            got = q.arena[k].parts[i].cpu().numpy()
            want = R.write_state(x[i], u, k)
            assert np.array_equal(got[:n], want[:n]) and np.array_equal(got[R.scales_at(n):], want[R.scales_at(n):])


def test_every_code_converts():
    """All codes of both states at every scale, exactly."""
    byte = np.repeat(np.arange(256, dtype=np.uint8), 8)
    n = 32 * len(byte)
    codes = np.tile(np.arange(256, dtype=np.uint8), len(byte) // 8)
    buf = np.concatenate([codes, byte])
    assert len(buf) == R.state_bytes(n)
    state = torch.from_numpy(buf).to(dev())
    p = torch.empty(n, device=dev())
    out = [torch.empty(n, device=dev()) for _ in range(2)]
    F.fsdp_adam_convert(F.AdamTensors([p], [p], [state], [state], states="8bit"), F.AdamTensors(None, None, [out[0]], [out[1]]))
    for o, k in zip(out, "mv"):
        with np.errstate(over="ignore"):
            want = R.read_state(buf, n, k).astype(np.float32)
        got = o.cpu().numpy()
        # scales below the smallest that a rounding writes are only ever those of zeros
        told = np.repeat(byte >= (3 if k == "m" else 11), 32) & ~(np.isnan(want) if k == "m" else np.tile(np.arange(256) > 247, len(byte) // 8))
        assert np.array_equal(got[told], want[told], equal_nan=True)
        assert np.isnan(got[np.repeat(byte == 255, 32)]).all()


def test_refusals():
    n = 40
    t = [torch.zeros(n, device=dev()) for _ in range(4)]
    with pytest.raises(TypeError):
        F.AdamTensors([t[0].bfloat16()], [t[1]], [t[2]], [t[3]])
    with pytest.raises(TypeError):
        F.AdamTensors([t[0], t[1]], [t[1], t[1].bfloat16()], [t[2]] * 2, [t[3]] * 2)
    with pytest.raises(TypeError):
        F.AdamTensors([t[0]], [t[1]], [t[2]], [t[3]], states="8bit")
    with pytest.raises(ValueError, match="holds"):
        F.AdamTensors([t[0]], [t[1][:39]], [t[2]], [t[3]])
    with pytest.raises(ValueError, match="holds"):
        F.AdamTensors([t[0]], [t[1]], [torch.zeros(n, dtype=torch.uint8, device=dev())], [t[3]], states="8bit")
    with pytest.raises(ValueError, match="contiguous"):
        F.AdamTensors([torch.zeros(n, 2, device=dev())[:, 0]], [t[1]], [t[2]], [t[3]])
    with pytest.raises(ValueError, match="entries"):
        F.AdamTensors([t[0]], [t[1]], [t[2]], [t[3]], groups=[0, 1])
    with pytest.raises(ValueError, match="GPU"):
        F.AdamTensors([t[0].cpu()], [t[1]], [t[2]], [t[3]])
    a = F.AdamTensors([t[0]], [t[1]], [t[2]], [t[3]], groups=[1])
    with pytest.raises(F.FsdpError, match="group"):
        F.fsdp_adam_tensors(a, CFG)
    with pytest.raises(ValueError, match="GPU"):
        F.fsdp_adam_tensors(a, [CFG, CFG], grad_scale=torch.ones(1))
    b = F.AdamTensors(None, None, [t[0].bfloat16()], [t[0].bfloat16()], states="bf16")
    with pytest.raises(ValueError, match="params"):
        F.fsdp_adam_tensors(b, CFG)
    with pytest.raises(F.FsdpError, match="8BIT"):
        F.fsdp_adam_convert(a, b)


@pytest.mark.parametrize("copy", [False, True])
@pytest.mark.parametrize("states", ["f32", "8bit"])
@pytest.mark.parametrize("n", [64, 65, 79, 80, 87, 88, 97, 98, 250])
def test_lists_about_as_long_as_a_launch(n, states, copy):
    g = np.random.Generator(np.random.PCG64(n))
    sizes = [int(x) for x in g.integers(1, 70, n)]
    sizes[n // 2] = 5000
    c = Case(sizes, states, "f32", copy, groups=[int(x) for x in g.integers(0, 2, n)])
    cfgs = [CFG, dict(lr=1e-2, step=3)]
    F.fsdp_adam_tensors(c.list, cfgs, seed=8)
    c.reference(cfgs, seed=8)
    c.check()
    if states == "8bit":
        out = [[torch.empty(k, device=dev()) for k in sizes] for _ in range(2)]
        F.fsdp_adam_convert(c.list, F.AdamTensors(None, None, *out))
        for k, x, o in (("m", c.m, out[0]), ("v", c.v, out[1])):
            for i, size in enumerate(sizes):
                same(f32(o[i]), R.read_state(x[i], size, k).astype(np.float32), "%s %d" % (k, i))


def test_a_long_tensor_goes_on_in_the_next_launch():
    """Two short tensors, one of more tiles than a launch takes, and one behind it: every element steps once."""
    sizes = [3000, 7, (1 << 30) + 3000, 50]
    p, g, m, v = ([torch.full((n,), x, device=dev()) for n in sizes] for x in (0.5, 0.25, 0.0, 0.0))
    F.fsdp_adam_tensors(F.AdamTensors(p, g, m, v, groups=[0, 1, 0, 1]), [CFG, dict(CFG, lr=0.5)])
    for i, cfg in enumerate([CFG, dict(CFG, lr=0.5)] * 2):
        one = lambda x: np.full(1, x, np.float32)  # noqa: E731
        want = R.adam_f32(one(0.5), one(0.25), one(0), one(0), cfg)
        for got, w in zip((p[i], m[i], v[i]), want):
            assert float(got.min()) == float(got.max()) == float(w[0]), i
