"""Rotary positions, token log probabilities and AdamW over many tensors as a training step uses them: together,
with gradients against 64-bit autograd; captured into graphs and replayed; on streams of their own; past 32-bit
offsets and in several launches."""
import numpy as np
import pytest
import torch

import sharded_fsdp_flatten_amd as F
import train_ref as R
from gpu_util import dev

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def normal(seed, *shape, scale=1.0, dtype=torch.float32):
    g = torch.Generator(device=dev()).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=dev()) * scale).to(dtype)


# ---------------------------------------------------------------------------
# a training step of one attention layer over a small vocabulary
# ---------------------------------------------------------------------------
class Layer:
    """h = embed[tokens]; q, k, v = h Wqkv; rotary q, k; causal attention; h + o Wo; logits = that embed^T;
    the loss is the mean of -log p of the next tokens that are not padding, less 0.01 of the mean entropy."""

    B, T, H, D, V = 2, 24, 3, 16, 97
    names = ("embed", "qkv", "out")

    def __init__(self, seed):
        d = self.H * self.D
        self.params = {"embed": normal(seed, self.V, d, scale=0.5), "qkv": normal(seed + 1, d, 3 * d, scale=d ** -0.5),
                       "out": normal(seed + 2, d, d, scale=d ** -0.5)}
        g = torch.Generator(device=dev()).manual_seed(seed + 3)
        self.tokens = torch.randint(0, self.V, (self.B, self.T), generator=g, device=dev())
        self.labels = torch.randint(0, self.V, (self.B, self.T), generator=g, device=dev())
        self.labels[0, -5:] = -100
        self.freqs = F.fsdp_rotary_freqs(self.D, scaling="linear", factor=2.0)

    def gradients(self):
        """Through the library's calls; matrix products and attention are torch's, in fp32."""
        B, T, H, D, V = self.B, self.T, self.H, self.D, self.V
        f = self.freqs.to(dev())
        p = {k: v.clone().requires_grad_() for k, v in self.params.items()}
        h = p["embed"][self.tokens.view(-1)]
        qkv = (h @ p["qkv"]).view(B, T, 3, H, D)
        rot = qkv.detach().clone()
        F.fsdp_rotary_forward(rot[:, :, 0], rot[:, :, 0], f, k=rot[:, :, 1], k_out=rot[:, :, 1])
        rot.requires_grad_()
        q, k, v = (rot[:, :, i].transpose(1, 2) for i in range(3))
        s = (q @ k.transpose(2, 3)) * D ** -0.5
        s = s.masked_fill(torch.ones(T, T, dtype=torch.bool, device=dev()).triu(1), -float("inf"))
        o = (s.softmax(-1) @ v).transpose(1, 2).reshape(B * T, H * D)
        top = h + o @ p["out"]
        logits = top @ p["embed"].t()
        n = B * T
        lp, mx, ls, ent = (torch.empty(n, device=dev()) for _ in range(4))
        labels = self.labels.view(-1)
        F.fsdp_logprob_forward(logits.detach(), labels, lp, mx, ls, entropy=ent)
        count = int((labels >= 0).sum())
        loss = -lp.sum() / count - 0.01 * ent.mean()
        dl, dh = torch.full((n,), -1.0 / count, device=dev()), torch.full((n,), -0.01 / n, device=dev())
        dlogits = logits.detach().clone()
        F.fsdp_logprob_backward(dlogits, labels, dl, mx, ls, dlogits, dentropy=dh, entropy=ent)
        drot, = torch.autograd.grad(logits, rot, dlogits, retain_graph=True)
        grads = dict(zip(self.names, torch.autograd.grad(logits, [p[k] for k in self.names], dlogits, retain_graph=True, allow_unused=True)))
        F.fsdp_rotary_backward(drot[:, :, 0], drot[:, :, 0], f, k=drot[:, :, 1], k_out=drot[:, :, 1])
        for name, g in zip(("embed", "qkv"), torch.autograd.grad(qkv, [p["embed"], p["qkv"]], drot)):
            grads[name] = g if grads[name] is None else grads[name] + g
        return float(loss), {k: g.contiguous() for k, g in grads.items()}

    def reference(self):
        """The same in float64 on the CPU, by autograd of the definitions."""
        B, T, H, D, V = self.B, self.T, self.H, self.D, self.V
        p = {k: v.detach().cpu().double().requires_grad_() for k, v in self.params.items()}
        h = p["embed"][self.tokens.cpu().view(-1)]
        qkv = (h @ p["qkv"]).view(B, T, 3, H, D)
        w = torch.arange(T, dtype=torch.float64)[:, None] * self.freqs
        c, s = w.cos()[:, None], w.sin()[:, None]

        def turn(x):
            a, b = x[..., : D // 2], x[..., D // 2:]
            return torch.cat([a * c - b * s, a * s + b * c], -1).transpose(1, 2)

        q, k, v = turn(qkv[:, :, 0]), turn(qkv[:, :, 1]), qkv[:, :, 2].transpose(1, 2)
        a = (q @ k.transpose(2, 3)) * D ** -0.5
        a = a.masked_fill(torch.ones(T, T, dtype=torch.bool).triu(1), -float("inf"))
        o = (a.softmax(-1) @ v).transpose(1, 2).reshape(B * T, H * D)
        logp = ((h + o @ p["out"]) @ p["embed"].t()).log_softmax(-1)
        labels = self.labels.cpu().view(-1)
        has = labels >= 0
        ent = -(logp.exp() * logp).sum(-1)
        loss = -logp[has, labels[has]].mean() - 0.01 * ent.mean()
        return float(loss.detach()), dict(zip(self.names, torch.autograd.grad(loss, [p[k] for k in self.names])))


def test_a_training_step():
    """Loss and gradients within the roundings of fp32: ten operations one after another, sums of at most 144 terms
    (embedding gradients: B T + V), each rounding relative to its terms' size, which stay within 8 of the largest
    gradient: 10 x 144 x 8 U.  Then clipped AdamW with fp32 and 8-bit states takes the same gradients."""
    layer = Layer(5)
    loss, grads = layer.gradients()
    want_loss, want = layer.reference()
    assert abs(loss - want_loss) <= 10 * 144 * U * max(1.0, abs(want_loss))
    for k in layer.names:
        off = (grads[k].cpu().double() - want[k]).abs().max() / want[k].abs().max()
        assert off <= 10 * 144 * 8 * U, (k, float(off))
    sizes = [layer.params[k].numel() for k in layer.names]
    unit = F.fsdp_unit_create(F.FSDP_FLAT, [(n,) for n in sizes], 1)
    flat = torch.cat([grads[k].view(-1) for k in layer.names])
    sq, ws = torch.empty(3, dtype=torch.float64, device=dev()), torch.empty(F.fsdp_grad_sqnorm_workspace(unit, 0), dtype=torch.float64, device=dev())
    F.fsdp_grad_sqnorm(unit, 0, flat, sq, ws)
    clip = (0.5 / sq.sum().sqrt()).clamp(max=1.0).float().view(1)
    groups = [dict(lr=1e-2, step=1, weight_decay=0.1), dict(lr=1e-3, step=1)]
    for states in ("f32", "8bit"):
        p = [layer.params[k].clone().view(-1) for k in layer.names]
        held = (lambda n: torch.zeros(F.fsdp_adam_state_bytes(n), dtype=torch.uint8, device=dev())) if states == "8bit" else (
            lambda n: torch.zeros(n, device=dev()))
        m, v = [held(n) for n in sizes], [held(n) for n in sizes]
        g = [grads[k].view(-1) for k in layer.names]
        F.fsdp_adam_tensors(F.AdamTensors(p, g, m, v, states=states, groups=[0, 0, 1]), groups, grad_scale=clip, seed=3)
        for i, k in enumerate(layer.names):
            zero = np.zeros(sizes[i], np.float32)
            q, _, _, off = R.adam_f32(layer.params[k].view(-1).cpu().numpy(), g[i].cpu().numpy(), zero, zero, groups[0 if i < 2 else 1],
                                      clip.cpu().numpy()[0])
            d = np.abs(p[i].cpu().numpy().astype(float) - q)
            assert (d <= (0 if states == "f32" else off)).all(), (states, k)


# ---------------------------------------------------------------------------
# graphs
# ---------------------------------------------------------------------------
def captured(step):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    return g


@pytest.mark.parametrize("rows,cols,top", [(3, 200003, 20), (40, 5003, 5), (700, 3001, 0)])
def test_logprob_graph(rows, cols, top):
    """Forward (split rows and whole ones) and backward in one graph, replayed on new logits with eager work
    between, gives the eager calls' bits."""
    x = normal(1, rows, cols, scale=3.0, dtype=torch.bfloat16)
    tok = torch.randint(0, cols, (rows,), device=dev())

    def buffers():
        o = {k: torch.empty(rows, device=dev()) for k in ("lp", "mx", "ls", "ent")}
        o |= {"dx": torch.empty_like(x), "ws": torch.empty(F.fsdp_logprob_workspace(rows, cols, top), device=dev())}
        if top:
            o |= {"tl": torch.empty(rows, top, device=dev()), "tt": torch.empty(rows, top, dtype=torch.int64, device=dev())}
        return o

    dl, dh = normal(2, rows), normal(3, rows)

    def step(o):
        F.fsdp_logprob_forward(x, tok, o["lp"], o["mx"], o["ls"], o["ws"], scale=0.9, entropy=o["ent"], top_logprob=o.get("tl"), top_token=o.get("tt"))
        F.fsdp_logprob_backward(x, tok, dl, o["mx"], o["ls"], o["dx"], scale=0.9, dentropy=dh, entropy=o["ent"])

    a, b = buffers(), buffers()
    g = captured(lambda: step(a))
    for i in range(4):
        x.copy_(normal(10 + i, rows, cols, scale=3.0, dtype=torch.bfloat16))
        tok.copy_(torch.randint(-1, cols, (rows,), device=dev()))
        step(b)
        torch.cuda.synchronize()
        a["ws"].fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        for k in set(a) - {"ws"}:
            assert torch.equal(a[k], b[k]), (i, k)


@pytest.mark.parametrize("states", ["f32", "8bit"])
def test_adam_graph(states):
    """A step over more tensors than a launch holds, clipped and skipped from the device, replayed."""
    sizes = [100 + 37 * i for i in range(70)]

    def make():
        p = [normal(i, n) for i, n in enumerate(sizes)]
        held = (lambda n: torch.zeros(F.fsdp_adam_state_bytes(n), dtype=torch.uint8, device=dev())) if states == "8bit" else (
            lambda n: torch.zeros(n, device=dev()))
        return p, [held(n) for n in sizes], [held(n) for n in sizes]

    grads = [normal(1000 + i, n) for i, n in enumerate(sizes)]
    scale, skip = torch.ones(1, device=dev()), torch.zeros(1, device=dev())
    sides = []
    for _ in range(2):
        p, m, v = make()
        sides.append((p, m, v, F.AdamTensors(p, grads, m, v, states=states)))
    run = lambda s: F.fsdp_adam_tensors(s[3], dict(lr=0.01, step=5), seed=2, grad_scale=scale, skip=skip)  # noqa: E731
    g = captured(lambda: run(sides[0]))
    run(sides[1])    # the warm-up was a step; the capture was none
    for i in range(4):
        for t in grads:
            t.mul_(0.9)
        scale.fill_(0.5 + i)
        skip.fill_(float(i == 2))
        run(sides[1])
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for k in range(3):
            for a, b in zip(sides[0][k], sides[1][k]):
                assert torch.equal(a, b), (i, k)


def test_rotary_and_convert_graph():
    q, k = normal(1, 2, 9, 5, 32, dtype=torch.bfloat16), normal(2, 2, 9, 2, 32, dtype=torch.bfloat16)
    f = F.fsdp_rotary_freqs(32).to(dev())
    pos = torch.zeros(2, 9, dtype=torch.int64, device=dev())
    n = 5000
    p = torch.empty(n, device=dev())
    m, v = normal(3, n), normal(4, n).square()
    small = [torch.empty(F.fsdp_adam_state_bytes(n), dtype=torch.uint8, device=dev()) for _ in range(2)]
    out = [torch.empty(n, device=dev()) for _ in range(2)]
    lists = [F.AdamTensors(None, None, [m], [v]), F.AdamTensors([p], [p], [small[0]], [small[1]], states="8bit"), F.AdamTensors(None, None, [out[0]], [out[1]])]
    qo, ko = torch.empty_like(q), torch.empty_like(k)

    def step():
        F.fsdp_rotary_forward(q, qo, f, k=k, k_out=ko, positions=pos)
        F.fsdp_adam_convert(lists[0], lists[1], seed=1, step=2)
        F.fsdp_adam_convert(lists[1], lists[2])

    g = captured(step)
    for i in range(3):
        pos.random_(0, 5000)
        m.mul_(1.7)
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (qo, ko, *out)]
        for t in (qo, ko, *out):
            t.zero_()
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (qo, ko, *out)):
            assert torch.equal(a, b), i


# ---------------------------------------------------------------------------
# streams
# ---------------------------------------------------------------------------
def test_two_streams_at_once():
    """Calls on two streams, each with a workspace of its own, disturb neither."""
    rows, cols, top = 4, 150001, 40
    xs = [normal(i, rows, cols, scale=3.0) for i in range(2)]
    tok = torch.randint(0, cols, (rows,), device=dev())

    def buffers():
        return ([torch.empty(rows, device=dev()) for _ in range(4)], torch.empty(rows, top, device=dev()),
                torch.empty(rows, top, dtype=torch.int64, device=dev()), torch.empty(F.fsdp_logprob_workspace(rows, cols, top), device=dev()),
                torch.empty(rows, cols, device=dev()))

    def step(x, b, stream=None):
        F.fsdp_logprob_forward(x, tok, b[0][0], b[0][1], b[0][2], b[3], entropy=b[0][3], top_logprob=b[1], top_token=b[2], stream=stream)
        F.fsdp_logprob_backward(x, tok, b[0][0], b[0][1], b[0][2], b[4], stream=stream)

    alone, both = [buffers() for _ in range(2)], [buffers() for _ in range(2)]
    for x, b in zip(xs, alone):
        step(x, b)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for x, b, s in zip(xs, both, streams):
            step(x, b, s)
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        for i in (1, 2, 4):
            assert torch.equal(a[i], b[i])
        for u, v in zip(a[0], b[0]):
            assert torch.equal(u, v)


# ---------------------------------------------------------------------------
# long
# ---------------------------------------------------------------------------
def test_logits_past_32_bits():
    """70000 x 50257 bf16 logits: 3.5e9 elements; the last rows, and the gradient in their place."""
    rows, cols = 70000, 50257
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device=dev())
    x.fill_(-3.0)
    some = [0, 1, rows // 2, 42725, 42726, rows - 2, rows - 1]   # 2^31 lies in row 42729
    for i, r in enumerate(some):
        x[r] = normal(i, cols, scale=3.0, dtype=torch.bfloat16)
    tok = torch.arange(rows, device=dev()) % cols
    o = [torch.empty(rows, device=dev()) for _ in range(4)]
    tl, tt = torch.empty(rows, 3, device=dev()), torch.empty(rows, 3, dtype=torch.int64, device=dev())
    F.fsdp_logprob_forward(x, tok, o[0], o[1], o[2], entropy=o[3], top_logprob=tl, top_token=tt)
    part = x[some].double().cpu().numpy()
    want = R.logprob(part, tok[some].cpu().numpy(), 1.0)
    for got, k, e in ((o[0], "logprob", "elogprob"), (o[2], "logsum", "elogsum"), (o[3], "entropy", "eentropy")):
        assert (np.abs(got[some].double().cpu().numpy() - want[k]) <= want[e]).all(), k
    assert np.array_equal(tt[some].cpu().numpy(), R.top(part, 3))
    dl = torch.ones(rows, device=dev())
    F.fsdp_logprob_backward(x, tok, dl, o[1], o[2], x)
    ones, zero = np.ones(len(some)), np.zeros(len(some))
    f = lambda t: t[some].double().cpu().numpy()  # noqa: E731
    grad, bound = R.logprob_grad(part, tok[some].cpu().numpy(), ones, zero, f(o[1]), f(o[2]), zero, 1.0, "bf16")
    assert (np.abs(f(x) - grad) <= bound).all()


def test_rows_of_several_launches():
    """More rows than one launch of the forward pass takes (2^20), and than one of the backward pass (2^24)."""
    rows, cols = (1 << 24) + 77, 3
    x = normal(1, rows, cols)
    tok = torch.randint(-1, cols + 1, (rows,), device=dev())
    lp, mx, ls = (torch.empty(rows, device=dev()) for _ in range(3))
    F.fsdp_logprob_forward(x, tok, lp, mx, ls)
    dl, dx = normal(2, rows), torch.empty_like(x)
    F.fsdp_logprob_backward(x, tok, dl, mx, ls, dx)
    for lo in (0, (1 << 20) - 50, (1 << 23) - 50, rows - 200):
        part = slice(lo, lo + 200)
        xs, ts = x[part].double().cpu().numpy(), tok[part].cpu().numpy()
        want = R.logprob(xs, ts, 1.0)
        f = lambda t: t[part].double().cpu().numpy()  # noqa: E731
        assert (np.abs(f(lp) - want["logprob"]) <= want["elogprob"]).all()
        grad, bound = R.logprob_grad(xs, ts, f(dl), np.zeros(200), f(mx), f(ls), np.zeros(200), 1.0, "f32")
        assert (np.abs(f(dx) - grad) <= bound).all()


def test_a_tensor_past_32_bits():
    """One tensor of 2^32 + 5003 elements in 8 bits: several launches, element numbers past 32 bits, the last
    group short; and a neighbour behind it."""
    n = (1 << 32) + 5003
    p = torch.full((n,), 0.5, device=dev())
    g = torch.full((n,), 0.25, dtype=torch.bfloat16, device=dev())
    m, v = (torch.zeros(F.fsdp_adam_state_bytes(n), dtype=torch.uint8, device=dev()) for _ in range(2))
    q = [torch.full((7,), 0.5, device=dev()), torch.full((7,), 0.25, dtype=torch.bfloat16, device=dev()),
         *(torch.zeros(F.fsdp_adam_state_bytes(7), dtype=torch.uint8, device=dev()) for _ in range(2))]
    places = [0, (1 << 30) - 64, (1 << 31) - 64, (1 << 32) - 64, (1 << 32) + 4800]
    for at in places:
        g[at:at + 200] = normal(at % 1000, 200, dtype=torch.bfloat16)
    cfg = dict(lr=1e-2, step=4)
    F.fsdp_adam_tensors(F.AdamTensors([p, q[0]], [g, q[1]], [m, q[2]], [v, q[3]], states="8bit"), cfg, seed=6)
    scales = R.scales_at(n)
    for at in places:
        lo = at // 32 * 32
        hi = min(n, lo + 256)
        k = hi - lo
        zero = np.zeros(k, np.float32)
        want, mm, vv, off = R.adam_f32(np.full(k, 0.5, np.float32), g[lo:hi].float().cpu().numpy(), zero, zero, cfg)
        assert (np.abs(p[lo:hi].cpu().numpy().astype(float) - want) <= off).all()
        r = R.random16(k, R.key(6, 4, 0), first=lo)
        for buf, x, u, which in ((m, mm, r[0], "m"), (v, vv, r[1], "v")):
            state = R.write_state(x, u, which)
            assert np.array_equal(buf[lo:hi].cpu().numpy(), state[:k]), (at, which)
            got = buf[scales + lo // 32:scales + -(-hi // 32)].cpu().numpy()
            assert np.array_equal(got, state[R.scales_at(k):]), (at, which)
    assert (q[0] < 0.5).all() and (q[2][:7] != 0).all()


def test_rotary_of_several_launches_and_far_offsets():
    """More tokens than a launch's workgroups (2^20) with heads far apart, so that offsets pass 32 bits."""
    tokens, heads = (1 << 20) + 99, 300
    x = torch.empty(heads, tokens, 8, dtype=torch.bfloat16, device=dev()).transpose(0, 1)   # 2.5e9 elements
    x.fill_(1.0)
    f = F.fsdp_rotary_freqs(8).to(dev())
    some = [0, 1 << 19, (1 << 20) - 1, 1 << 20, tokens - 1]
    src = normal(1, len(some), heads, 8, dtype=torch.bfloat16)
    x[some] = src
    F.fsdp_rotary_forward(x, x, f)
    want, bound = R.rotary(src[None].double().cpu().numpy(), f.cpu().numpy(), np.array([some]), "half", 1.0, 1, "bf16")
    assert (np.abs(x[some][None].double().cpu().numpy() - want) <= bound).all()


# ---------------------------------------------------------------------------
# lists of tensors
# ---------------------------------------------------------------------------
def test_a_list_refuses_what_is_there_twice():
    p, m, v = (torch.zeros(100, device=dev()) for _ in range(3))
    q, r = torch.zeros(200, device=dev()), torch.zeros(200, device=dev())
    good = ([p, q[:100]], [p, q[:100]], [m, r[:100]], [v, r[100:]])
    F.AdamTensors(*good)
    F.AdamTensors([p, p[:0]], [p, p[:0]], [m, m[:0]], [v, v[:0]])                    # nothing overlaps nothing
    one = torch.zeros(1, device=dev())
    for bad in (([p, p], *good[1:]), ([p, p[99:]], [p, one], [m, one], [v, one.clone()]), (*good[:2], [m, m], good[3]),
                (*good[:3], [v, r[99:199]]), (*good[:2], [m, p], good[3])):
        with pytest.raises(ValueError, match="overlap"):
            F.fsdp_adam_tensors(F.AdamTensors(*bad), dict(lr=1e-3, step=1))
    copy = F.AdamTensors([p], [m], [q[:100]], [v], param_bf16=[q[50:100].view(torch.bfloat16)])
    with pytest.raises(ValueError, match="overlap"):
        F.fsdp_adam_tensors(copy, dict(lr=1e-3, step=1))
    state = torch.zeros(F.fsdp_adam_state_bytes(100), dtype=torch.uint8, device=dev())
    small = F.AdamTensors([p], [p], [state], [state], states="8bit")
    F.fsdp_adam_convert(small, F.AdamTensors(None, None, [m], [v]))           # read twice
    with pytest.raises(ValueError, match="overlap"):
        F.fsdp_adam_convert(F.AdamTensors(None, None, [m], [v]), small)
    with pytest.raises(TypeError, match=r"params\[1\]"):
        F.AdamTensors([p, None], [p, p], [m, r[:100]], [v, r[100:]])


@pytest.mark.parametrize("states", ["f32", "8bit"])
def test_a_list_holds_its_memory(states):
    """Where a parameter is given other storage after the list was made, a step writes what the list holds."""
    n = 1 << 20
    held = F.fsdp_adam_state_bytes(n) if states == "8bit" else n
    kind = torch.uint8 if states == "8bit" else torch.float32
    p, g = torch.ones(n, device=dev()), torch.ones(n, device=dev())
    m, v = torch.zeros(held, dtype=kind, device=dev()), torch.zeros(held, dtype=kind, device=dev())
    t = F.AdamTensors([p], [g], [m], [v], states=states)
    for x in (p, g, m, v):
        x.data = torch.zeros(1, dtype=x.dtype, device=dev())
    others = [torch.full((n,), 7.0, device=dev()) for _ in range(8)]    # would take freed memory
    F.fsdp_adam_tensors(t, dict(lr=0.1, step=1))
    torch.cuda.synchronize()
    assert all(bool((x == 7).all()) for x in others) and float(p.sum()) == 0.0


@pytest.mark.parametrize("scale", [2.0 ** 127, 2.0 ** -100])
def test_logprob_at_the_ends_of_the_scale(scale):
    x = normal(1, 5, 700)
    if scale > 1:
        x = x.sign() * 2.0 ** -120 * x.abs()
    tok = torch.arange(5, device=dev())
    o = [torch.empty(5, device=dev()) for _ in range(4)]
    F.fsdp_logprob_forward(x, tok, o[0], o[1], o[2], scale=scale, entropy=o[3])
    want = R.logprob(x.double().cpu().numpy(), tok.cpu().numpy(), scale)
    for got, k, e in ((o[0], "logprob", "elogprob"), (o[2], "logsum", "elogsum"), (o[3], "entropy", "eentropy")):
        assert (np.abs(got.double().cpu().numpy() - want[k]) <= want[e]).all(), k


# ---------------------------------------------------------------------------
# arguments that may be left out, shapes of several dimensions
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("batch,tokens,cols", [(2, 3, 50257), (2, 3, 200000), (64, 33, 50257), (5, 7, 300), (3, 70, 9000)])
def test_logprob_of_a_batch_with_and_without_tokens(batch, tokens, cols):
    """[batch, tokens, cols] logits; statistics are the same bits with tokens and without."""
    x = normal(1, batch, tokens, cols, scale=3.0, dtype=torch.bfloat16)
    tok = torch.randint(-1, cols, (batch, tokens), device=dev())
    n, top = (batch, tokens), 5
    ws = torch.empty(F.fsdp_logprob_workspace(batch * tokens, cols, top), device=dev())
    lp, m1, s1, m2, s2, m3, s3, h = (torch.full(n, 7.0, device=dev()) for _ in range(8))
    tl, tt = torch.empty(*n, top, device=dev()), torch.empty(*n, top, dtype=torch.int64, device=dev())
    F.fsdp_logprob_forward(x, tok, lp, m1, s1, ws, entropy=h)
    F.fsdp_logprob_forward(x, None, None, m2, s2, ws)
    F.fsdp_logprob_forward(x, None, None, m3, s3, ws, top_logprob=tl, top_token=tt)
    assert torch.equal(m1, m2) and torch.equal(s1, s2) and torch.equal(m1, m3)
    rows = slice(0, 50)
    want = R.logprob(x.view(-1, cols)[rows].double().cpu().numpy(), tok.view(-1)[rows].cpu().numpy(), 1.0)
    # with alternatives a row's sum may be taken by another number of lanes, in another order: each of the two is within the
    # bound of the exact one
    for s in (s1, s3):
        assert (np.abs(s.view(-1)[rows].double().cpu().numpy() - want["logsum"]) <= want["elogsum"]).all()
    assert (np.abs(lp.view(-1)[rows].double().cpu().numpy() - want["logprob"]) <= want["elogprob"]).all()
    assert np.array_equal(tt.view(-1, top)[rows].cpu().numpy(), R.top(x.view(-1, cols)[rows].double().cpu().numpy(), top))
    # the gradient of the entropies alone, and of both as the sum of the parts
    dl, dh, zero = normal(2, *n), normal(3, *n), torch.zeros(n, device=dev())
    both, only, with_zero = (torch.empty_like(x) for _ in range(3))
    F.fsdp_logprob_backward(x, None, None, m1, s1, only, dentropy=dh, entropy=h)
    F.fsdp_logprob_backward(x, tok, zero, m1, s1, with_zero, dentropy=dh, entropy=h)
    assert torch.equal(only, with_zero)
    F.fsdp_logprob_backward(x, tok, dl, m1, s1, both, dentropy=dh, entropy=h)
    F.fsdp_logprob_backward(x, tok, dl, m1, s1, x)
    f = lambda t: t.view(-1, cols)[rows].double()  # noqa: E731
    # three roundings to bf16, of each part and of the sum
    assert ((f(both) - f(x) - f(only)).abs() <= 2.0 ** -8 * (f(both).abs() + f(x).abs() + f(only).abs()) * 1.01 + 1e-6).all()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_without_queries_or_batch(layout):
    k = normal(1, 9, 3, 24)
    f = F.fsdp_rotary_freqs(16).to(dev())
    want = torch.empty_like(k)
    F.fsdp_rotary_forward(k, want, f, start=5, layout=layout)
    got, q = torch.empty_like(k), torch.empty(9, 0, 24, device=dev())
    F.fsdp_rotary_forward(q, q, f, k=k, k_out=got, start=5, layout=layout)
    assert torch.equal(got, want)
    batched = torch.empty(1, 9, 3, 24, device=dev())
    F.fsdp_rotary_forward(k[None], batched, f, positions=torch.arange(5, 14, device=dev())[None], layout=layout)
    assert torch.equal(batched[0], want)
