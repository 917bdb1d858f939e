"""The layer operators of an FSDP unit as measured work: 8-bit activation checkpoints, the norms and the
activations of a transformer block, forward and backward.

`run` computes them in their plain form from elementary torch operations, or, where `own` is true, through
sharded_fsdp_flatten_amd.  A case is one of five paths:

  ckpt       an activation is packed to 8 bits and read back
  norm_fwd   (residual add and) LayerNorm or RMSNorm of the tokens, with the statistics the backward pass needs
  norm_bwd   gradients of the norm's input, weight and bias from the saved input (and the residual stream's
             gradient added to the input's)
  norm_step  both with the input saved in 8 bits: forward with checkpoint, then backward from it, which also
             gives the norm's output again (the next matrix product's weight gradient needs it)
  act_step   the same for the MLP's activation; its backward pass gives the gradient of the bias before it
"""
import math

import torch

own = False

GROUP = 32          # columns that share one scale
EPS = {"layer": 1e-5, "rms": 1e-6}
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # a GPT-2 Large block's norm on a handful of tokens: launch latency
        dict(name="norm_fwd few tokens", op="norm_fwd", rows=16, cols=1280, dtype="bf16", kind="layer", residual=False),
        # the same norm wide, as a GPT-175B block has it, with the residual add before it
        dict(name="norm_fwd 175B residual", op="norm_fwd", rows=4096, cols=12288, dtype="bf16", kind="layer", residual=True),
        # T5's RMSNorm with fp32 activations, an odd number of tokens
        dict(name="norm_fwd T5 f32", op="norm_fwd", rows=4099, cols=1024, dtype="f32", kind="rms", residual=False),
        # backward of a GPT-2 Large norm on a 4 x 1024 micro-batch, the residual stream's gradient added
        dict(name="norm_bwd GPT-2-L", op="norm_bwd", rows=4096, cols=1280, dtype="bf16", kind="layer", residual=True),
        # backward of a GPT-175B norm on 8192 tokens
        dict(name="norm_bwd 175B", op="norm_bwd", rows=8192, cols=12288, dtype="bf16", kind="layer", residual=False),
        # a ragged batch of odd width: rows start at any element
        dict(name="norm_bwd ragged", op="norm_bwd", rows=777, cols=5003, dtype="bf16", kind="rms", residual=False),
        # a GPT-2 Large norm, forward with an 8-bit checkpoint and backward from it
        dict(name="norm_step GPT-2-L e4m3", op="norm_step", rows=16384, cols=1280, dtype="bf16", kind="layer", format="e4m3"),
        # T5's, integer codes
        dict(name="norm_step T5 int8", op="norm_step", rows=32768, cols=1024, dtype="bf16", kind="rms", format="int8"),
        # the input of a GPT-175B block saved in 8 bits and read back
        dict(name="ckpt 175B e4m3", op="ckpt", rows=8192, cols=12288, dtype="bf16", format="e4m3"),
        # odd width in fp32: rows end inside a group
        dict(name="ckpt ragged f32", op="ckpt", rows=1023, cols=1283, dtype="f32", format="int8"),
        # a GPT-2 Large MLP's GELU on a 4 x 1024 micro-batch
        dict(name="act_step GPT-2-L", op="act_step", rows=4096, cols=5120, dtype="bf16", kind="gelu_tanh", format="e4m3"),
        # T5-11B's wide ReLU
        dict(name="act_step T5", op="act_step", rows=2048, cols=65536, dtype="bf16", kind="relu", format="int8"),
    ]


def draw(rng):
    op = rng.choice(["ckpt", "norm_fwd", "norm_bwd", "norm_step", "act_step"])
    most = 96 * 1024 * 1024 if op != "norm_step" else 24 * 1024 * 1024
    cols = int(round(math.exp(rng.uniform(math.log(33), math.log(65536 if op == "act_step" else 16384)))))
    if rng.random() < 0.5:
        cols = -(-cols // 64) * 64
    rows = int(round(math.exp(rng.uniform(math.log(1), math.log(min(32768, most // cols))))))
    c = dict(op=op, rows=rows, cols=cols, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if c["dtype"] == "f32":
        c["rows"] = max(1, rows // 2)
    if op.startswith("norm"):
        c["kind"] = rng.choice(["layer", "rms"])
    if op in ("norm_fwd", "norm_bwd"):
        c["residual"] = rng.random() < 0.5
    if op == "act_step":
        c["kind"] = rng.choice(["relu", "gelu", "gelu_tanh", "silu"])
    if op in ("ckpt", "norm_step", "act_step"):
        c["format"] = rng.choice(["e4m3", "int8"])
    return c


def _inputs(case, seed):
    """Inputs of a case: activations with a few large channels and tokens of different size, as a residual
    stream has them; gradients small against them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    R, C, t = case["rows"], case["cols"], DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    x = normal(R, C)
    if case["op"] != "act_step":
        channel = torch.where(torch.rand(C, device="cuda", generator=g) < 0.004, 20.0, 1.0)
        x = x * channel * torch.exp(0.5 * normal(R, 1)) + 0.1 * normal(C)
    inp = {"x": x.to(t)}
    if case["op"] == "ckpt":
        return inp
    if case["op"].startswith("norm"):
        inp["w"] = (1.0 + 0.1 * normal(C)).to(torch.bfloat16)
        inp["b"] = (0.1 * normal(C)).to(torch.bfloat16) if case["kind"] == "layer" else None
    if case.get("residual"):
        inp["r"] = (0.01 * normal(R, C) if case["op"] == "norm_bwd" else normal(R, C)).to(t)
    if case["op"] != "norm_fwd":
        inp["dy"] = (0.01 * normal(R, C)).to(t)
    if case["op"] == "norm_bwd":
        x64 = inp["x"].double()
        m = x64.mean(1) if case["kind"] == "layer" else torch.zeros(R, device="cuda", dtype=torch.float64)
        v = (x64 - m[:, None]).square().mean(1)
        inp["mean"] = m.float() if case["kind"] == "layer" else None
        inp["rstd"] = (v + EPS[case["kind"]]).rsqrt().float()
    return inp


def prepare(case, seed):
    inp = _inputs(case, seed)
    st = dict(case=case, **inp)
    R, C, t = case["rows"], case["cols"], DTYPES[case["dtype"]]
    new = lambda *shape, dtype=t: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    f32 = torch.float32
    op = case["op"]
    st["y"] = new(R, C)
    if op.startswith("norm"):
        st["rstd_out"] = new(R, dtype=f32)
        st["mean_out"] = new(R, dtype=f32) if case["kind"] == "layer" else None
        st["sum"] = new(R, C) if op == "norm_fwd" and case["residual"] else None
    if op in ("norm_bwd", "norm_step", "act_step"):
        st["dx"] = new(R, C)
        st["again"] = new(R, C) if op != "norm_bwd" else None
        st["dw"] = new(C, dtype=f32) if op != "act_step" else None
        st["db"] = new(C, dtype=f32) if op == "act_step" or case["kind"] == "layer" else None
    if own:
        import sharded_fsdp_flatten_amd as F
        st["F"] = F
        if "format" in case:
            st["ckpt"] = F.Ckpt.empty(R, C, case["format"], device="cuda")
        if op in ("norm_bwd", "norm_step"):
            st["ws"] = new(F.fsdp_norm_workspace(R, C), dtype=f32)
        if op == "act_step":
            st["ws"] = new(F.fsdp_act_workspace(R, C), dtype=f32)
    return st


def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    F, case = st["F"], st["case"]
    op = case["op"]
    if op == "ckpt":
        F.fsdp_ckpt_pack(st["x"], st["ckpt"])
        F.fsdp_ckpt_unpack(st["ckpt"], st["y"])
        return {"back": st["y"]}
    if op == "norm_fwd":
        F.fsdp_norm_forward(st["x"], st["w"], st["b"], st["y"], st["mean_out"], st["rstd_out"],
                            kind=case["kind"], eps=EPS[case["kind"]], residual=st.get("r"), sum=st["sum"])
        return {k: v for k, v in (("y", st["y"]), ("sum", st["sum"]), ("mean", st["mean_out"]),
                                  ("rstd", st["rstd_out"])) if v is not None}
    if op == "norm_bwd":
        F.fsdp_norm_backward(st["dy"], st["x"], st["w"], st["mean"], st["rstd"], st["dx"], st["dw"], st["db"],
                             st["ws"], kind=case["kind"], dres=st.get("r"))
    elif op == "norm_step":
        F.fsdp_norm_forward(st["x"], st["w"], st["b"], st["y"], st["mean_out"], st["rstd_out"],
                            kind=case["kind"], eps=EPS[case["kind"]], ckpt=st["ckpt"])
        F.fsdp_norm_backward(st["dy"], st["ckpt"], st["w"], st["mean_out"], st["rstd_out"], st["dx"], st["dw"],
                             st["db"], st["ws"], kind=case["kind"], y=st["again"], bias=st["b"])
    else:
        F.fsdp_act_forward(st["x"], st["y"], kind=case["kind"], ckpt=st["ckpt"])
        F.fsdp_act_backward(st["dy"], st["ckpt"], st["dx"], st["db"], st["ws"], kind=case["kind"], y=st["again"])
    got = {"dx": st["dx"], "dw": st["dw"], "db": st["db"]}
    if op != "norm_bwd":
        got |= {"y": st["y"], "again": st["again"]}
    return {k: v for k, v in got.items() if v is not None}


# ---------------------------------------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------------------------------------

def _pow2(e):
    """2^e for whole e in -140..127, exactly: the exponent field of a binary64, then cast."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64).float()


def _held(x, fmt):
    """The values that an 8-bit checkpoint of x (fp32) stands for: groups of GROUP columns, each with the
    smallest power-of-two scale that keeps its largest element inside the codes' range."""
    R, C = x.shape
    n = -(-C // GROUP)
    x = torch.nn.functional.pad(x, (0, n * GROUP - C)).view(R, n, GROUP)
    amax = x.abs().amax(2, keepdim=True)
    _, e = torch.frexp(amax)                               # amax in [2^(e-1), 2^e)
    if fmt == "e4m3":
        s = (e - 9).clamp(-124, 120)                       # amax 2^-s in [256, 512)
        s = s + (amax * _pow2(-s) > 464)                   # above 464 it would round past 448
    else:
        s = (e - 7).clamp(-127, 121)                       # amax 2^-s in [64, 128)
        s = s + (amax * _pow2(-s) >= 127.5)                # from 127.5 on it would round past 127
    scale = _pow2(s)
    v = x * _pow2(-s)
    if fmt == "e4m3":
        _, ve = torch.frexp(v)
        step = _pow2((ve - 1).clamp(min=-6) - 3)           # 3 mantissa bits, subnormals below 2^-6
        v = torch.round(v / step) * step
    else:
        v = torch.round(v)
    v = torch.where(torch.isfinite(amax), v * scale, torch.nan)
    return v.view(R, n * GROUP)[:, :C]


def _stats(x, kind):
    m = x.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(x[:, :1])
    v = (x - m).square().mean(1, keepdim=True)
    return m, torch.rsqrt(v + EPS[kind])


def _act(h, kind):
    """f(h) and f'(h)"""
    if kind == "relu":
        return torch.clamp(h, min=0), (h > 0).to(h.dtype)
    if kind == "silu":
        s = torch.sigmoid(h)
        return h * s, s * (1 + h * (1 - s))
    if kind == "gelu":
        c = 0.5 * (1 + torch.erf(h * math.sqrt(0.5)))
        return h * c, c + h * torch.exp(-0.5 * h * h) * (1 / math.sqrt(2 * math.pi))
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (h + 0.044715 * h * h * h))
    return 0.5 * h * (1 + t), 0.5 * (1 + t) + 0.5 * h * (1 - t * t) * k * (1 + 3 * 0.044715 * h * h)


def _norm_grads(dy, x, w, m, rstd, kind, dres=None):
    xh = (x - m) * rstd
    g = dy * w
    dx = g - xh * (g * xh).mean(1, keepdim=True)
    if kind == "layer":
        dx = dx - g.mean(1, keepdim=True)
    dx = rstd * dx
    if dres is not None:
        dx = dx + dres
    return xh, dx, (dy * xh).sum(0), dy.sum(0)


def _run_plain(st):
    case = st["case"]
    op, t = case["op"], DTYPES[case["dtype"]]
    x = st["x"].float()
    if op == "ckpt":
        return {"back": _held(x, case["format"]).to(t)}
    if op == "act_step":
        y, _ = _act(x, case["kind"])
        again, d = _act(_held(x, case["format"]), case["kind"])
        dx = st["dy"].float() * d
        return {"y": y.to(t), "again": again.to(t), "dx": dx.to(t), "db": dx.sum(0)}
    kind = case["kind"]
    layer = kind == "layer"
    w = st["w"].float()
    b = st["b"].float() if layer else None
    if op == "norm_bwd":
        m = st["mean"][:, None] if layer else torch.zeros_like(st["rstd"][:, None])
        dres = st["r"].float() if case["residual"] else None
        _, dx, dw, db = _norm_grads(st["dy"].float(), x, w, m, st["rstd"][:, None], kind, dres)
        return {"dx": dx.to(t), "dw": dw, **({"db": db} if layer else {})}
    got = {}
    if case.get("residual"):
        got["sum"] = (x + st["r"].float()).to(t)
        x = got["sum"].float()
    m, rstd = _stats(x, kind)
    y = (x - m) * rstd * w
    y = (y + b if layer else y).to(t)
    if op == "norm_fwd":
        return {"y": y, "rstd": rstd[:, 0], **got, **({"mean": m[:, 0]} if layer else {})}
    xh, dx, dw, db = _norm_grads(st["dy"].float(), _held(x, case["format"]), w, m, rstd, kind)
    again = xh * w
    again = again + b if layer else again
    return {"y": y, "again": again.to(t), "dx": dx.to(t), "dw": dw, **({"db": db} if layer else {})}


# ---------------------------------------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------------------------------------

def _table(fmt):
    """Every value that a code can have, ascending: e4m3 has sign, 4 exponent bits (bias 7) and 3 mantissa
    bits, 448 the largest; the integers are -127..127."""
    if fmt == "int8":
        v = [float(i) for i in range(-127, 128)]
    else:
        pos = [m / 8 * 2.0 ** -6 for m in range(8)]
        pos += [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8) if not (e == 15 and m == 7)]
        v = [-p for p in reversed(pos[1:])] + pos
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _exact_held(x, fmt):
    """Each element's nearest code value (of two as near the even code) at the smallest scale 2^s, s >= low,
    at which no element of its group would need a value past the largest."""
    table = _table(fmt)
    top, low = (464.0, -124) if fmt == "e4m3" else (127.5, -127)
    powers = torch.tensor([2.0 ** k for k in range(-500, 500)], dtype=torch.float64, device="cuda")
    two = lambda k: powers[k.nan_to_num(0.0, 0.0, 0.0).long() + 500]  # noqa: E731
    zero = (table.numel() - 1) // 2
    out = torch.empty_like(x)
    for lo in range(0, x.shape[1], GROUP * 64):
        part = x[:, lo:lo + GROUP * 64]
        pad = -part.shape[1] % GROUP
        p = torch.cat([part, part.new_zeros(part.shape[0], pad)], 1).view(part.shape[0], -1, GROUP)
        big = p.abs().max(2, keepdim=True).values
        s = torch.ceil(torch.log2((big / top).clamp(min=2.0 ** -400)))
        # the logarithm is rounded: take s, or the power beside it, by the definition itself
        fits = (lambda k: big <= top * two(k)) if fmt == "e4m3" else (lambda k: big < top * two(k))
        s = torch.where(fits(s - 1), s - 1, torch.where(fits(s), s, s + 1)).clamp(min=low)
        v = (p / two(s)).contiguous()
        hi = torch.searchsorted(table, v).clamp(1, table.numel() - 1)
        below, above = table[hi - 1], table[hi]
        even_below = (hi - 1 - zero) % 2 == 0               # codes count up from zero on either side
        take = (v - below < above - v) | ((v - below == above - v) & even_below)
        q = torch.where(take, below, above) * two(s)
        q = torch.where((p.isfinite().all(2, keepdim=True)), q, torch.nan)
        out[:, lo:lo + GROUP * 64] = q.view(q.shape[0], -1)[:, :part.shape[1]]
    return out


def _exact_act(h, kind):
    if kind == "relu":
        return torch.where(h > 0, h, 0.0), torch.where(h > 0, 1.0, 0.0).double()
    if kind == "silu":
        e = torch.exp(-h)
        return h / (1 + e), (1 + e + h * e) / (1 + e) ** 2
    if kind == "gelu":
        phi = torch.special.ndtr(h)
        return h * phi, phi + h * torch.exp(-h * h / 2) / math.sqrt(2 * math.pi)
    a, c = math.sqrt(2 / math.pi), 0.044715
    u = a * (h + c * h ** 3)
    sig = torch.sigmoid(2 * u)                              # (1 + tanh u) / 2
    return h * sig, sig + h * 2 * sig * (1 - sig) * a * (1 + 3 * c * h ** 2)


def exact(case, seed):
    i = _inputs(case, seed)
    op, n = case["op"], case["cols"]
    x = i["x"].double()
    if op == "ckpt":
        return {"back": _exact_held(x, case["format"])}
    if op == "act_step":
        y, _ = _exact_act(x, case["kind"])
        again, slope = _exact_act(_exact_held(x, case["format"]), case["kind"])
        dx = i["dy"].double() * slope
        return {"y": y, "again": again, "dx": dx, "db": torch.einsum("rc->c", dx)}
    w = i["w"].double()
    b = 0.0 if i["b"] is None else i["b"].double()
    layer = case["kind"] == "layer"
    out = {}
    if op != "norm_bwd":
        if case.get("residual"):
            x = (x + i["r"].double()).to(DTYPES[case["dtype"]]).double()   # kept, and normalised, as rounded
            out["sum"] = x
        mean = torch.einsum("rc->r", x) / n if layer else x.new_zeros(x.shape[0])
        c = x - mean[:, None]
        rstd = 1 / torch.sqrt(torch.einsum("rc,rc->r", c, c) / n + EPS[case["kind"]])
        out["y"] = c * rstd[:, None] * w + b
        if op == "norm_fwd":
            out["rstd"] = rstd
            if layer:
                out["mean"] = mean
            return out
        c = _exact_held(x, case["format"]) - mean[:, None]
    else:
        rstd = i["rstd"].double()
        c = x - (i["mean"].double() if layer else x.new_zeros(x.shape[0]))[:, None]
    # y_j = w_j h_j + b_j with h = (x - mean) rstd: the gradient of x from those of h
    h = c * rstd[:, None]
    dy = i["dy"].double()
    dh = dy * w
    along = torch.einsum("rc,rc->r", dh, h) / n
    dx = dh - along[:, None] * h
    if layer:
        dx = dx - (torch.einsum("rc->r", dh) / n)[:, None]
    dx = dx * rstd[:, None]
    if case.get("residual"):
        dx = dx + i["r"].double()
    out |= {"dx": dx, "dw": torch.einsum("rc,rc->c", dy, h)}
    if layer:
        out["db"] = torch.einsum("rc->c", dy)
    if op == "norm_step":
        out["again"] = h * w + b
    return out


def work(case):
    """Bytes: every input read once, every output written once (a checkpoint is both: written by the forward
    pass, read by the backward pass).  Operations: adds, multiplies and one per function value."""
    R, C, op = case["rows"], case["cols"], case["op"]
    e = 2 if case["dtype"] == "bf16" else 4
    q = 1 + 1 / GROUP
    per, extra, flops = {
        "ckpt": (2 * e + 2 * q, 0, 4),
        "norm_fwd": (e * (4 if case.get("residual") else 2), 8 * R + 4 * C, 8),
        "norm_bwd": (e * (4 if case.get("residual") else 3), 8 * R + 10 * C, 16),
        "norm_step": (5 * e + 2 * q, 16 * R + 14 * C, 30),
        "act_step": (5 * e + 2 * q, 4 * C, 30),
    }[op]
    return {"bytes": int(per * R * C + extra), "flops": int(flops * R * C)}
