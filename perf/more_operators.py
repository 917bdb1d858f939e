"""More operators of a training step as measured work: rotary positions, token log probabilities with their
gradient, and AdamW over many tensors.

`run` computes them in their plain form from elementary torch operations, or, where `own` is true, through
sharded_fsdp_flatten_amd.  A case is one of:

  logprob_fwd   log probabilities of given tokens under a row of logits each, with the entropy and the top
                alternatives where asked for
  logprob_bwd   the gradient of the logits from those of the log probabilities (and of the entropies)
  logprob_step  both, as a loss takes them
  adam          one AdamW step over a list of tensors with fp32 or 8-bit states; 8-bit states come back as the
                values that they stand for (bf16 numbers), as a checkpoint saves them
  rotary_fwd    positions rotated into queries and keys
  rotary_bwd    the gradients of queries and keys
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
GROUP = 32                  # elements of an 8-bit state that share one scale
LR, BETA1, BETA2, EPS, STEP, SEED = 1e-3, 0.9, 0.999, 1e-8, 7, 20240607
WEIGHT_DECAY = (0.01, 0.0)  # matrices; norms and biases


def listed():
    return [
        # the last position of a few sequences, with its eight likeliest tokens: launch latency
        dict(name="logprob_fwd few tokens", op="logprob_fwd", rows=16, cols=50257, dtype="bf16", scale=1.0, top=8, entropy=False, ignored=0.0, masked=0),
        # four positions over a wide vocabulary whose tail is padding: rows long enough to be split
        dict(name="logprob_fwd wide", op="logprob_fwd", rows=4, cols=262144, dtype="bf16", scale=1.0, top=64, entropy=True, ignored=0.0, masked=1000),
        # scoring 2048 sampled tokens in fp32 at a temperature, with entropy and alternatives
        dict(name="logprob_fwd f32 top 20", op="logprob_fwd", rows=2048, cols=50257, dtype="f32", scale=1.25, top=20, entropy=True, ignored=0.0, masked=0),
        # the loss of a GPT-2 Large micro-batch of 4 x 1024 and its gradient, a tenth of the tokens padding
        dict(name="logprob_step GPT-2-L", op="logprob_step", rows=4096, cols=50257, dtype="bf16", scale=1.0, top=0, entropy=False, ignored=0.1, masked=0),
        # a ragged batch with an entropy bonus: gradients of both
        dict(name="logprob_bwd ragged", op="logprob_bwd", rows=777, cols=32003, dtype="bf16", scale=0.7, top=0, entropy=True, ignored=0.2, masked=61),
        # norms and biases of GPT-2 Large blocks, sharded in 8: many short tensors
        dict(name="adam short tensors", op="adam", unit="gpt", d=1280, shards=8, blocks=12, matrices=False, states="f32", grad="f32", copy=False, clip=False),
        # a rank's share of a GPT-175B block (128 ranks), with the bf16 copy that the next gather sends
        dict(name="adam 175B share", op="adam", unit="gpt", d=12288, shards=128, blocks=1, matrices=True, states="f32", grad="f32", copy=True, clip=False),
        # a rank's shares of twelve GPT-2 Large blocks (8 ranks) with 8-bit states and clipped bf16 gradients
        dict(name="adam GPT-2-L 8 bit", op="adam", unit="gpt", d=1280, shards=8, blocks=12, matrices=True, states="8bit", grad="bf16", copy=True, clip=True),
        # queries and keys of a few new tokens
        dict(name="rotary_fwd few tokens", op="rotary_fwd", batch=16, tokens=1, heads=20, kv_heads=20, dim=64, rot=64, dtype="bf16", layout="half", order="bthd", scaling="none", far=1024),
        # a GPT-175B attention's queries and keys over 4096 tokens at far positions of a stretched context
        dict(name="rotary_fwd 175B far", op="rotary_fwd", batch=2, tokens=2048, heads=96, kv_heads=96, dim=128, rot=128, dtype="bf16", layout="half", order="packed", scaling="parts", far=1048576),
        # the gradients of a GPT-2 Large micro-batch in the attention's own layout, a quarter of the key heads
        dict(name="rotary_bwd GPT-2-L", op="rotary_bwd", batch=4, tokens=1024, heads=20, kv_heads=5, dim=64, rot=64, dtype="bf16", layout="half", order="bhtd", scaling="none", far=1024),
        # half of every 80-wide head, neighbouring pairs, fp32, an odd number of tokens
        dict(name="rotary_fwd part f32", op="rotary_fwd", batch=1, tokens=4099, heads=13, kv_heads=13, dim=80, rot=40, dtype="f32", layout="interleaved", order="bthd", scaling="linear", far=32768),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprob_fwd", "logprob_fwd", "logprob_bwd", "logprob_step", "adam", "adam", "rotary_fwd", "rotary_bwd"])
    if op.startswith("logprob"):
        c = dict(op=op, cols=_log(rng, 100, 262144), dtype=rng.choice(["bf16", "bf16", "f32"]))
        if rng.random() < 0.3:
            c["cols"] = max(128, c["cols"] // 128 * 128)
        most = 96 * 1024 * 1024 // (2 if c["dtype"] == "f32" else 1)
        c["rows"] = _log(rng, 1, min(16384, max(1, most // c["cols"])))
        c["scale"] = rng.choice([1.0, 1.0, 0.5, 1.3])
        c["top"] = rng.choice([0, 1, 5, 20, 33, 64]) if op == "logprob_fwd" else 0
        c["entropy"] = rng.random() < 0.5
        c["ignored"] = rng.choice([0.0, 0.1, 0.5])
        c["masked"] = rng.choice([0, c["cols"] // 10])
        return c
    if op == "adam":
        c = dict(op=op, unit="drawn", tensors=_log(rng, 1, 200), largest=_log(rng, 40, 6000000), sizes=rng.randrange(1 << 30))
        return c | dict(states=rng.choice(["f32", "8bit"]), grad=rng.choice(["f32", "bf16"]), copy=rng.random() < 0.5, clip=rng.random() < 0.5)
    dim = rng.choice([32, 64, 80, 96, 128, 128, 256, rng.randrange(2, 130)])
    rot = rng.choice([dim // 2 * 2, dim // 4 * 2 or 2])
    heads = _log(rng, 1, 96)
    most = 64 * 1024 * 1024 // (heads * dim)
    batch = rng.choice([1, 1, 2, 3, 8])
    tokens = _log(rng, 1, max(1, min(16384, most) // batch))
    return dict(op=op, batch=batch, tokens=tokens, heads=heads, kv_heads=rng.choice([0, 1, heads, max(1, heads // 4)]), dim=dim, rot=rot,
                dtype=rng.choice(["bf16", "bf16", "f32"]), layout=rng.choice(["half", "interleaved"]), order=rng.choice(["bthd", "bhtd", "packed"]),
                scaling=rng.choice(["none", "linear", "ntk", "parts"]) if rot > 2 else "none", far=_log(rng, 1000, 1000000))


# ---------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------

def _sizes(case):
    """(elements, hyperparameter group) of each tensor of an AdamW case: a rank's share of a parameter is
    its rows divided among the ranks, rounded up."""
    if case["unit"] == "drawn":
        r = random.Random(case["sizes"])
        left, out = 24 * 1024 * 1024, []
        for _ in range(case["tensors"]):
            n = min(_log(r, 1, case["largest"]), left)
            left -= n
            out.append((n, r.randrange(2)))
        return [s for s in out if s[0]]
    d = case["d"]
    shapes = [(d,), (d,), (d,), (d,), (3 * d, d), (3 * d,), (d, d), (d,), (4 * d, d), (4 * d,), (d, 4 * d), (d,)]
    one = [(-(-s[0] // case["shards"]) * (s[1] if len(s) > 1 else 1), 0 if len(s) > 1 else 1) for s in shapes
           if case["matrices"] or len(s) == 1]
    return one * case["blocks"]


def _state_bytes(n):
    """An 8-bit state: n codes, filled up to a multiple of 16, then one scale for every 32 of them."""
    return -(-n // 16) * 16 + -(-n // GROUP)


_M_VALUES = [m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)][:127]  # e4m3
_V_VALUES = [m * 2.0 ** -17 if e == 0 else (8 + m) * 2.0 ** (e - 18) for e in range(31) for m in range(8)]       # e5m3


def _random_codes(x, values, top):
    """A state's codes and scales for the values x, each code just below its value."""
    n = x.numel()
    g = torch.nn.functional.pad(x.abs().double(), (0, -n % GROUP)).view(-1, GROUP)
    s = torch.ceil(torch.log2((g.amax(1) / top).clamp(min=2.0 ** -100)))
    table = torch.tensor(values, dtype=torch.float64, device="cuda")
    i = torch.searchsorted(table, (g / torch.exp2(s)[:, None]).view(-1)[:n], right=True) - 1
    codes = torch.where(x < 0, i + 128, i)
    return codes.to(torch.uint8), (s + 127).to(torch.uint8)


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    def uniform(*shape):
        return torch.rand(*shape, device="cuda", generator=gen)

    if op.startswith("logprob"):
        R, C, t = case["rows"], case["cols"], DTYPES[case["dtype"]]
        # a few tokens stand out, rows are more or less certain, the vocabulary's padded tail is masked
        x = normal(R, C) * (1.0 + 2.0 * uniform(R, 1)) + 2.0 * normal(C)
        if case["masked"]:
            x[:, C - case["masked"]:] = -math.inf
        tokens = torch.randint(0, C - case["masked"], (R,), device="cuda", generator=gen)
        tokens[uniform(R) < case["ignored"]] = -100
        inp = {"x": x.to(t), "tokens": tokens}
        if op != "logprob_fwd":
            inp["dl"] = (-1.0 / R) * (0.5 + uniform(R))
            if case["entropy"]:
                inp["dh"] = 0.01 / R * normal(R)
        if op == "logprob_bwd":
            z = inp["x"].double() * case["scale"]
            mx = z.amax(1)
            e = torch.exp(z - mx[:, None])
            inp["max"], inp["logsum"] = mx.float(), e.sum(1).log().float()
            inp["h"] = (e.sum(1).log() - (e * (z - mx[:, None]).clamp(min=-1e30)).sum(1) / e.sum(1)).float()
        return inp
    if op == "adam":
        sizes = _sizes(case)
        T = sum(n for n, _ in sizes)
        group = [g for _, g in sizes]
        offsets = [0]
        for n, _ in sizes:
            offsets.append(offsets[-1] + n)
        size = torch.exp(0.7 * normal(T))                   # elements' gradients differ in size
        g = 1e-3 * size * normal(T)
        m, v = 2e-4 * size * normal(T), (1e-3 * size) ** 2 * (0.2 + uniform(T))
        inp = {"sizes": sizes, "offsets": offsets, "group": group, "p": 0.02 * normal(T), "g": g.to(DTYPES[case["grad"]]),
               "clip": 0.5 + uniform(1) if case["clip"] else None}
        if case["states"] == "f32":
            return inp | {"m": m, "v": v}
        starts = [0]
        for n, _ in sizes:
            starts.append(starts[-1] + -(-_state_bytes(n) // 16) * 16)
        inp |= {"starts": starts}
        for name, x, values, top in (("m", m, _M_VALUES, 448.0), ("v", v, _V_VALUES, 61440.0)):
            buf = torch.zeros(starts[-1], dtype=torch.uint8, device="cuda")
            for i, (n, _) in enumerate(sizes):
                codes, scales = _random_codes(x[offsets[i]:offsets[i] + n], values, top)
                buf[starts[i]:starts[i] + n] = codes
                at = starts[i] + -(-n // 16) * 16
                buf[at:at + scales.numel()] = scales
            inp[name] = buf
        return inp
    B, T, H, K, D, t = case["batch"], case["tokens"], case["heads"], case["kv_heads"], case["dim"], DTYPES[case["dtype"]]

    def heads(n):
        if case["order"] == "bhtd":
            return normal(B, n, T, D).to(t).transpose(1, 2)
        return normal(B, T, n, D).to(t)

    if case["order"] == "packed":                           # one matrix product gave queries, keys and values
        qkv = normal(B, T, H + 2 * K, D).to(t)
        q, k = qkv[:, :, :H], qkv[:, :, H:H + K]
    else:
        q, k = heads(H), heads(K)
    first = torch.randint(0, max(1, case["far"] - T), (B, 1), device="cuda", generator=gen)
    return {"q": q, "k": k if K else None, "positions": first + torch.arange(T, device="cuda")}


def prepare(case, seed):
    st = dict(case=case, **_inputs(case, seed))
    op = case["op"]
    new = lambda *shape, dtype=torch.float32: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    if own:
        import sharded_fsdp_flatten_amd as F
        st["F"] = F
    if op.startswith("logprob"):
        R, C, k = case["rows"], case["cols"], case["top"]
        if op != "logprob_bwd":
            st |= {"logprob": new(R), "max": new(R), "logsum": new(R), "h": new(R) if case["entropy"] else None}
            st |= {"top_logprob": new(R, k) if k else None, "top_token": new(R, k, dtype=torch.int64) if k else None}
            if own:
                st["ws"] = new(F.fsdp_logprob_workspace(R, C, k))
        if op != "logprob_fwd":
            st["dx"] = new(R, C, dtype=DTYPES[case["dtype"]])
    elif op == "adam":
        T = st["offsets"][-1]
        if case["copy"]:
            st["pb"] = new(T, dtype=torch.bfloat16)
        if case["states"] == "8bit":
            st |= {"m16": new(T, dtype=torch.bfloat16), "v16": new(T, dtype=torch.bfloat16)}
        if own:
            cut = lambda b: [b[o:o + n] for (n, _), o in zip(st["sizes"], st["offsets"])]  # noqa: E731
            small = lambda b: [b[o:o + _state_bytes(n)] for (n, _), o in zip(st["sizes"], st["starts"])]  # noqa: E731
            of = cut if case["states"] == "f32" else small
            st["list"] = F.AdamTensors(cut(st["p"]), cut(st["g"]), of(st["m"]), of(st["v"]), states=case["states"], groups=st["group"],
                                       param_bf16=cut(st["pb"]) if case["copy"] else None)
            if case["states"] == "8bit":
                st["values"] = F.AdamTensors(None, None, cut(st["m16"]), cut(st["v16"]), states="bf16")
    else:
        st["freqs"] = torch.tensor(_freqs(case), dtype=torch.float64, device="cuda")
        st["q_out"] = torch.empty_like(st["q"])             # the input's layout, or its own rows where that is packed
        st["k_out"] = torch.empty_like(st["k"]) if case["kv_heads"] else None
        st["stretch"] = _stretch(case)
    return st


def run(st):
    op = st["case"]["op"]
    if op.startswith("logprob"):
        return (_own_logprob if own else _plain_logprob)(st)
    if op == "adam":
        return (_own_adam if own else _plain_adam)(st)
    return (_own_rotary if own else _plain_rotary)(st)


def _given(**outputs):
    return {k: v for k, v in outputs.items() if v is not None}


# ---------------------------------------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------------------------------------

def _own_logprob(st):
    F, case = st["F"], st["case"]
    got = {}
    if case["op"] != "logprob_bwd":
        F.fsdp_logprob_forward(st["x"], st["tokens"], st["logprob"], st["max"], st["logsum"], st["ws"], scale=case["scale"],
                               entropy=st["h"], top_logprob=st["top_logprob"], top_token=st["top_token"])
        got = _given(logprob=st["logprob"], max=st["max"], logsum=st["logsum"], entropy=st["h"], top_logprob=st["top_logprob"],
                     top_token=st["top_token"])
    if case["op"] != "logprob_fwd":
        F.fsdp_logprob_backward(st["x"], st["tokens"], st["dl"], st["max"], st["logsum"], st["dx"], scale=case["scale"],
                                dentropy=st.get("dh"), entropy=st.get("h"))
        got["dx"] = st["dx"]
    return got


def _own_adam(st):
    F, case = st["F"], st["case"]
    groups = [dict(lr=LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=w, step=STEP) for w in WEIGHT_DECAY]
    F.fsdp_adam_tensors(st["list"], groups, grad_scale=st["clip"], seed=SEED)
    if case["states"] == "f32":
        return _given(p=st["p"], m=st["m"], v=st["v"], copy=st.get("pb"))
    F.fsdp_adam_convert(st["list"], st["values"])
    return _given(p=st["p"], m=st["m16"], v=st["v16"], copy=st.get("pb"))


def _own_rotary(st):
    F, case = st["F"], st["case"]
    f = F.fsdp_rotary_forward if case["op"] == "rotary_fwd" else F.fsdp_rotary_backward
    f(st["q"], st["q_out"], st["freqs"], k=st["k"], k_out=st["k_out"], positions=st["positions"], layout=case["layout"],
      scale=st["stretch"])
    return _given(q=st["q_out"], k=st["k_out"])


# ---------------------------------------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------------------------------------

def _plain_logprob(st):
    case, x = st["case"], st["x"]
    t = DTYPES[case["dtype"]]
    z = x.float() * case["scale"]
    tok = st["tokens"]
    valid = (tok >= 0) & (tok < case["cols"])
    at = torch.where(valid, tok, 0)[:, None]
    got = {}
    if case["op"] != "logprob_bwd":
        mx = z.amax(1, keepdim=True)
        d = z - mx
        e = torch.exp(d)
        s = e.sum(1, keepdim=True)
        logsum = torch.log(s)
        lp = torch.where(valid, (d.gather(1, at) - logsum)[:, 0], 0.0)
        h = None
        if case["entropy"]:
            h = (logsum - torch.where(e > 0, e * d, 0.0).sum(1, keepdim=True) / s)[:, 0]
        got = _given(logprob=lp, max=mx[:, 0], logsum=logsum[:, 0], entropy=h)
        if case["top"]:
            left, col = x.float(), torch.arange(case["cols"], device="cuda")
            toks = []
            for _ in range(case["top"]):                    # the largest left, the first of equal ones
                best = left.amax(1, keepdim=True)
                i = torch.where(left == best, col, case["cols"]).amin(1, keepdim=True)
                toks.append(i)
                left = torch.where(col == i, -math.inf, left)
            got["top_token"] = torch.cat(toks, 1)
            got["top_logprob"] = d.gather(1, got["top_token"]) - logsum
    else:
        mx, logsum, h = st["max"][:, None], st["logsum"][:, None], st.get("h")
    if case["op"] != "logprob_fwd":
        lp = z - mx - logsum
        p = torch.exp(lp)
        dl = torch.where(valid, st["dl"], 0.0)[:, None]
        dz = -dl * p
        dz.scatter_add_(1, at, dl)
        if case["entropy"]:
            dz = dz - torch.where(p > 0, st["dh"][:, None] * p * (lp + h[:, None]), 0.0)
        got["dx"] = (dz * case["scale"]).to(t)
    return got


def _u16(n, tensor):
    """The two 16-bit random numbers of every element of a tensor in the list: a 64-bit key of the seed, the
    step and the tensor's number, and a 32-bit hash of the key and the element's number."""
    key = _mix64(_mix64(SEED + 0x9E3779B97F4A7C15 * STEP) + 0x9E3779B97F4A7C15 * (tensor + 1)) & 0xFFFFFFFF
    low = 0xFFFFFFFF
    x = (torch.arange(n, device="cuda") * 0x9E3779B1 + key) & low
    x = x ^ (x >> 15)
    x = (x * 0xB504F333) & low
    x = x ^ (x >> 13)
    x = (x * 0xDDB3D743) & low
    x = x ^ (x >> 16)
    return x >> 16, x & 0xFFFF


def _mix64(k):
    low = (1 << 64) - 1
    k &= low
    k = ((k ^ (k >> 30)) * 0xBF58476D1CE4E5B9) & low
    k = ((k ^ (k >> 27)) * 0x94D049BB133111EB) & low
    return k ^ (k >> 31)


def _pow2(e):
    """2^e for whole e in -149..127, exactly."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64).float()


def _exponent(x):
    """floor(log2 x) of positive x."""
    return torch.frexp(x)[1] - 1


def _encode(x, r, emin, top, low):
    """x rounded at random to codes times its group's scale, as codes (without sign), signs and scale bytes: the
    scale is the smallest power of two, 2^low at least, at which the group's largest magnitude does not pass `top`;
    steps are an eighth of the power of two below a value, 2^(emin - 3) at least."""
    n = x.numel()
    pad = -n % GROUP
    amax = torch.nn.functional.pad(x.abs(), (0, pad)).view(-1, GROUP).amax(1)
    e = _exponent(torch.where(amax > 0, amax, 1.0))
    s = e - int(math.log2(top))
    s = s + (amax > top * _pow2(s).double()).to(s.dtype)
    s = torch.where(amax > 0, s, low).clamp(min=low)
    y = x.abs() * _pow2(-s).repeat_interleave(GROUP)[:n]
    q = _exponent(torch.where(y > 0, y, 2.0 ** -40)).clamp(min=emin)
    k = torch.floor(y * _pow2(3 - q) + r.float() * 2.0 ** -16)
    q, k = torch.where(k == 16, q + 1, q), torch.where(k == 16, 8.0, k)
    code = torch.where(k < 8, k, (q - emin + 1) * 8 + k - 8)
    return code.to(torch.uint8), (s + 127).to(torch.uint8)


def _plain_adam(st):
    case = st["case"]
    step_size, bc2 = LR / (1 - BETA1 ** STEP), math.sqrt(1 - BETA2 ** STEP)
    small = case["states"] == "8bit"
    mvals = torch.tensor(_M_VALUES + [math.nan] + [-x for x in _M_VALUES] + [math.nan], device="cuda") if small else None
    vvals = torch.tensor(_V_VALUES + [math.nan] * 8, device="cuda") if small else None

    for i, (n, group) in enumerate(st["sizes"]):
        o = st["offsets"][i]
        p, g = st["p"][o:o + n], st["g"][o:o + n].float()
        if case["clip"]:
            g = g * st["clip"]
        if small:
            a = st["starts"][i]
            b, c = a + -(-n // 16) * 16, a + _state_bytes(n)

            def held(buf, values):
                scale = _pow2(buf[b:c].to(torch.int64) - 127).repeat_interleave(GROUP)[:n]
                return values[buf[a:a + n].to(torch.int64)] * scale

            m, v = held(st["m"], mvals), held(st["v"], vvals)
        else:
            m, v = st["m"][o:o + n], st["v"][o:o + n]
        m = m * BETA1 + g * (1 - BETA1)
        v = v * BETA2 + (g * g) * (1 - BETA2)
        den = torch.sqrt(v) / bc2 + EPS
        p.copy_(p * (1 - LR * WEIGHT_DECAY[group]) - (m / den) * step_size)
        if case["copy"]:
            st["pb"][o:o + n] = p.to(torch.bfloat16)
        if small:
            rm, rv = _u16(n, i)
            for buf, x, r, args, values, out in ((st["m"], m, rm, (-6, 448.0, -124), mvals, st["m16"]),
                                                 (st["v"], v, rv, (-14, 61440.0, -116), vvals, st["v16"])):
                code, byte = _encode(x, r, *args)
                buf[a:a + n] = torch.where(x < 0, code + 128, code)
                buf[b:c] = byte
                out[o:o + n] = held(buf, values)
        else:
            st["m"][o:o + n] = m
            st["v"][o:o + n] = v
    if small:
        return _given(p=st["p"], m=st["m16"], v=st["v16"], copy=st.get("pb"))
    return _given(p=st["p"], m=st["m"], v=st["v"], copy=st.get("pb"))


FACTOR, TRAINED, FEW, MANY = 8.0, 4096, 1.0, 32.0    # a context stretched by 8 from 4096 positions


def _freqs(case):
    """Angle a position of every pair."""
    rot, base = case["rot"], 10000.0
    if case["scaling"] == "ntk":
        base *= FACTOR ** (rot / (rot - 2))
    f = [base ** (-2 * i / rot) for i in range(rot // 2)]
    if case["scaling"] == "linear":
        f = [x / FACTOR for x in f]
    if case["scaling"] == "parts":
        # pairs that turn often over the trained context keep their angle, those that turn seldom are stretched
        keep = [min(1.0, max(0.0, (TRAINED * x / (2 * math.pi) - FEW) / (MANY - FEW))) for x in f]
        f = [x * k + x / FACTOR * (1 - k) for x, k in zip(f, keep)]
    return f


def _stretch(case):
    return 0.1 * math.log(FACTOR) + 1 if case["scaling"] == "parts" else 1.0


def _plain_rotary(st):
    case = st["case"]
    angle = st["positions"].double()[:, :, None, None] * st["freqs"]
    c, s = (torch.cos(angle) * st["stretch"]).float(), (torch.sin(angle) * st["stretch"]).float()
    if case["op"] == "rotary_bwd":
        s = -s
    half, rot = case["rot"] // 2, case["rot"]
    for x, out in ((st["q"], st["q_out"]), (st["k"], st["k_out"])):
        if x is None:
            continue
        a, b = (slice(0, half), slice(half, rot)) if case["layout"] == "half" else (slice(0, rot, 2), slice(1, rot, 2))
        xa, xb = x[..., a].float(), x[..., b].float()
        out[..., a] = (xa * c - xb * s).to(out.dtype)
        out[..., b] = (xa * s + xb * c).to(out.dtype)
        out[..., rot:] = x[..., rot:]
    return _given(q=st["q_out"], k=st["k_out"])


# ---------------------------------------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------------------------------------

def exact(case, seed):
    i = _inputs(case, seed)
    if case["op"].startswith("logprob"):
        return _exact_logprob(case, i)
    return _exact_adam(case, i) if case["op"] == "adam" else _exact_rotary(case, i)


def _exact_logprob(case, i):
    R, C = case["rows"], case["cols"]
    parts = []
    step = max(1, (1 << 27) // C)
    for lo in range(0, R, step):                            # row by row in chunks: 64 bits are wide
        z = i["x"][lo:lo + step].double() * case["scale"]
        tok = i["tokens"][lo:lo + step]
        has = (tok >= 0) & (tok < C)
        hot = torch.zeros_like(z)
        hot[has.nonzero()[:, 0], tok[has]] = 1.0
        out = {}
        lse = torch.logsumexp(z, 1, keepdim=True)
        logp = z - lse
        p = logp.exp()
        plogp = torch.where(p > 0, p * logp, 0.0)
        H = -plogp.sum(1, keepdim=True)
        if case["op"] != "logprob_bwd":
            top = z.max(1).values
            out |= {"logprob": torch.where(hot > 0, logp, 0.0).sum(1), "max": top, "logsum": lse[:, 0] - top}
            if case["entropy"]:
                out["entropy"] = H[:, 0]
            if case["top"]:
                order = torch.sort(i["x"][lo:lo + step].double(), dim=1, descending=True, stable=True).indices[:, :case["top"]]
                out |= {"top_token": order, "top_logprob": torch.gather(logp, 1, order)}
        if case["op"] != "logprob_fwd":
            dl = i["dl"][lo:lo + step].double()[:, None] * has[:, None]
            dz = dl * (hot - p)
            if case["entropy"]:
                dz = dz - i["dh"][lo:lo + step].double()[:, None] * (plogp + p * H)
            out["dx"] = (dz * case["scale"]).float() if R * C > 1 << 27 else dz * case["scale"]
        parts.append(out)
    return {k: torch.cat([q[k] for q in parts]) for k in parts[0]}


def _exact_state(codes, scales, fmt):
    """What an 8-bit state stands for: sign, exponent and fraction taken apart."""
    c = codes.long()
    if fmt == "m":
        sign, e, f = 1.0 - 2.0 * (c // 128), c % 128 // 8, c % 8
        v = sign * torch.where(e == 0, f / 512.0, (1 + f / 8.0) * torch.pow(2.0, e.double() - 7))
    else:
        e, f = c // 8, c % 8
        v = torch.where(e == 0, f / 131072.0, (1 + f / 8.0) * torch.pow(2.0, e.double() - 15))
    n = v.numel()
    return v.double() * torch.pow(2.0, scales.double() - 127).repeat_interleave(GROUP)[:n]


def _exact_rounded(x, u, values, low):
    """Each magnitude between two neighbours of `values` times the scale goes to the upper one where u reaches
    the part of the way that it lacks."""
    table = torch.tensor(values, dtype=torch.float64, device="cuda")
    n = x.numel()
    g = torch.cat([x.abs(), x.new_zeros(-n % GROUP)]).view(-1, GROUP)
    big = g.max(1, keepdim=True).values
    s = torch.full_like(big, low)
    for k in range(low, 120):
        s = torch.where(big > values[-1] * 2.0 ** k, k + 1.0, s)
    y = (g / torch.pow(2.0, s)).view(-1)[:n]
    hi = torch.searchsorted(table, y, right=True).clamp(max=len(values) - 1)
    a, b = table[hi - 1], table[hi]
    got = torch.where((y - a) / (b - a) + u >= 1, b, a)
    return torch.sign(x) * got * torch.pow(2.0, s).expand(-1, GROUP).reshape(-1)[:n]


def _exact_adam(case, i):
    out = {k: [] for k in ("p", "m", "v")}
    clip = i["clip"].double() if case["clip"] else 1.0
    small = case["states"] == "8bit"
    for j, (n, group) in enumerate(i["sizes"]):
        at = slice(i["offsets"][j], i["offsets"][j] + n)
        g = i["g"][at].double() * clip
        if small:
            a = i["starts"][j]
            b = a + -(-n // 16) * 16
            m, v = (_exact_state(i[k][a:a + n], i[k][b:b + -(-n // GROUP)], k) for k in ("m", "v"))
        else:
            m, v = i["m"][at].double(), i["v"][at].double()
        m = m + (1 - BETA1) * (g - m)
        v = v + (1 - BETA2) * (g * g - v)
        mhat, vhat = m / (1 - BETA1 ** STEP), v / (1 - BETA2 ** STEP)
        p = i["p"][at].double()
        out["p"].append(p - LR * WEIGHT_DECAY[group] * p - LR * mhat / (vhat.sqrt() + EPS))
        if small:
            um, uv = (r.double() / 65536 for r in _u16(n, j))
            m, v = _exact_rounded(m, um, _M_VALUES, -124), _exact_rounded(v, uv, _V_VALUES, -116)
        out["m"].append(m)
        out["v"].append(v)
    got = {k: torch.cat(x) for k, x in out.items()}
    return got | {"copy": got["p"]} if case["copy"] else got


def _exact_rotary(case, i):
    turn = i["positions"].double().unsqueeze(-1) * torch.tensor(_freqs(case), dtype=torch.float64, device="cuda")
    turn = turn if case["op"] == "rotary_fwd" else -turn
    w = torch.polar(torch.full_like(turn, _stretch(case)), turn).unsqueeze(2)
    out, n = {}, case["rot"] // 2
    for name in ("q", "k"):
        if i[name] is None:
            continue
        x = i[name].double()
        r = x[..., :2 * n]
        z = torch.complex(r[..., :n], r[..., n:]) if case["layout"] == "half" else torch.view_as_complex(r.reshape(*r.shape[:-1], n, 2).contiguous())
        z = z * w
        r = torch.cat([z.real, z.imag], -1) if case["layout"] == "half" else torch.view_as_real(z).reshape(r.shape)
        out[name] = torch.cat([r, x[..., 2 * n:]], -1)
    return out


def work(case):
    """Bytes: every input read once, every output written once.  Operations: adds, multiplies and one per
    function value."""
    op = case["op"]
    if op.startswith("logprob"):
        R, C, e = case["rows"], case["cols"], 2 if case["dtype"] == "bf16" else 4
        passes = {"logprob_fwd": 1, "logprob_bwd": 2, "logprob_step": 3}[op]
        flops = {"logprob_fwd": 5, "logprob_bwd": 5, "logprob_step": 10}[op] + (3 if case["entropy"] else 0)
        return {"bytes": passes * e * R * C + R * (32 + 12 * case["top"]), "flops": flops * R * C}
    if op == "adam":
        T = sum(n for n, _ in _sizes(case))
        # parameter and states both ways, the gradient, the copy; 8-bit states are also read and written out in bf16
        per = 8 + (4 if case["grad"] == "f32" else 2) + (2 if case["copy"] else 0) + (16 if case["states"] == "f32" else 6 * 33 / 32 + 4)
        return {"bytes": int(per * T), "flops": (16 if case["states"] == "f32" else 36) * T}
    e = 2 if case["dtype"] == "bf16" else 4
    n = case["batch"] * case["tokens"]
    values = n * (case["heads"] + case["kv_heads"]) * case["dim"]
    return {"bytes": 2 * e * values + 8 * n + 4 * case["rot"], "flops": 3 * values + 2 * n * case["rot"]}
