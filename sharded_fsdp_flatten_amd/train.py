"""ctypes binding of a training step's other operators, with the C ABI's names: rotary positions, token log
probabilities and their gradient, AdamW over many tensors.

Argument marshalling only, as in ``binding`` and ``layer``: dtypes, sizes and strides are read off the
tensors, the stream defaults to torch's current one on their GPU.

>>> freqs = fsdp_rotary_freqs(128).cuda()
>>> fsdp_rotary_forward(q, q, freqs, k=k, k_out=k)                 # q, k: [batch, tokens, heads, 128], in place
>>> ws = torch.empty(fsdp_logprob_workspace(tokens, vocab, 0), device="cuda")
>>> fsdp_logprob_forward(logits, labels, logprob, mx, logsum, ws)
>>> fsdp_logprob_backward(logits, labels, dlogprob, mx, logsum, logits)    # the gradient in the logits' place
>>> shards = AdamTensors(params, grads, exp_avgs, exp_avg_sqs, states="8bit")
>>> fsdp_adam_tensors(shards, dict(lr=1e-4, weight_decay=0.1, step=step), seed=17)
"""
from __future__ import annotations

import ctypes
import struct

from . import binding as B
from . import layer as L

FSDP_ROTARY_HALF = 1
FSDP_ROTARY_INTERLEAVED = 2
FSDP_ROTARY_NONE = 0
FSDP_ROTARY_LINEAR = 1
FSDP_ROTARY_NTK = 2
FSDP_ROTARY_PARTS = 3
FSDP_LOGPROB_MAX_TOP = 64
FSDP_STATE_F32 = 1
FSDP_STATE_8BIT = 2
FSDP_STATE_BF16 = 3
FSDP_ADAM_MAX_GROUPS = 16

_LAYOUTS = {"half": FSDP_ROTARY_HALF, "interleaved": FSDP_ROTARY_INTERLEAVED}
_SCALINGS = {"none": FSDP_ROTARY_NONE, "linear": FSDP_ROTARY_LINEAR, "ntk": FSDP_ROTARY_NTK,
             "parts": FSDP_ROTARY_PARTS}
_STATES = {"f32": FSDP_STATE_F32, "8bit": FSDP_STATE_8BIT, "bf16": FSDP_STATE_BF16}


class fsdp_heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch_pitch", ctypes.c_int64),
                ("token_pitch", ctypes.c_int64), ("head_pitch", ctypes.c_int64)]


class fsdp_rotary_cfg(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("tokens", ctypes.c_int64), ("heads", ctypes.c_int64),
                ("kv_heads", ctypes.c_int64), ("head_dim", ctypes.c_int64), ("rot", ctypes.c_int64),
                ("start", ctypes.c_int64), ("dtype", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("scale", ctypes.c_float), ("reserved", ctypes.c_int32)]


class fsdp_rotary_io(ctypes.Structure):
    _fields_ = [("q", fsdp_heads), ("q_out", fsdp_heads), ("k", fsdp_heads), ("k_out", fsdp_heads),
                ("positions", ctypes.c_void_p), ("freqs", ctypes.c_void_p)]


class fsdp_logprob_cfg(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("top", ctypes.c_int32), ("scale", ctypes.c_float), ("reserved", ctypes.c_int32)]


class fsdp_logprob_fwd(ctypes.Structure):
    _fields_ = [("logits", L.fsdp_rows), ("tokens", ctypes.c_void_p), ("logprob", ctypes.c_void_p),
                ("max", ctypes.c_void_p), ("logsum", ctypes.c_void_p), ("entropy", ctypes.c_void_p),
                ("top_logprob", ctypes.c_void_p), ("top_token", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("workspace_len", ctypes.c_int64)]


class fsdp_logprob_bwd(ctypes.Structure):
    _fields_ = [("logits", L.fsdp_rows), ("dlogits", L.fsdp_rows), ("tokens", ctypes.c_void_p),
                ("dlogprob", ctypes.c_void_p), ("dentropy", ctypes.c_void_p),
                ("max", ctypes.c_void_p), ("logsum", ctypes.c_void_p), ("entropy", ctypes.c_void_p)]


class fsdp_adam_tensor(ctypes.Structure):
    _fields_ = [("numel", ctypes.c_int64), ("param", ctypes.c_void_p), ("grad", ctypes.c_void_p),
                ("exp_avg", ctypes.c_void_p), ("exp_avg_sq", ctypes.c_void_p),
                ("param_bf16", ctypes.c_void_p), ("group", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class fsdp_adam_list(ctypes.Structure):
    _fields_ = [("n_tensors", ctypes.c_int32), ("n_groups", ctypes.c_int32),
                ("state_format", ctypes.c_int32), ("grad_dtype", ctypes.c_int32),
                ("seed", ctypes.c_uint64), ("grad_scale", ctypes.c_void_p),
                ("skip", ctypes.c_void_p)]


# The same structures packed in one call each: filling ctypes fields one by one costs more than a short
# launch.
_ROTARY_CFG = struct.Struct("@qqqqqqqiifi")
_ROTARY_IO = struct.Struct("@" + "Pqqq" * 4 + "PP")
_LOGPROB_CFG = struct.Struct("@qqiifi")
_LOGPROB_FWD = struct.Struct("@PqPPPPPPPPq")
_LOGPROB_BWD = struct.Struct("@PqPqPPPPPP")
_ADAM_LIST = struct.Struct("@iiiiQPP")
_ADAM_CFG = struct.Struct("@dddddq")
_NO_HEADS = (0, 0, 0, 0)

_fn = None
_i64 = None
_f64 = None


def _lib():
    """The library, with the argument types of this module's calls set once."""
    global _fn, _i64, _f64
    if _fn is None:
        import torch
        lib = L._lib()
        io, vp = ctypes.c_char_p, ctypes.c_void_p
        i64, i32, f64 = ctypes.c_int64, ctypes.c_int32, ctypes.c_double
        lib.fsdp_rotary_freqs.argtypes = [i64, f64, i32, f64, i64, f64, f64, vp]
        lib.fsdp_logprob_workspace.argtypes = [i64, i64, i32, ctypes.POINTER(i64)]
        lib.fsdp_adam_state_bytes.argtypes = [i64, ctypes.POINTER(i64)]
        for f in (lib.fsdp_rotary_forward, lib.fsdp_rotary_backward, lib.fsdp_logprob_forward,
                  lib.fsdp_logprob_backward):
            f.argtypes = [io, io, vp]
        lib.fsdp_adam_tensors.argtypes = [io, vp, io, vp]
        lib.fsdp_adam_convert.argtypes = [i32, vp, i32, vp, i32, ctypes.c_uint64, i64, vp]
        for f in (lib.fsdp_rotary_freqs, lib.fsdp_rotary_forward, lib.fsdp_rotary_backward,
                  lib.fsdp_logprob_workspace, lib.fsdp_logprob_forward, lib.fsdp_logprob_backward,
                  lib.fsdp_adam_state_bytes, lib.fsdp_adam_tensors, lib.fsdp_adam_convert):
            f.restype = i32
        _i64, _f64 = torch.int64, torch.float64
        _fn = lib
    return _fn


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------

def fsdp_rotary_freqs(rot: int, base: float = 10000.0, *, scaling: str = "none", factor: float = 1.0,
                      trained_len: int = 0, low: float = 1.0, high: float = 32.0):
    """Frequencies (radians a position) of rot / 2 pairs, a float64 tensor on the CPU; `scaling` one of
    "none", "linear", "ntk", "parts" (which reads trained_len, low and high)."""
    import torch
    out = torch.empty(max(0, rot // 2), dtype=torch.float64)
    B._check(_lib().fsdp_rotary_freqs(rot, base, L._kind(scaling, _SCALINGS, "scaling"), factor,
                                      trained_len, low, high, out.data_ptr() or 8))
    return out


def _heads(t, name: str, shape, dtype, device: int):
    """(address, batch, token and head pitch) of a tensor of heads of this shape."""
    if not isinstance(t, L._Tensor) or t.get_device() != device:
        L._refuse(t, name, device)
    if t.dtype is not dtype:
        raise TypeError("%s is %s, the others are %s" % (name, t.dtype, dtype))
    if t.shape != shape:
        raise ValueError("%s has shape %s, %s is needed" % (name, tuple(t.shape), tuple(shape)))
    if len(shape) == 4:
        b, n, h, e = t.stride()
    else:
        b, (n, h, e) = 0, t.stride()
    if e != 1 and shape[-1] > 1:
        raise ValueError("the elements of a head of %s must be next to each other, got stride %d" % (name, e))
    return t.data_ptr(), b, n, h


def _rotary(fn, q, q_out, freqs, k, k_out, positions, start, layout, scale, stream):
    if not isinstance(q, L._Tensor):
        L._refuse(q, "q", 0)
    code = L._dtype_code(q, "q")
    if not q.is_cuda:
        L._refuse(q, "q", 0)
    shape, t, dev = q.shape, q.dtype, q.get_device()
    if len(shape) == 4:
        batch, tokens, heads, dim = shape
    elif len(shape) == 3:
        batch, (tokens, heads, dim) = 1, shape
    else:
        raise ValueError("q must be [batch, tokens, heads, head_dim] or [tokens, heads, head_dim]")
    if k is None:
        if k_out is not None:
            raise TypeError("k and k_out must be given together")
        kv, kin, kout = 0, _NO_HEADS, _NO_HEADS
    else:
        if k_out is None:
            raise TypeError("k and k_out must be given together")
        kshape = getattr(k, "shape", ())
        if len(kshape) != len(shape) or kshape[:-2] != shape[:-2] or kshape[-1] != dim:
            raise ValueError("k must have the shape of q but for the number of heads, got %s" % (tuple(kshape),))
        kv = kshape[-2]
        kin = _heads(k, "k", kshape, t, dev)
        kout = _heads(k_out, "k_out", kshape, t, dev)
    if not isinstance(freqs, L._Tensor):
        raise TypeError("freqs must be a tensor, got %r" % type(freqs))
    pairs = freqs.numel()
    cfg = _ROTARY_CFG.pack(batch, tokens, heads, kv, dim, 2 * pairs, start, code,
                           L._kind(layout, _LAYOUTS, "layout"), scale, 0)
    io = _ROTARY_IO.pack(*_heads(q, "q", shape, t, dev), *_heads(q_out, "q_out", shape, t, dev), *kin, *kout,
                         0 if positions is None else L._vector(positions, "positions", batch * tokens, dev, _i64),
                         L._vector(freqs, "freqs", pairs, dev, _f64))
    L._call(fn, dev, stream, cfg, io)


def fsdp_rotary_forward(q, q_out, freqs, *, k=None, k_out=None, positions=None, start: int = 0,
                        layout: str = "half", scale: float = 1.0, stream=None) -> None:
    """Rotate the first 2 len(freqs) elements of every head of q, and of k where given, by their positions.
    Heads are [batch, tokens, heads, head_dim] or [tokens, heads, head_dim], of any strides but the last;
    the outputs may be the inputs.  positions: int64, one a token (else start + the token's number)."""
    _rotary((_fn or _lib()).fsdp_rotary_forward, q, q_out, freqs, k, k_out, positions, start, layout, scale, stream)


def fsdp_rotary_backward(dq, dq_out, freqs, *, k=None, k_out=None, positions=None, start: int = 0,
                         layout: str = "half", scale: float = 1.0, stream=None) -> None:
    """Gradients of fsdp_rotary_forward's inputs from those of its outputs, with the same arguments."""
    _rotary((_fn or _lib()).fsdp_rotary_backward, dq, dq_out, freqs, k, k_out, positions, start, layout, scale,
            stream)


# ---------------------------------------------------------------------------
# log probabilities
# ---------------------------------------------------------------------------

def fsdp_logprob_workspace(rows: int, cols: int, top: int = 0) -> int:
    """fp32 elements of workspace fsdp_logprob_forward needs (0 where no row is split)."""
    n = ctypes.c_int64()
    B._check(_lib().fsdp_logprob_workspace(rows, cols, top, ctypes.byref(n)))
    return int(n.value)


def fsdp_logprob_forward(logits, tokens, logprob, max, logsum, workspace=None, *, scale: float = 1.0,
                         entropy=None, top_logprob=None, top_token=None, stream=None) -> None:
    """Log probabilities of `tokens` (int64; outside the vocabulary: none, 0) under rows of logits, with the
    maximum and logarithm of the sum that the backward pass takes; the entropy and the alternatives
    (top_logprob, top_token: [rows, top]) where given.  tokens and logprob may be None."""
    rows, cols, t, code, dev = L._first(logits, "logits")
    fn = _lib()
    top, tl, tt = 0, 0, 0
    if top_logprob is not None or top_token is not None:
        for x, name in ((top_logprob, "top_logprob"), (top_token, "top_token")):
            if not isinstance(x, L._Tensor):
                raise TypeError("%s must be a tensor, got %r" % (name, type(x)))
        if not top_token.dim():
            raise ValueError("top_token must have at least one dimension")
        top = top_token.shape[-1]
        tl = L._vector(top_logprob, "top_logprob", rows * top, dev, L._f32)
        tt = L._vector(top_token, "top_token", rows * top, dev, _i64)
    f32 = L._f32
    cfg = _LOGPROB_CFG.pack(rows, cols, code, top, scale, 0)
    io = _LOGPROB_FWD.pack(
        *L._rows(logits, "logits", rows, cols, t, dev), L._vector(tokens, "tokens", rows, dev, _i64),
        L._vector(logprob, "logprob", rows, dev, f32), L._vector(max, "max", rows, dev, f32),
        L._vector(logsum, "logsum", rows, dev, f32), L._vector(entropy, "entropy", rows, dev, f32),
        tl, tt, *L._workspace(workspace, dev))
    L._call(fn.fsdp_logprob_forward, dev, stream, cfg, io)


def fsdp_logprob_backward(logits, tokens, dlogprob, max, logsum, dlogits, *, scale: float = 1.0,
                          dentropy=None, entropy=None, stream=None) -> None:
    """Gradient of the logits from those of the log probabilities and, with `entropy` as the forward pass
    wrote it, of the entropies (either may be None); dlogits may be the logits themselves."""
    rows, cols, t, code, dev = L._first(logits, "logits")
    fn = _lib()
    f32 = L._f32
    cfg = _LOGPROB_CFG.pack(rows, cols, code, 0, scale, 0)
    io = _LOGPROB_BWD.pack(
        *L._rows(logits, "logits", rows, cols, t, dev), *L._rows(dlogits, "dlogits", rows, cols, t, dev),
        L._vector(tokens, "tokens", rows, dev, _i64), L._vector(dlogprob, "dlogprob", rows, dev, f32),
        L._vector(dentropy, "dentropy", rows, dev, f32), L._vector(max, "max", rows, dev, f32),
        L._vector(logsum, "logsum", rows, dev, f32), L._vector(entropy, "entropy", rows, dev, f32))
    L._call(fn.fsdp_logprob_backward, dev, stream, cfg, io)


# ---------------------------------------------------------------------------
# AdamW over many tensors
# ---------------------------------------------------------------------------

def fsdp_adam_state_bytes(numel: int) -> int:
    """Bytes (uint8 elements) of the 8-bit state of numel elements; zeros are a state of zeros."""
    n = ctypes.c_int64()
    B._check(_lib().fsdp_adam_state_bytes(numel, ctypes.byref(n)))
    return int(n.value)


class _Held:
    """The storages of lists of tensors (a dict by the lists' names, entries may be None): kept from being freed, and
    checked to be the same memory as now.  `upto[name]`: how many storages the lists up to this one lie in."""

    def __init__(self, lists):
        storages, self.upto = {}, {}
        for name, tensors in lists.items():
            for i, t in enumerate(tensors):
                if t is not None:
                    s = t.untyped_storage()
                    k = s._cdata
                    if k not in storages:
                        storages[k] = name, i, s
            self.upto[name] = len(storages)
        self.names = [x[:2] for x in storages.values()]
        self.probes = [f for _, _, s in storages.values() for f in (s.data_ptr, s.nbytes)]   # (which hold them)
        self.found = [f() for f in self.probes]

    def check(self, upto=None) -> None:
        """A storage that was resized has freed the memory whose address was taken."""
        probes, found = self.probes, self.found
        if upto is not None:
            k = 2 * self.upto[upto]
            probes, found = probes[:k], found[:k]
        now = [f() for f in probes]
        if now != found:
            i = next(i for i in range(len(now)) if now[i] != found[i])
            raise ValueError("the storage of %s[%d] was resized since the list was made: make a new list" % self.names[i // 2])


class AdamTensors:
    """A list of tensors with their gradients and states, as the C ABI takes it.

    params (fp32), grads (all fp32 or all bf16), exp_avgs and exp_avg_sqs by `states`: "f32" and "bf16" tensors of
    as many elements, "8bit" uint8 tensors of fsdp_adam_state_bytes.  groups: each tensor's index into the
    hyper-parameters of a step (default 0).  param_bf16: a list, entries may be None.  For fsdp_adam_convert params and
    grads may be None.  In a list that a call writes no two params, states or copies may overlap.

    The list holds the tensors' memory as it was when the list was made, which takes 2.5 to 3.5 us a tensor: where a parameter
    or gradient is replaced by another tensor (as by zero_grad(set_to_none=True)), or its storage is resized, make a new
    list.  A resized storage is refused; to see that costs a call 60 ns for each storage that the tensors lie in."""

    def __init__(self, params, grads, exp_avgs, exp_avg_sqs, *, states: str = "f32", groups=None,
                 param_bf16=None):
        import torch
        _lib()
        self.format = L._kind(states, _STATES, "states")
        sdtype = {"f32": torch.float32, "bf16": torch.bfloat16, "8bit": torch.uint8}[states]
        exp_avgs, exp_avg_sqs = list(exp_avgs), list(exp_avg_sqs)
        self.n = n = len(exp_avgs)
        lists = {"exp_avgs": exp_avgs, "exp_avg_sqs": exp_avg_sqs}
        if (params is None) != (grads is None):
            raise TypeError("params and grads must be given together")
        self.steps = params is not None
        if self.steps:
            lists |= {"params": list(params), "grads": list(grads)}
        elif states == "8bit":
            raise TypeError("8-bit states need params, which say how many elements they have")
        if param_bf16 is not None:
            lists["param_bf16"] = list(param_bf16)
        if groups is not None:
            lists["groups"] = [int(g) for g in groups]
        for name, v in lists.items():
            if len(v) != n:
                raise ValueError("%s holds %d entries, %d are needed" % (name, len(v), n))
        self.groups = lists.get("groups", [0] * n)
        self.grad_dtype, gdtype = L.FSDP_F32, None
        if self.steps and n:
            if not isinstance(lists["grads"][0], L._Tensor):
                L._refuse(lists["grads"][0], "grads[0]", 0)
            self.grad_dtype = L._dtype_code(lists["grads"][0], "grads[0]")
            gdtype = lists["grads"][0].dtype
        self.device = None
        if n:
            if not isinstance(exp_avgs[0], L._Tensor) or not exp_avgs[0].is_cuda:
                L._refuse(exp_avgs[0], "exp_avgs[0]", 0)
            self.device = exp_avgs[0].get_device()
        sized = "params" if self.steps else "exp_avgs"
        for i, t in enumerate(lists[sized]):
            if not isinstance(t, L._Tensor):
                L._refuse(t, "%s[%d]" % (sized, i), 0)
        self.numels = [t.numel() for t in lists[sized]]
        dev = self.device
        table = (fsdp_adam_tensor * max(1, n))()
        spans, width = [], {"f32": 4, "bf16": 2, "8bit": 1}[states]
        for i in range(n):
            e, k = table[i], self.numels[i]
            e.numel = k
            e.group = self.groups[i]
            held = k if states != "8bit" else fsdp_adam_state_bytes(k)
            e.exp_avg = L._vector(exp_avgs[i], "exp_avgs[%d]" % i, held, dev, sdtype)
            e.exp_avg_sq = L._vector(exp_avg_sqs[i], "exp_avg_sqs[%d]" % i, held, dev, sdtype)
            if self.steps:
                e.param = L._vector(lists["params"][i], "params[%d]" % i, k, dev, torch.float32)
                e.grad = L._vector(lists["grads"][i], "grads[%d]" % i, k, dev, gdtype)
                spans.append((e.param, 4 * k, "params", i))
            if param_bf16 is not None and lists["param_bf16"][i] is not None:
                e.param_bf16 = L._vector(lists["param_bf16"][i], "param_bf16[%d]" % i, k, dev, torch.bfloat16)
                spans.append((e.param_bf16, 2 * k, "param_bf16", i))
            spans += (e.exp_avg, width * held, "exp_avgs", i), (e.exp_avg_sq, width * held, "exp_avg_sqs", i)
        self._overlap = None
        spans = sorted(x for x in spans if x[0] and x[1])
        for (a, size, first, i), (b, _, second, j) in zip(spans, spans[1:]):
            if a + size > b:
                self._overlap = "%s[%d] and %s[%d] overlap" % (first, i, second, j)
                break
        # the memory stays where the caller's tensors are given other storage
        self._held = _Held({name: v for name, v in lists.items() if name != "groups"})
        self._table = table
        self._address = ctypes.addressof(table)


def fsdp_adam_tensors(tensors: AdamTensors, groups, *, seed: int = 0, grad_scale=None, skip=None,
                      stream=None) -> None:
    """One AdamW step over the list.  groups: the hyper-parameters of every group, a dict (or a list of
    them) with lr, step and, where not the defaults, betas, eps and weight_decay.  grad_scale and skip: fp32
    tensors of one element on the GPU; where skip is not 0 nothing changes.  seed: of 8-bit states' rounding."""
    if not isinstance(tensors, AdamTensors):
        raise TypeError("tensors must be an AdamTensors, got %r" % type(tensors))
    if not tensors.steps:
        raise ValueError("the list has no params and grads")
    if tensors._overlap:
        raise ValueError(tensors._overlap)
    tensors._held.check()
    if isinstance(groups, dict):
        groups = (groups,)
    cfg = b"".join([_adam_cfg(**g) for g in groups])
    dev = tensors.device
    if dev is None:
        grad_scale = skip = None
    head = _ADAM_LIST.pack(tensors.n, len(groups), tensors.format, tensors.grad_dtype,
                           seed & 0xFFFFFFFFFFFFFFFF,
                           0 if grad_scale is None else L._vector(grad_scale, "grad_scale", 1, dev, L._f32),
                           0 if skip is None else L._vector(skip, "skip", 1, dev, L._f32))
    if dev is None:   # an empty list: its arguments are checked
        B._check(_fn.fsdp_adam_tensors(head, tensors._address, cfg, None))
        return
    L._call(_fn.fsdp_adam_tensors, dev, stream, head, tensors._address, cfg)


def _adam_cfg(lr, step, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0) -> bytes:
    return _ADAM_CFG.pack(lr, betas[0], betas[1], eps, weight_decay, step)


def fsdp_adam_convert(src: AdamTensors, dst: AdamTensors, *, seed: int = 0, step: int = 1,
                      stream=None) -> None:
    """Copy the states of one list to another of another format; one of the two is "8bit".  No state of dst may
    overlap another of either list."""
    for t, name in ((src, "src"), (dst, "dst")):
        if not isinstance(t, AdamTensors):
            raise TypeError("%s must be an AdamTensors, got %r" % (name, type(t)))
    if src.numels != dst.numels:
        raise ValueError("the lists hold tensors of different sizes")
    if dst._overlap:
        raise ValueError(dst._overlap)
    src._held.check("exp_avg_sqs")   # (the states come first)
    dst._held.check("exp_avg_sqs")
    dev = src.device
    if dst.device != dev:
        raise ValueError("the lists are on different GPUs")
    if dev is None:
        return
    L._call(_fn.fsdp_adam_convert, dev, stream, src.n, src._address, src.format, dst._address, dst.format,
            seed & 0xFFFFFFFFFFFFFFFF, step)
