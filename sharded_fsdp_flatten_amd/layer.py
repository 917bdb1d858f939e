"""ctypes binding of the layer operators, with the C ABI's names: 8-bit activation checkpoints,
LayerNorm / RMSNorm and the MLP activation, forward and backward.

Argument marshalling only, as in ``binding``: activations are tensors of rows x cols (the last
dimension is cols, the ones before it count as rows; two-dimensional tensors may have any row
stride), dtypes are read off the tensors, the stream defaults to torch's current one.  Where a
backward pass takes the forward pass's input, it takes the tensor or a ``Ckpt`` of it.

>>> q = Ckpt.empty(tokens, 1280, "e4m3", device="cuda")
>>> fsdp_norm_forward(x, w, b, y, mean, rstd, kind="layer", eps=1e-5, ckpt=q)
>>> ws = torch.empty(fsdp_norm_workspace(tokens, 1280), device="cuda")
>>> fsdp_norm_backward(dy, q, w, mean, rstd, dx, dw, db, ws, kind="layer")
"""
from __future__ import annotations

import ctypes
import struct

from . import binding as B

FSDP_BF16 = 1
FSDP_F32 = 2
FSDP_CKPT_E4M3 = 1
FSDP_CKPT_INT8 = 2
FSDP_CKPT_GROUP = 32
FSDP_NORM_LAYER = 1
FSDP_NORM_RMS = 2
FSDP_ACT_RELU = 1
FSDP_ACT_GELU = 2
FSDP_ACT_GELU_TANH = 3
FSDP_ACT_SILU = 4

_FORMATS = {"e4m3": FSDP_CKPT_E4M3, "int8": FSDP_CKPT_INT8}
_NORMS = {"layer": FSDP_NORM_LAYER, "rms": FSDP_NORM_RMS}
_ACTS = {"relu": FSDP_ACT_RELU, "gelu": FSDP_ACT_GELU, "gelu_tanh": FSDP_ACT_GELU_TANH,
         "silu": FSDP_ACT_SILU}


class fsdp_rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("pitch", ctypes.c_int64)]


class fsdp_ckpt(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("code_pitch", ctypes.c_int64), ("scale_pitch", ctypes.c_int64),
                ("format", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class fsdp_layer_cfg(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("param_dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32),
                ("accumulate", ctypes.c_int32), ("kind", ctypes.c_int32), ("eps", ctypes.c_float)]


class fsdp_norm_fwd(ctypes.Structure):
    _fields_ = [("x", fsdp_rows), ("residual", fsdp_rows), ("sum", fsdp_rows), ("y", fsdp_rows),
                ("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("mean", ctypes.c_void_p),
                ("rstd", ctypes.c_void_p), ("ckpt", ctypes.c_void_p)]


class fsdp_norm_bwd(ctypes.Structure):
    _fields_ = [("dy", fsdp_rows), ("x", fsdp_rows), ("dres", fsdp_rows), ("dx", fsdp_rows),
                ("y", fsdp_rows), ("ckpt", ctypes.c_void_p), ("weight", ctypes.c_void_p),
                ("bias", ctypes.c_void_p), ("mean", ctypes.c_void_p), ("rstd", ctypes.c_void_p),
                ("dweight", ctypes.c_void_p), ("dbias", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("workspace_len", ctypes.c_int64)]


class fsdp_act_fwd(ctypes.Structure):
    _fields_ = [("x", fsdp_rows), ("y", fsdp_rows), ("ckpt", ctypes.c_void_p)]


class fsdp_act_bwd(ctypes.Structure):
    _fields_ = [("dy", fsdp_rows), ("x", fsdp_rows), ("dx", fsdp_rows), ("y", fsdp_rows),
                ("ckpt", ctypes.c_void_p), ("dbias", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("workspace_len", ctypes.c_int64)]


# The same structures packed in one call each: filling ctypes fields one by one costs more than
# a short launch.
_CFG = struct.Struct("@qqiiiiif")
_NORM_FWD = struct.Struct("@" + "Pq" * 4 + "PPPPP")
_NORM_BWD = struct.Struct("@" + "Pq" * 5 + "PPPPPPPPq")
_ACT_FWD = struct.Struct("@" + "Pq" * 2 + "P")
_ACT_BWD = struct.Struct("@" + "Pq" * 4 + "PPPq")
_NONE = (0, 0)

_fn = None
_Tensor = None      # torch.Tensor
_codes = None       # torch dtype -> fsdp_dtype
_f32 = None
_device = None      # the current GPU's index
_raw_stream = None  # its current stream's handle


def _lib():
    """The library, with the argument types of this module's calls set once."""
    global _fn, _Tensor, _codes, _f32, _device, _raw_stream
    if _fn is None:
        import torch
        lib = B.load()
        cfg, io, vp = ctypes.c_char_p, ctypes.c_char_p, ctypes.c_void_p
        i64, i32 = ctypes.c_int64, ctypes.c_int32
        lib.fsdp_ckpt_pack.argtypes = [i64, i64, i32, fsdp_rows, vp, vp]
        lib.fsdp_ckpt_unpack.argtypes = [i64, i64, i32, vp, fsdp_rows, vp]
        for f in (lib.fsdp_norm_forward, lib.fsdp_norm_backward, lib.fsdp_act_forward,
                  lib.fsdp_act_backward):
            f.argtypes = [cfg, io, vp]
        for f in (lib.fsdp_norm_workspace, lib.fsdp_act_workspace):
            f.argtypes = [i64, i64, ctypes.POINTER(i64)]
        for f in (lib.fsdp_ckpt_pack, lib.fsdp_ckpt_unpack, lib.fsdp_norm_forward,
                  lib.fsdp_norm_backward, lib.fsdp_norm_workspace, lib.fsdp_act_forward,
                  lib.fsdp_act_backward, lib.fsdp_act_workspace):
            f.restype = i32
        _Tensor, _f32 = torch.Tensor, torch.float32
        _codes = {torch.bfloat16: FSDP_BF16, torch.float32: FSDP_F32}
        _device = torch.cuda.current_device
        # the handle alone costs 0.1 us, torch.cuda.current_stream's object 2 us
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda d: torch.cuda.current_stream(d).cuda_stream)
        _fn = lib
    return _fn


def _dtype_code(t, name: str) -> int:
    try:
        return _codes[t.dtype]
    except KeyError:
        raise TypeError("%s must be bfloat16 or float32, got %s" % (name, t.dtype)) from None


def _refuse(t, name: str, device: int) -> None:
    """Why a value is no tensor on this GPU."""
    if not isinstance(t, _Tensor):
        raise TypeError("%s must be a tensor, got %r" % (name, type(t)))
    if not t.is_cuda:
        # a host address would reach the kernels and fault the GPU
        raise ValueError("tensors passed to the library must be on the GPU, %s is on %s"
                         % (name, t.device))
    raise ValueError("%s is on GPU %d, the others are on GPU %d" % (name, t.get_device(), device))


def _first(t, name: str):
    """(rows, cols, dtype, its code, GPU) of the activation that sets them for a call: the last
    dimension is cols, the ones before it count as rows."""
    if _fn is None:
        _lib()
    if not isinstance(t, _Tensor):
        _refuse(t, name, 0)
    code = _dtype_code(t, name)
    if not t.is_cuda:
        _refuse(t, name, 0)
    shape = t.shape
    if len(shape) == 2:
        rows, cols = shape
    elif shape:
        cols, rows = shape[-1], 1
        for d in shape[:-1]:
            rows *= d
    else:
        raise ValueError("%s must have at least one dimension" % name)
    return rows, cols, t.dtype, code, t.get_device()


def _rows(t, name: str, rows: int, cols: int, dtype, device: int):
    """(address, pitch) of an activation of rows x cols elements."""
    if not isinstance(t, _Tensor) or t.get_device() != device:
        _refuse(t, name, device)
    if t.dtype is not dtype:
        raise TypeError("%s is %s, the others are %s" % (name, t.dtype, dtype))
    shape = t.shape
    if len(shape) == 2:
        if shape[0] != rows or shape[1] != cols:
            raise ValueError("%s has shape %s, %d rows of %d columns are needed"
                             % (name, tuple(shape), rows, cols))
        pitch, inner = t.stride()
        if inner != 1 and cols > 1:
            raise ValueError("the columns of %s must be next to each other (stride 1), got stride %d"
                             % (name, inner))
        return t.data_ptr(), pitch
    if _first(t, name)[:2] != (rows, cols):
        raise ValueError("%s has shape %s, %d rows of %d columns are needed"
                         % (name, tuple(shape), rows, cols))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous or two-dimensional" % name)
    return t.data_ptr(), cols


def _vector(t, name: str, n: int, device: int, dtype=None) -> int:
    if t is None:
        return 0
    if not isinstance(t, _Tensor) or t.get_device() != device:
        _refuse(t, name, device)
    if dtype is not None and t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.numel() != n:
        raise ValueError("%s holds %d elements, %d are needed" % (name, t.numel(), n))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _grad_code(dweight, dbias) -> int:
    if dweight is None:
        return FSDP_F32 if dbias is None else _dtype_code(dbias, "dbias")
    if dbias is not None and isinstance(dbias, _Tensor) and dbias.dtype is not dweight.dtype:
        raise TypeError("dweight and dbias must have the same dtype")
    return _dtype_code(dweight, "dweight")


def _kind(kind, names: dict, what: str) -> int:
    try:
        return names[kind]
    except (KeyError, TypeError):
        raise ValueError("%s must be one of %s, got %r" % (what, ", ".join(names), kind)) from None


def _call(fn, device: int, stream, *args) -> None:
    """The call on the tensors' GPU and its current stream, or the one given."""
    current = _device()
    if current != device:
        import torch
        with torch.cuda.device(device):
            return _call(fn, device, stream, *args)
    if stream is None:
        stream = _raw_stream(device)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    status = fn(*args, stream)
    if status:
        B._check(status)


class Ckpt:
    """An 8-bit checkpoint of a rows x cols activation: `codes` (uint8, rows x cols) and `scales`
    (uint8, rows x ceil(cols / 32)), either with any row stride, and the format, "e4m3" or "int8"."""

    def __init__(self, codes, scales, format: str):
        _lib()
        for t, name in ((codes, "codes"), (scales, "scales")):
            if not isinstance(t, _Tensor) or not t.is_cuda or t.get_device() != codes.get_device():
                _refuse(t, name, codes.get_device() if isinstance(codes, _Tensor) else 0)
            if str(t.dtype) != "torch.uint8" or t.dim() != 2:
                raise TypeError("%s must be a two-dimensional uint8 tensor" % name)
            if t.shape[1] > 1 and t.stride(1) != 1:
                raise ValueError("the columns of %s must be next to each other" % name)
        self.rows, self.cols = codes.shape
        groups = -(-self.cols // FSDP_CKPT_GROUP)
        if tuple(scales.shape) != (self.rows, groups):
            raise ValueError("scales has shape %s, %s is needed"
                             % (tuple(scales.shape), (self.rows, groups)))
        self.codes, self.scales, self.format = codes, scales, format
        self.device = codes.get_device()
        self._c = fsdp_ckpt(codes.data_ptr() or None, scales.data_ptr() or None, codes.stride(0),
                            scales.stride(0), _kind(format, _FORMATS, "format"), 0)
        self._address = ctypes.addressof(self._c)

    @classmethod
    def empty(cls, rows: int, cols: int, format: str = "e4m3", device="cuda") -> "Ckpt":
        """A checkpoint of newly allocated tensors."""
        import torch
        return cls(torch.empty(rows, cols, dtype=torch.uint8, device=device),
                   torch.empty(rows, -(-cols // FSDP_CKPT_GROUP), dtype=torch.uint8, device=device),
                   format)

    def check(self, rows: int, cols: int, device: int) -> int:
        """Address of the C structure, for an activation of these sizes."""
        if (self.rows, self.cols) != (rows, cols):
            raise ValueError("the checkpoint holds %d x %d, %d x %d is needed"
                             % (self.rows, self.cols, rows, cols))
        if self.device != device:
            raise ValueError("the checkpoint is on GPU %d, the others are on GPU %d"
                             % (self.device, device))
        return self._address


def _ckpt(ckpt, rows: int, cols: int, device: int) -> int:
    if not isinstance(ckpt, Ckpt):
        raise TypeError("ckpt must be a Ckpt, got %r" % type(ckpt))
    return ckpt.check(rows, cols, device)


def fsdp_ckpt_pack(x, ckpt: Ckpt, stream=None) -> None:
    """Save x in 8 bits."""
    rows, cols, t, code, dev = _first(x, "x")
    xr = _rows(x, "x", rows, cols, t, dev)
    _call(_fn.fsdp_ckpt_pack, dev, stream, rows, cols, code, fsdp_rows(*xr),
          _ckpt(ckpt, rows, cols, dev))


def fsdp_ckpt_unpack(ckpt: Ckpt, x, stream=None) -> None:
    """Write the values a checkpoint holds to x (exact in bf16 and fp32)."""
    rows, cols, t, code, dev = _first(x, "x")
    xr = _rows(x, "x", rows, cols, t, dev)
    _call(_fn.fsdp_ckpt_unpack, dev, stream, rows, cols, code, _ckpt(ckpt, rows, cols, dev),
          fsdp_rows(*xr))


def _params(weight, bias, cols: int, dev: int):
    w = _vector(weight, "weight", cols, dev)
    if not w and cols:
        raise TypeError("weight must be a tensor, got %r" % type(weight))
    code = _dtype_code(weight, "weight")
    return code, w, 0 if bias is None else _vector(bias, "bias", cols, dev, weight.dtype)


def fsdp_norm_forward(x, weight, bias, y, mean, rstd, *, kind: str = "layer", eps: float = 1e-5,
                      residual=None, sum=None, ckpt=None, stream=None) -> None:
    """y = norm(x) or, with `residual`, norm(x + residual); the sum goes to `sum`, the statistics
    to mean (None for "rms") and rstd, and the norm's input in 8 bits to `ckpt`, where given."""
    rows, cols, t, code, dev = _first(x, "x")
    pcode, w, b = _params(weight, bias, cols, dev)
    cfg = _CFG.pack(rows, cols, code, pcode, FSDP_F32, 0, _kind(kind, _NORMS, "kind"), eps)
    io = _NORM_FWD.pack(
        *_rows(x, "x", rows, cols, t, dev),
        *(_NONE if residual is None else _rows(residual, "residual", rows, cols, t, dev)),
        *(_NONE if sum is None else _rows(sum, "sum", rows, cols, t, dev)),
        *_rows(y, "y", rows, cols, t, dev), w, b,
        _vector(mean, "mean", rows, dev, _f32), _vector(rstd, "rstd", rows, dev, _f32),
        0 if ckpt is None else _ckpt(ckpt, rows, cols, dev))
    _call(_fn.fsdp_norm_forward, dev, stream, cfg, io)


def fsdp_norm_workspace(rows: int, cols: int) -> int:
    """fp32 elements of workspace fsdp_norm_backward needs."""
    n = ctypes.c_int64()
    B._check(_lib().fsdp_norm_workspace(rows, cols, ctypes.byref(n)))
    return int(n.value)


def _input(x, rows: int, cols: int, t, dev: int):
    """(address, pitch, checkpoint) of a backward pass's input, a tensor or a checkpoint."""
    if isinstance(x, Ckpt):
        return 0, 0, x.check(rows, cols, dev)
    return (*_rows(x, "x", rows, cols, t, dev), 0)


def _workspace(ws, dev: int):
    if ws is None:
        return 0, 0
    n = ws.numel() if isinstance(ws, _Tensor) else 0
    return _vector(ws, "workspace", n, dev, _f32), n


def fsdp_norm_backward(dy, x, weight, mean, rstd, dx, dweight, dbias, workspace, *,
                       kind: str = "layer", dres=None, y=None, bias=None,
                       accumulate: bool = False, stream=None) -> None:
    """Gradients of the norm's input (plus `dres`, where given), weight and bias (either may be
    None) from the input x, a tensor or a Ckpt; `y` receives the norm's output again (`bias` is
    read for it alone).  With `accumulate` dweight and dbias are added to."""
    rows, cols, t, code, dev = _first(dy, "dy")
    pcode, w, b = _params(weight, bias, cols, dev)
    xp, xpitch, q = _input(x, rows, cols, t, dev)
    dw, db = _vector(dweight, "dweight", cols, dev), _vector(dbias, "dbias", cols, dev)
    cfg = _CFG.pack(rows, cols, code, pcode, _grad_code(dweight, dbias), 1 if accumulate else 0,
                    _kind(kind, _NORMS, "kind"), 0.0)
    io = _NORM_BWD.pack(
        *_rows(dy, "dy", rows, cols, t, dev), xp, xpitch,
        *(_NONE if dres is None else _rows(dres, "dres", rows, cols, t, dev)),
        *_rows(dx, "dx", rows, cols, t, dev),
        *(_NONE if y is None else _rows(y, "y", rows, cols, t, dev)), q, w, b,
        _vector(mean, "mean", rows, dev, _f32), _vector(rstd, "rstd", rows, dev, _f32), dw, db,
        *_workspace(workspace, dev))
    _call(_fn.fsdp_norm_backward, dev, stream, cfg, io)


def fsdp_act_forward(x, y, *, kind: str, ckpt=None, stream=None) -> None:
    """y = f(x), f one of "relu", "gelu", "gelu_tanh", "silu"; x in 8 bits to `ckpt`, where given."""
    rows, cols, t, code, dev = _first(x, "x")
    cfg = _CFG.pack(rows, cols, code, FSDP_F32, FSDP_F32, 0, _kind(kind, _ACTS, "kind"), 0.0)
    io = _ACT_FWD.pack(*_rows(x, "x", rows, cols, t, dev), *_rows(y, "y", rows, cols, t, dev),
                       0 if ckpt is None else _ckpt(ckpt, rows, cols, dev))
    _call(_fn.fsdp_act_forward, dev, stream, cfg, io)


def fsdp_act_workspace(rows: int, cols: int) -> int:
    """fp32 elements of workspace fsdp_act_backward needs for dbias."""
    n = ctypes.c_int64()
    B._check(_lib().fsdp_act_workspace(rows, cols, ctypes.byref(n)))
    return int(n.value)


def fsdp_act_backward(dy, x, dx, dbias=None, workspace=None, *, kind: str, y=None,
                      accumulate: bool = False, stream=None) -> None:
    """dx = dy f'(x) from the input x, a tensor or a Ckpt; dbias (optional) receives the column
    sums of dx, y (optional) the activation's output again."""
    rows, cols, t, code, dev = _first(dy, "dy")
    xp, xpitch, q = _input(x, rows, cols, t, dev)
    db = _vector(dbias, "dbias", cols, dev)
    cfg = _CFG.pack(rows, cols, code, FSDP_F32, _grad_code(None, dbias), 1 if accumulate else 0,
                    _kind(kind, _ACTS, "kind"), 0.0)
    io = _ACT_BWD.pack(*_rows(dy, "dy", rows, cols, t, dev), xp, xpitch,
                       *_rows(dx, "dx", rows, cols, t, dev),
                       *(_NONE if y is None else _rows(y, "y", rows, cols, t, dev)), q, db,
                       *_workspace(workspace, dev))
    _call(_fn.fsdp_act_backward, dev, stream, cfg, io)
