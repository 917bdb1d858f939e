"""What the layer operators refuse, through the C ABI and the binding: every check runs on the host
before any HIP call, so all of this runs without a GPU (the addresses given are never read)."""
import ctypes

import pytest
import torch

from sharded_fsdp_flatten_amd import binding as B
from sharded_fsdp_flatten_amd import layer as L

OK, ARG, RANGE, ALIGN, OVERFLOW = 0, 1, 2, 3, 4
P = 0x7F0000000000


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(B.LIB_PATH):
        from sharded_fsdp_flatten_amd import build
        build.build()
    return L._lib()


def rows(p=P, pitch=100):
    return L.fsdp_rows(p, pitch)


def ckpt(**kw):
    return L.fsdp_ckpt(**{**dict(codes=P, scales=P, code_pitch=100, scale_pitch=4, format=1, reserved=0), **kw})


def cfg(**kw):
    return L.fsdp_layer_cfg(**{**dict(rows=10, cols=100, dtype=1, param_dtype=1, grad_dtype=2,
                                      accumulate=0, kind=1, eps=1e-5), **kw})


def call(f, c, io):
    """status of a call that has to be refused"""
    as_bytes = lambda s: None if s is None else bytes(s)  # noqa: E731
    return f(as_bytes(c), as_bytes(io), None)


def norm_fwd(**kw):
    q = kw.pop("q", None)
    io = L.fsdp_norm_fwd(**{**dict(x=rows(), y=rows(), weight=P, bias=P, mean=P, rstd=P), **kw})
    if q is not None:
        io.ckpt = ctypes.addressof(q)
    return io


def norm_bwd(**kw):
    q = kw.pop("q", None)
    io = L.fsdp_norm_bwd(**{**dict(dy=rows(), x=rows(), dx=rows(), weight=P, mean=P, rstd=P, dweight=P,
                                   dbias=P, workspace=P, workspace_len=1 << 30), **kw})
    if q is not None:
        io.ckpt = ctypes.addressof(q)
    return io


def act_bwd(**kw):
    q = kw.pop("q", None)
    io = L.fsdp_act_bwd(**{**dict(dy=rows(), x=rows(), dx=rows(), dbias=P, workspace=P, workspace_len=1 << 30), **kw})
    if q is not None:
        io.ckpt = ctypes.addressof(q)
    return io


def test_structures_match_their_packed_form():
    for packed, s in ((L._CFG, L.fsdp_layer_cfg), (L._NORM_FWD, L.fsdp_norm_fwd), (L._NORM_BWD, L.fsdp_norm_bwd),
                      (L._ACT_FWD, L.fsdp_act_fwd), (L._ACT_BWD, L.fsdp_act_bwd)):
        assert packed.size == ctypes.sizeof(s)


BAD_CFG = [(dict(rows=-1), RANGE), (dict(cols=-1), RANGE), (dict(cols=(1 << 30) + 1), RANGE), (dict(rows=(1 << 63) - 1), OVERFLOW),
           (dict(rows=1 << 40, cols=1 << 30), OVERFLOW), (dict(dtype=0), RANGE),
           (dict(dtype=3), RANGE), (dict(kind=0), RANGE), (dict(kind=9), RANGE)]
BAD_ROWS = [(dict(p=0), ARG), (dict(p=P + 1), ALIGN), (dict(pitch=-1), RANGE), (dict(pitch=1 << 61), OVERFLOW)]


@pytest.mark.parametrize("kw,want", BAD_CFG + [(dict(param_dtype=0), RANGE), (dict(eps=-1.0), RANGE),
                                               (dict(eps=float("nan")), RANGE), (dict(eps=float("inf")), RANGE)])
def test_norm_forward_cfg(lib, kw, want):
    assert call(lib.fsdp_norm_forward, cfg(**kw), norm_fwd()) == want
    assert B.fsdp_last_error()


@pytest.mark.parametrize("kw,want", BAD_ROWS)
def test_every_matrix_is_checked(lib, kw, want):
    bad = rows(**kw)
    none = kw.get("p") == 0
    for name in ("x", "y", "residual", "sum"):
        io = norm_fwd(**{"residual": rows(), "sum": rows(), name: bad})
        if none and name in ("residual", "sum"):
            continue  # optional: not given
        assert call(lib.fsdp_norm_forward, cfg(), io) == want, name
    for name in ("dy", "x", "dres", "dx", "y"):
        if none and name in ("dres", "y"):
            continue
        assert call(lib.fsdp_norm_backward, cfg(), norm_bwd(**{name: bad})) == want, name
        if name != "dres":
            assert call(lib.fsdp_act_backward, cfg(), act_bwd(**{name: bad})) == want, name
    for name in ("x", "y"):
        io = L.fsdp_act_fwd(**{**dict(x=rows(), y=rows()), name: bad})
        assert call(lib.fsdp_act_forward, cfg(), io) == want, name
    q = ckpt()
    assert lib.fsdp_ckpt_pack(10, 100, 1, bad, ctypes.addressof(q), None) == want
    assert lib.fsdp_ckpt_unpack(10, 100, 1, ctypes.addressof(q), bad, None) == want


def test_outputs_rows_must_not_overlap(lib):
    assert call(lib.fsdp_norm_forward, cfg(), norm_fwd(y=rows(pitch=99))) == RANGE
    assert call(lib.fsdp_norm_forward, cfg(), norm_fwd(residual=rows(), sum=rows(pitch=0))) == RANGE
    for io in (norm_bwd(dx=rows(pitch=0)), norm_bwd(y=rows(pitch=99))):
        assert call(lib.fsdp_norm_backward, cfg(), io) == RANGE
    for io in (act_bwd(dx=rows(pitch=0)), act_bwd(y=rows(pitch=99))):
        assert call(lib.fsdp_act_backward, cfg(), io) == RANGE
    q = ckpt()
    assert lib.fsdp_ckpt_unpack(10, 100, 1, ctypes.addressof(q), rows(pitch=99), None) == RANGE


@pytest.mark.parametrize("kw,want", [(dict(codes=0), ARG), (dict(scales=0), ARG), (dict(code_pitch=99), RANGE),
                                     (dict(scale_pitch=3), RANGE), (dict(code_pitch=-1), RANGE),
                                     (dict(format=0), RANGE), (dict(format=3), RANGE),
                                     (dict(code_pitch=1 << 62), OVERFLOW)])
def test_checkpoints_are_checked(lib, kw, want):
    q = ckpt(**kw)
    assert lib.fsdp_ckpt_pack(10, 100, 1, rows(), ctypes.addressof(q), None) == want
    assert call(lib.fsdp_norm_forward, cfg(), norm_fwd(q=q)) == want
    io = L.fsdp_act_fwd(x=rows(), y=rows(), ckpt=ctypes.addressof(q))
    assert call(lib.fsdp_act_forward, cfg(), io) == want
    if kw not in (dict(code_pitch=99), dict(scale_pitch=3)):  # overlapping rows may be read
        assert lib.fsdp_ckpt_unpack(10, 100, 1, ctypes.addressof(q), rows(), None) == want
        assert call(lib.fsdp_norm_backward, cfg(), norm_bwd(q=q, x=rows(0))) == want
        assert call(lib.fsdp_act_backward, cfg(), act_bwd(q=q, x=rows(0))) == want


def test_missing_and_contradicting_arguments(lib):
    for f, io in ((lib.fsdp_norm_forward, norm_fwd()), (lib.fsdp_norm_backward, norm_bwd()),
                  (lib.fsdp_act_backward, act_bwd())):
        assert call(f, None, io) == ARG
        assert call(f, cfg(), None) == ARG
    assert lib.fsdp_ckpt_pack(10, 100, 1, rows(), None, None) == ARG
    assert lib.fsdp_ckpt_unpack(10, 100, 1, None, rows(), None) == ARG
    for name in ("weight", "mean", "rstd"):
        assert call(lib.fsdp_norm_forward, cfg(), norm_fwd(**{name: 0})) == ARG
        assert call(lib.fsdp_norm_backward, cfg(), norm_bwd(**{name: 0})) == ARG
    assert call(lib.fsdp_norm_forward, cfg(), norm_fwd(sum=rows())) == ARG
    q = ckpt()
    assert call(lib.fsdp_norm_backward, cfg(), norm_bwd(q=q)) == ARG             # both
    assert call(lib.fsdp_norm_backward, cfg(), norm_bwd(x=rows(0))) == ARG       # neither
    assert call(lib.fsdp_act_backward, cfg(), act_bwd(q=q)) == ARG
    assert call(lib.fsdp_act_backward, cfg(), act_bwd(x=rows(0))) == ARG
    for name in ("weight", "bias"):
        assert call(lib.fsdp_norm_forward, cfg(), norm_fwd(**{name: P + 1})) == ALIGN
    for name in ("mean", "rstd"):
        assert call(lib.fsdp_norm_forward, cfg(), norm_fwd(**{name: P + 2})) == ALIGN
    for name in ("dweight", "dbias"):
        assert call(lib.fsdp_norm_backward, cfg(), norm_bwd(**{name: P + 2})) == ALIGN
    assert call(lib.fsdp_norm_backward, cfg(grad_dtype=0), norm_bwd()) == RANGE
    assert call(lib.fsdp_act_backward, cfg(grad_dtype=5), act_bwd()) == RANGE


def test_workspaces(lib):
    n = ctypes.c_int64()
    for size, f, make in ((lib.fsdp_norm_workspace, lib.fsdp_norm_backward, norm_bwd),
                          (lib.fsdp_act_workspace, lib.fsdp_act_backward, act_bwd)):
        assert size(10, 100, ctypes.byref(n)) == OK and n.value > 0
        need = n.value
        assert call(f, cfg(), make(workspace_len=need - 1)) == RANGE
        assert call(f, cfg(), make(workspace=0)) == ARG
        assert call(f, cfg(), make(workspace=P + 4)) == ALIGN
        assert size(0, 100, ctypes.byref(n)) == OK and n.value == 0
        assert size(10, 0, ctypes.byref(n)) == OK and n.value == 0
        assert size(-1, 100, ctypes.byref(n)) == RANGE
        assert size(10, (1 << 30) + 1, ctypes.byref(n)) == RANGE
        assert size((1 << 63) - 1, 1, ctypes.byref(n)) == OVERFLOW
        assert size(1 << 58, 1, ctypes.byref(n)) == OK and n.value > 0
        assert size(10, 100, None) == ARG
        # a quarter byte an element at most where there are many, so no more than an eighth of a bf16 matrix
        for r, c in ((1 << 30, 1024), (1 << 20, 512), (8192, 12288), (2048, 65536), (4096, 100000)):
            assert size(r, c, ctypes.byref(n)) == OK and 0 < n.value <= r * c // 16 + 2 * r + 4096


def test_nothing_to_do_needs_no_buffers(lib):
    for r, c in ((0, 100), (10, 0), (0, 0)):
        k = cfg(rows=r, cols=c)
        z = L.fsdp_rows(0, 0)
        assert call(lib.fsdp_norm_forward, k, L.fsdp_norm_fwd()) == OK
        assert call(lib.fsdp_norm_backward, k, L.fsdp_norm_bwd()) == OK
        assert call(lib.fsdp_act_forward, k, L.fsdp_act_fwd()) == OK
        assert call(lib.fsdp_act_backward, k, L.fsdp_act_bwd()) == OK
        q = ckpt(codes=0, scales=0)
        assert lib.fsdp_ckpt_pack(r, c, 1, z, ctypes.addressof(q), None) == OK
        assert lib.fsdp_ckpt_unpack(r, c, 1, ctypes.addressof(q), z, None) == OK


def test_the_binding_takes_gpu_tensors_only():
    x, w = torch.zeros(4, 8), torch.zeros(8)
    m = torch.zeros(4)
    with pytest.raises(ValueError, match="GPU"):
        L.fsdp_norm_forward(x, w, None, x.clone(), m, m.clone())
    with pytest.raises(ValueError, match="GPU"):
        L.fsdp_act_forward(x, x.clone(), kind="relu")
    with pytest.raises(ValueError, match="GPU"):
        L.Ckpt.empty(4, 8, device="cpu")
    with pytest.raises(TypeError):
        L.fsdp_act_forward(x.double(), x.double(), kind="relu")
    with pytest.raises(TypeError):
        L.fsdp_norm_backward([1.0], x, w, m, m, x, w, w, None)
