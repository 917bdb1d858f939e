"""What the training step's other operators refuse, through the C ABI and the binding, and what their host
calls compute: every check runs before any HIP call, so all of this runs without a GPU (the addresses given
are never read)."""
import ctypes
import os

import numpy as np
import pytest
import torch

import train_ref as R
from sharded_fsdp_flatten_amd import binding as B
from sharded_fsdp_flatten_amd import layer as L
from sharded_fsdp_flatten_amd import train as T

OK, ARG, RANGE, ALIGN, OVERFLOW = 0, 1, 2, 3, 4
P = 0x7F0000000000


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from sharded_fsdp_flatten_amd import build
        build.build()
    return T._lib()


def as_bytes(s):
    return None if s is None else bytes(s)


def test_structures_match_their_packed_form():
    for packed, s in ((T._ROTARY_CFG, T.fsdp_rotary_cfg), (T._ROTARY_IO, T.fsdp_rotary_io), (T._LOGPROB_CFG, T.fsdp_logprob_cfg),
                      (T._LOGPROB_FWD, T.fsdp_logprob_fwd), (T._LOGPROB_BWD, T.fsdp_logprob_bwd), (T._ADAM_LIST, T.fsdp_adam_list),
                      (T._ADAM_CFG, B.fsdp_adamw_cfg)):
        assert packed.size == ctypes.sizeof(s)


# ---------------------------------------------------------------------------
# rotary
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("rot", [2, 6, 64, 128, 1024])
@pytest.mark.parametrize("kw", [dict(), dict(base=5e5), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
                                dict(scaling="parts", factor=8.0, trained_len=4096),
                                dict(scaling="parts", factor=32.0, trained_len=8192, low=1.0, high=4.0)])
def test_frequencies(lib, rot, kw):
    if kw.get("scaling") == "ntk" and rot == 2:
        with pytest.raises(B.FsdpError, match="more than one pair"):
            T.fsdp_rotary_freqs(rot, **kw)
        return
    got = T.fsdp_rotary_freqs(rot, **kw).numpy()
    # a power, a quotient, and sums of values of one sign: a few roundings, and the exponent's own
    assert np.allclose(got, R.freqs(rot, **kw), rtol=64 * 2.0 ** -53, atol=0)


@pytest.mark.parametrize("kw", [dict(rot=0), dict(rot=-2), dict(rot=3), dict(rot=1026), dict(rot=8, base=0.0), dict(rot=8, base=float("inf")),
                                dict(rot=8, scaling="linear", factor=0.0), dict(rot=8, scaling="ntk", factor=float("nan")),
                                dict(rot=8, scaling="parts", factor=2.0), dict(rot=8, scaling="parts", factor=2.0, trained_len=9, low=4.0, high=4.0),
                                dict(rot=8, scaling="parts", factor=2.0, trained_len=9, low=float("nan"))])
def test_frequencies_refused(lib, kw):
    with pytest.raises(B.FsdpError, match="FSDP_E_RANGE"):
        T.fsdp_rotary_freqs(**kw)


def test_frequency_scalings_by_name_and_null(lib):
    with pytest.raises(ValueError, match="scaling"):
        T.fsdp_rotary_freqs(8, scaling="yes")
    assert lib.fsdp_rotary_freqs(8, 1e4, 0, 1.0, 0, 0.0, 1.0, None) == ARG
    assert lib.fsdp_rotary_freqs(8, 1e4, 4, 1.0, 0, 0.0, 1.0, P) == RANGE


def heads(p=P, b=4096, t=512, h=64):
    return T.fsdp_heads(p, b, t, h)


def rotary(lib, cfg=None, io=None, f="fsdp_rotary_forward", null=None):
    c = T.fsdp_rotary_cfg(**{**dict(batch=2, tokens=8, heads=8, kv_heads=2, head_dim=64, rot=64, start=0, dtype=1, layout=1, scale=1.0), **(cfg or {})})
    i = T.fsdp_rotary_io(**{**dict(q=heads(), q_out=heads(), k=heads(), k_out=heads(), positions=P, freqs=P), **(io or {})})
    return getattr(lib, f)(None if null == "cfg" else bytes(c), None if null == "io" else bytes(i), None)


@pytest.mark.parametrize("kw,want", [(dict(batch=-1), RANGE), (dict(tokens=-1), RANGE), (dict(heads=-1), RANGE), (dict(heads=65537), RANGE),
                                     (dict(kv_heads=-1), RANGE), (dict(kv_heads=65537), RANGE), (dict(head_dim=0), RANGE),
                                     (dict(head_dim=1025), RANGE), (dict(rot=0), RANGE), (dict(rot=63), RANGE), (dict(rot=66), RANGE),
                                     (dict(dtype=0), RANGE), (dict(dtype=3), RANGE), (dict(layout=0), RANGE), (dict(layout=3), RANGE),
                                     (dict(scale=float("nan")), RANGE), (dict(scale=float("inf")), RANGE),
                                     (dict(tokens=1 << 60), OVERFLOW)])
def test_rotary_cfg(lib, kw, want):
    for f in ("fsdp_rotary_forward", "fsdp_rotary_backward"):
        assert rotary(lib, kw, f=f) == want
        assert B.fsdp_last_error()


@pytest.mark.parametrize("name", ["q", "q_out", "k", "k_out"])
def test_rotary_buffers(lib, name):
    assert rotary(lib, io={name: heads(p=0)}) == ARG
    assert rotary(lib, io={name: heads(p=P + 1)}) == ALIGN
    assert rotary(lib, dict(dtype=2), io={name: heads(p=P + 2)}) == ALIGN
    for kw in (dict(b=-1), dict(t=-1), dict(h=-1)):
        assert rotary(lib, io={name: heads(**kw)}) == RANGE
    assert rotary(lib, io={name: heads(b=1 << 62)}) == OVERFLOW
    if name.endswith("out"):
        for kw in (dict(h=63), dict(t=64), dict(b=3711), dict(h=0), dict(t=0), dict(b=0), dict(b=64, t=64 * 2, h=64)):
            assert rotary(lib, io={name: heads(**kw)}) == RANGE, kw


def test_rotary_missing_arguments(lib):
    assert rotary(lib, null="cfg") == ARG and rotary(lib, null="io") == ARG
    assert rotary(lib, io=dict(freqs=0)) == ARG
    assert rotary(lib, io=dict(freqs=P + 4)) == ALIGN
    assert rotary(lib, io=dict(positions=P + 4)) == ALIGN


def test_rotary_nothing_to_do(lib):
    none = T.fsdp_heads()
    for kw in (dict(batch=0), dict(tokens=0), dict(heads=0, kv_heads=0)):
        assert rotary(lib, kw, dict(q=none, q_out=none, k=none, k_out=none, positions=0, freqs=0)) == OK


# ---------------------------------------------------------------------------
# log probabilities
# ---------------------------------------------------------------------------
def lp_cfg(**kw):
    return T.fsdp_logprob_cfg(**{**dict(rows=10, cols=100, dtype=1, top=0, scale=1.0), **kw})


def rows(p=P, pitch=100):
    return L.fsdp_rows(p, pitch)


def lp_fwd(lib, cfg=None, **kw):
    io = T.fsdp_logprob_fwd(**{**dict(logits=rows(), tokens=P, logprob=P, max=P, logsum=P, entropy=P, top_logprob=P, top_token=P,
                                      workspace=P, workspace_len=1 << 40), **kw})
    return lib.fsdp_logprob_forward(bytes(lp_cfg(**(cfg or {}))), bytes(io), None)


def lp_bwd(lib, cfg=None, **kw):
    io = T.fsdp_logprob_bwd(**{**dict(logits=rows(), dlogits=rows(), tokens=P, dlogprob=P, dentropy=P, max=P, logsum=P, entropy=P), **kw})
    return lib.fsdp_logprob_backward(bytes(lp_cfg(**(cfg or {}))), bytes(io), None)


BAD_CFG = [(dict(rows=-1), RANGE), (dict(cols=-1), RANGE), (dict(cols=(1 << 30) + 1), RANGE), (dict(rows=1 << 40, cols=1 << 30), OVERFLOW),
           (dict(dtype=0), RANGE), (dict(dtype=3), RANGE), (dict(scale=0.0), RANGE), (dict(scale=-1.0), RANGE),
           (dict(scale=float("nan")), RANGE), (dict(scale=float("inf")), RANGE)]


@pytest.mark.parametrize("kw,want", BAD_CFG)
def test_logprob_cfg(lib, kw, want):
    assert lp_fwd(lib, kw) == want and B.fsdp_last_error()
    assert lp_bwd(lib, kw) == want


@pytest.mark.parametrize("top", [-1, 65, 101])
def test_logprob_top(lib, top):
    assert lp_fwd(lib, dict(top=top)) == RANGE
    n = ctypes.c_int64()
    assert lib.fsdp_logprob_workspace(10, 100, top, ctypes.byref(n)) == RANGE


def test_logprob_top_is_no_more_than_cols(lib):
    assert lp_fwd(lib, dict(cols=9, top=10)) == RANGE
    with pytest.raises(B.FsdpError):
        T.fsdp_logprob_workspace(10, 9, 10)


def test_logprob_buffers(lib):
    for bad, want in ((rows(0), ARG), (rows(P + 1), ALIGN), (rows(pitch=-1), RANGE), (rows(pitch=1 << 61), OVERFLOW)):
        assert lp_fwd(lib, logits=bad) == want
        assert lp_bwd(lib, logits=bad) == want
        assert lp_bwd(lib, dlogits=bad) == want
    assert lp_bwd(lib, dlogits=rows(pitch=99)) == RANGE
    for name in ("max", "logsum"):
        for v, want in ((0, ARG), (P + 2, ALIGN)):
            assert lp_fwd(lib, **{name: v}) == want
            assert lp_bwd(lib, **{name: v}) == want
    assert lp_fwd(lib, tokens=0) == ARG and lp_fwd(lib, logprob=0) == ARG
    assert lp_fwd(lib, tokens=P + 4) == ALIGN and lp_fwd(lib, logprob=P + 2) == ALIGN and lp_fwd(lib, entropy=P + 2) == ALIGN
    for name, off in (("top_logprob", 2), ("top_token", 4)):
        assert lp_fwd(lib, dict(top=5), **{name: 0}) == ARG
        assert lp_fwd(lib, dict(top=5), **{name: P + off}) == ALIGN
    assert lp_bwd(lib, dlogprob=0, dentropy=0) == ARG
    assert lp_bwd(lib, tokens=0) == ARG and lp_bwd(lib, entropy=0) == ARG
    for name, off in (("tokens", 4), ("dlogprob", 2), ("dentropy", 2), ("entropy", 2)):
        assert lp_bwd(lib, **{name: P + off}) == ALIGN
    assert lib.fsdp_logprob_forward(None, bytes(T.fsdp_logprob_fwd()), None) == ARG
    assert lib.fsdp_logprob_forward(bytes(lp_cfg()), None, None) == ARG
    assert lib.fsdp_logprob_backward(None, bytes(T.fsdp_logprob_bwd()), None) == ARG
    assert lib.fsdp_logprob_backward(bytes(lp_cfg()), None, None) == ARG


def test_logprob_workspace(lib):
    n = ctypes.c_int64()
    assert lib.fsdp_logprob_workspace(10, 100, 0, None) == ARG
    assert lib.fsdp_logprob_workspace(-1, 100, 0, ctypes.byref(n)) == RANGE
    assert lib.fsdp_logprob_workspace(1, (1 << 30) + 1, 0, ctypes.byref(n)) == RANGE
    for r, c in ((0, 100), (100, 0), (0, 0)):
        assert T.fsdp_logprob_workspace(r, c) == 0
    for r, c in ((1, 1), (1, 50257), (3, 262144), (1, 1 << 30), (300, 200001), (1 << 20, 50257)):
        for top in (0, 1, 64):
            need = T.fsdp_logprob_workspace(r, c, min(top, c))
            assert 0 <= need <= r * c  # never more than the logits themselves, in floats
            if need:
                big = dict(rows=r, cols=c, top=min(top, c))
                io = dict(logits=rows(pitch=c))
                assert lp_fwd(lib, big, workspace_len=need - 1, **io) == RANGE
                assert lp_fwd(lib, big, workspace=0, **io) == ARG
                assert lp_fwd(lib, big, workspace=P + 4, **io) == ALIGN


def test_logprob_nothing_to_do(lib):
    for r, c in ((0, 100), (10, 0), (0, 0)):
        k = bytes(lp_cfg(rows=r, cols=c))
        assert lib.fsdp_logprob_forward(k, bytes(T.fsdp_logprob_fwd()), None) == OK
        assert lib.fsdp_logprob_backward(k, bytes(T.fsdp_logprob_bwd(dlogprob=P)), None) == OK


# ---------------------------------------------------------------------------
# AdamW over many tensors
# ---------------------------------------------------------------------------
def tensor(**kw):
    return T.fsdp_adam_tensor(**{**dict(numel=100, param=P, grad=P, exp_avg=P, exp_avg_sq=P, param_bf16=P, group=0), **kw})


def group(**kw):
    return B.fsdp_adamw_cfg(**{**dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step=1), **kw})


def adam(lib, tensors=None, groups=None, **kw):
    tensors = [tensor()] if tensors is None else tensors
    groups = [group()] if groups is None else groups
    t, g = (T.fsdp_adam_tensor * max(1, len(tensors)))(*tensors), (B.fsdp_adamw_cfg * max(1, len(groups)))(*groups)
    head = T.fsdp_adam_list(**{**dict(n_tensors=len(tensors), n_groups=len(groups), state_format=1, grad_dtype=2, seed=0), **kw})
    return lib.fsdp_adam_tensors(bytes(head), ctypes.addressof(t), bytes(g), None)


@pytest.mark.parametrize("kw,want", [(dict(n_tensors=-1), RANGE), (dict(n_groups=0), RANGE), (dict(n_groups=17), RANGE), (dict(state_format=0), RANGE),
                                     (dict(state_format=3), RANGE), (dict(grad_dtype=0), RANGE), (dict(grad_dtype=3), RANGE),
                                     (dict(grad_scale=P + 2), ALIGN), (dict(skip=P + 2), ALIGN)])
def test_adam_list(lib, kw, want):
    assert adam(lib, **kw) == want and B.fsdp_last_error()


@pytest.mark.parametrize("kw,want", [(dict(numel=-1), RANGE), (dict(numel=(1 << 40) + 1), OVERFLOW), (dict(group=-1), RANGE), (dict(group=1), RANGE),
                                     (dict(param=0), ARG), (dict(grad=0), ARG), (dict(exp_avg=0), ARG), (dict(exp_avg_sq=0), ARG),
                                     (dict(param=P + 2), ALIGN), (dict(grad=P + 2), ALIGN), (dict(exp_avg=P + 2), ALIGN),
                                     (dict(exp_avg_sq=P + 1), ALIGN), (dict(param_bf16=P + 1), ALIGN)])
def test_adam_tensor(lib, kw, want):
    assert adam(lib, [tensor(numel=0), tensor(**kw)]) == want


@pytest.mark.parametrize("kw", [dict(step=0), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=float("nan")), dict(lr=float("inf")),
                                dict(eps=-1.0), dict(eps=float("nan")), dict(weight_decay=float("inf"))])
def test_adam_group(lib, kw):
    assert adam(lib, groups=[group(), group(**kw)]) == RANGE


def test_adam_missing_arguments_and_nothing_to_do(lib):
    head = bytes(T.fsdp_adam_list(n_tensors=1, n_groups=1, state_format=1, grad_dtype=2))
    g, t = bytes(group()), tensor()
    assert lib.fsdp_adam_tensors(None, ctypes.addressof(t), g, None) == ARG
    assert lib.fsdp_adam_tensors(head, None, g, None) == ARG
    assert lib.fsdp_adam_tensors(head, ctypes.addressof(t), None, None) == ARG
    assert adam(lib, []) == OK
    assert adam(lib, [T.fsdp_adam_tensor()] * 3) == OK


def test_adam_state_bytes(lib):
    n = ctypes.c_int64()
    for k, want in ((0, 0), (1, 17), (16, 17), (17, 33), (32, 33), (33, 50), (1000, 1008 + 32)):
        assert T.fsdp_adam_state_bytes(k) == want == R.state_bytes(k)
    assert lib.fsdp_adam_state_bytes(-1, ctypes.byref(n)) == RANGE
    assert lib.fsdp_adam_state_bytes((1 << 40) + 1, ctypes.byref(n)) == OVERFLOW
    assert lib.fsdp_adam_state_bytes(5, None) == ARG


def convert(lib, a=None, b=None, n=1, f=1, to=2, step=1):
    a, b = tensor() if a is None else a, tensor() if b is None else b
    return lib.fsdp_adam_convert(n, ctypes.addressof(a) if a else None, f, ctypes.addressof(b) if b else None, to, 0, step, None)


def test_adam_convert(lib):
    for f, to in ((1, 1), (2, 2), (3, 3), (1, 3), (3, 1), (0, 2), (2, 4)):
        assert convert(lib, f=f, to=to) == RANGE
    assert convert(lib, n=-1) == RANGE and convert(lib, step=0) == RANGE
    assert convert(lib, a=False) == ARG and convert(lib, b=False) == ARG
    assert convert(lib, b=tensor(numel=101)) == RANGE
    assert convert(lib, a=tensor(exp_avg=P + 2)) == ALIGN
    assert convert(lib, a=tensor(exp_avg_sq=P + 1), f=3) == ALIGN
    assert convert(lib, b=tensor(exp_avg_sq=0)) == ARG
    assert convert(lib, n=0, a=False, b=False) == OK
    assert convert(lib, a=T.fsdp_adam_tensor(), b=T.fsdp_adam_tensor()) == OK


def test_the_binding_takes_gpu_tensors_only(lib):
    x = torch.zeros(4, 8)
    v, tok = torch.zeros(4), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="GPU"):
        T.fsdp_logprob_forward(x, tok, v, v, v)
    with pytest.raises(ValueError, match="GPU"):
        T.fsdp_logprob_backward(x, tok, v, v, v, x)
    with pytest.raises(TypeError):
        T.fsdp_logprob_forward([1.0], tok, v, v, v)
    q = torch.zeros(2, 3, 4, 8)
    with pytest.raises(ValueError, match="GPU"):
        T.fsdp_rotary_forward(q, q, torch.zeros(4, dtype=torch.float64))
    with pytest.raises(TypeError):
        T.fsdp_rotary_forward(q.double(), q.double(), torch.zeros(4, dtype=torch.float64))
    with pytest.raises(ValueError, match="GPU"):
        T.AdamTensors([v], [v], [v], [v])
    with pytest.raises(ValueError, match="states"):
        T.AdamTensors([v], [v], [v], [v], states="16bit")
    with pytest.raises(TypeError):
        T.AdamTensors(None, None, [v], [v], states="8bit")
    with pytest.raises(TypeError):
        T.AdamTensors([v], None, [v], [v])
    with pytest.raises(TypeError):
        T.fsdp_adam_tensors([v], dict(lr=1.0, step=1))


def test_random_numbers_are_spread():
    """Every bit of the 16-bit numbers is set half of the time, within and between tensors and steps, and
    neighbours do not follow one another: counts of n trials within 5 standard deviations (fixed seeds)."""
    n = 1 << 16
    for k in (R.key(0, 1, 0), R.key(0, 1, 1), R.key(0, 2, 0), R.key(7, 1, 0)):
        for r in R.random16(n, k):
            for bit in range(16):
                b = r >> bit & 1
                assert abs(b.sum() - n / 2) < 5 * n ** 0.5 / 2
                assert abs((b[1:] ^ b[:-1]).sum() - n / 2) < 5 * n ** 0.5 / 2
            assert np.bincount(r >> 8, minlength=256).std() < 1.3 * (n / 256) ** 0.5
    a, b = R.random16(n, R.key(0, 1, 0))
    c, d = R.random16(n, R.key(0, 2, 0))
    for x, y in ((a, b), (a, c), (b, d)):
        assert abs(np.corrcoef(x, y)[0, 1]) < 5 / n ** 0.5


# ---------------------------------------------------------------------------
# ends of the ranges
# ---------------------------------------------------------------------------
def test_logprob_scale_whose_product_with_log2_e_overflows(lib):
    big = float(np.float32(3e38))
    for f in (lp_fwd, lp_bwd):
        assert f(lib, dict(scale=big)) == RANGE
        assert f(lib, dict(scale=2.0 ** 127, rows=0)) == OK
        assert f(lib, dict(scale=2.0 ** -149, rows=0)) == OK


def test_rotary_positions_from_start_stay_in_int64(lib):
    last = (1 << 63) - 1
    for f in ("fsdp_rotary_forward", "fsdp_rotary_backward"):
        assert rotary(lib, dict(start=last - 6), dict(positions=None), f=f) == OVERFLOW   # 8 tokens
        assert rotary(lib, dict(start=last - 6, tokens=0), f=f) == OK


def test_an_empty_list_of_tensors_is_checked(lib):
    t = T.AdamTensors([], [], [], [])
    T.fsdp_adam_tensors(t, dict(lr=1e-3, step=1))
    with pytest.raises(B.FsdpError, match="step"):
        T.fsdp_adam_tensors(t, dict(lr=1e-3, step=0))
    with pytest.raises(B.FsdpError, match="n_groups"):
        T.fsdp_adam_tensors(t, [])
    with pytest.raises(TypeError, match="positional|unexpected|missing"):
        T.fsdp_adam_tensors(t, dict(lr=1e-3))


@pytest.mark.parametrize("name", ["param", "grad", "exp_avg", "exp_avg_sq", "param_bf16"])
def test_adam_addresses_have_48_bits(lib, name):
    assert adam(lib, [tensor(**{name: 1 << 48})]) == RANGE


def test_the_profile_was_taken_on_the_current_sources():
    import hashlib
    import re
    from conftest import ROOT
    with open(os.path.join(ROOT, "profiles", "train_ops_gpt2l_block.md")) as f:
        given = dict(re.findall(r"^(\S+\.hip) sha256: `([0-9a-f]{64})`", f.read(), re.M))
    assert set(given) >= {"rotary.hip", "logprob.hip", "adam_tensors.hip"}
    for name, h in given.items():
        with open(os.path.join(ROOT, "sharded_fsdp_flatten_amd", "csrc", name), "rb") as f:
            assert hashlib.sha256(f.read()).hexdigest() == h, name
