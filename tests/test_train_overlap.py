"""Conversions of AdamW states refuse buffers that overlap: on the host before any HIP call (the addresses given are
never read), and through the binding, where buffers that only touch, or are read twice, are converted."""
import ctypes
import os

import pytest
import torch

import train_ref as R
from sharded_fsdp_flatten_amd import binding as B
from sharded_fsdp_flatten_amd import train as T

RANGE = 2
P = 0x7F0000000000
F32, SMALL, BF16 = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from sharded_fsdp_flatten_amd import build
        build.build()
    return T._lib()


def state(m, v, n=100):
    return T.fsdp_adam_tensor(numel=n, exp_avg=P + m, exp_avg_sq=P + v)


def convert(lib, a, b, f, to):
    n = len(a)
    one, two = (T.fsdp_adam_tensor * n)(*a), (T.fsdp_adam_tensor * n)(*b)
    return lib.fsdp_adam_convert(n, ctypes.addressof(one), f, ctypes.addressof(two), to, 0, 1, None)


# 100 elements: 400 bytes in 32 bits, 200 in bf16, 112 + 4 in 8 bits
@pytest.mark.parametrize("a,b,f,to", [
    ([state(0, 400)], [state(0, 4096)], F32, SMALL),                                # in place
    ([state(0, 400)], [state(4096, 796)], F32, SMALL),                              # the last element
    ([state(4096, 8192)], [state(0, 115)], F32, SMALL),                             # the state with its own other half: its last scale
    ([state(4096, 8192)], [state(0, 396)], SMALL, F32),
    ([state(4096, 8192)], [state(4096 + 114, 0)], SMALL, BF16),                     # the last two scales
    ([state(4096, 8192)], [state(4096 - 198, 0)], SMALL, BF16),
    ([state(4096, 8192), state(0, 400)], [state(16384, 20480), state(24576, 398)], BF16, SMALL),    # another tensor's
    ([state(4096, 8192)] * 3, [state(30000, 20000), state(10000, 40000), state(50000, 30100)], SMALL, F32),   # written twice
    ([state(100, 2000)], [state(0, 100000)], SMALL, F32),                           # inside the longer values
    ([state(0, 100000, 5000)], [state(19996, 200000, 5000)], F32, SMALL)])
def test_overlapping_buffers(lib, a, b, f, to):
    assert convert(lib, a, b, f, to) == RANGE
    assert "overlaps" in B.fsdp_last_error()


@pytest.mark.gpu
def test_through_the_binding():
    n = 100
    held = T.fsdp_adam_state_bytes(n)
    base = torch.zeros(8192, dtype=torch.uint8, device="cuda")
    full = [torch.arange(n, dtype=torch.float32, device="cuda") / 8, torch.full((n,), 2.5, device="cuda")]
    p = torch.zeros(n, device="cuda")
    src = T.AdamTensors(None, None, *([x] for x in full))
    small = T.AdamTensors([p], [p], [base[:held]], [base[held:2 * held]], states="8bit")     # they touch
    T.fsdp_adam_convert(src, small)
    got = [R.read_state(x.cpu().numpy(), n, k) for x, k in ((base[:held], "m"), (base[held:2 * held], "v"))]
    assert abs(got[0] - full[0].cpu().numpy()).max() <= 1.0 and (abs(got[1] - 2.5) <= 0.25).all()
    # values into the memory around the state, then into the state itself
    at = -(-2 * held // 4) * 4
    out = [base[at:at + 4 * n].view(torch.float32), base[at + 4 * n:at + 8 * n].view(torch.float32)]
    T.fsdp_adam_convert(small, T.AdamTensors(None, None, [out[0]], [out[1]]))
    for x, want in zip(out, got):
        assert (x.double().cpu().numpy() == want).all()
    before = base.clone()
    over = base[at - 4:at - 4 + 4 * n].view(torch.float32)
    with pytest.raises(B.FsdpError, match="overlaps"):
        T.fsdp_adam_convert(small, T.AdamTensors(None, None, [over], [out[1]]))
    with pytest.raises(B.FsdpError, match="overlaps"):
        T.fsdp_adam_convert(T.AdamTensors(None, None, [over], [out[1]]), small)
    assert torch.equal(base, before)
    # one state's values read into two places
    twice = T.AdamTensors([p, p], [p, p], [base[:held]] * 2, [base[held:2 * held]] * 2, states="8bit")
    outs = [torch.empty(n, device="cuda") for _ in range(4)]
    T.fsdp_adam_convert(twice, T.AdamTensors(None, None, outs[:2], outs[2:]))
    assert all((x.double().cpu().numpy() == want).all() for x, want in zip(outs, (got[0], got[0], got[1], got[1])))
