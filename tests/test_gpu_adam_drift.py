"""What 8-bit AdamW states settle at: rounded at random with odds of 16 bits, exp_avg_sq stays where 32 bits put it, but for
the part of the odds that is cut off, over all the steps that it remembers."""
import numpy as np
import pytest
import torch

import sharded_fsdp_flatten_amd as F
import train_ref as R
from gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("beta2", [0.99, 0.999, 0.9999])
def test_where_a_constant_gradient_settles(beta2):
    """A step keeps beta2 of what is missing and cuts off up to 2^-16 of the codes' distance, 2^-17 on average: the mean
    of many elements is low by up to 2^-16 / (1 - beta2) distances in the end, and not high; five standard deviations
    of a mean of values that stay within two distances, and three roundings of binary32 a step."""
    n, f = 1 << 16, np.float32
    g = f(1.3) ** f(0.5)
    b2, rest = float(f(beta2)), float(f(1 - beta2))
    want = rest * float(g) ** 2 / (1 - b2)
    gap = 0.125   # of codes between 1 and 2
    p, grad = torch.zeros(n, device=dev()), torch.full((n,), float(g), device=dev())
    m, v = (torch.zeros(F.fsdp_adam_state_bytes(n), dtype=torch.uint8, device=dev()) for _ in range(2))
    tensors = F.AdamTensors([p], [grad], [m], [v], states="8bit")
    first = [torch.full((n,), float(x), device=dev()) for x in (g, want)]
    F.fsdp_adam_convert(F.AdamTensors(None, None, *([x] for x in first)), tensors, seed=1)
    for step in range(1, int(6 / (1 - beta2))):
        F.fsdp_adam_tensors(tensors, dict(lr=0.0, betas=(0.9, beta2), step=step), seed=7)
    got = R.read_state(v.cpu().numpy(), n, "v")
    assert np.abs(got - want).max() < 12 * gap
    noise = 5 * got.std() / n ** 0.5 + 3 * R.U * want / (1 - beta2)
    assert got.std() < 2 * gap
    assert want - gap * 2.0 ** -16 / (1 - beta2) - noise <= got.mean() <= want + noise
