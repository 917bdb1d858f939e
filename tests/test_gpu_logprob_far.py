"""Token log probabilities of fp32 logits about as large as the kernels' exponents are held, scale x log2 e near
2^24 (x near 1.16e7 at a scale of 1) on either side of 0: maxima of lanes, waves, runs and rows just below that,
just above, and both in one row.  Against the 64-bit reference and its bounds (train_ref.py)."""
import numpy as np
import pytest
import torch

from test_gpu_logprob import check_forward

pytestmark = pytest.mark.gpu

EDGE = 2.0 ** 24 / np.log2(np.e)   # 11629079.9..., where neighbouring binary32 numbers are 1 apart


def rows_around(cols, sign, scale, seed):
    """Rows whose logits, times scale, lie within a few units of the edge."""
    g = np.random.Generator(np.random.PCG64(seed))
    j = np.arange(cols)
    near = lambda d: sign * (EDGE + d) / scale  # noqa: E731
    rows = [np.where(j < cols // 2, near(10), near(-1)),                    # halves on the two sides
            np.where(j < cols // 2, near(-1), near(10)),
            np.where(j % 2 == 0, near(4), near(-4)),                        # neighbours
            np.where(j // 64 % 2 == 0, near(3), near(0)),
            np.where(j == cols * 2 // 3, near(-1), near(6)),                # one logit on its own side
            np.where(j == cols // 3, near(8), near(-3)),
            near(g.integers(-20, 20, cols)),
            near(g.integers(1, 30, cols)),                                  # all beyond it
            near(-g.integers(1, 30, cols)),                                 # all short of it
            # waves (of 64 vectors of 4) on their own side, their lanes' maxima apart
            np.where(j // 256 % 4 == 0, near(-1), near(1 + j // 4 % 4)),
            np.where(j // 256 % 16 == 3, near(-1), near(1 + j // 4 % 4)),
            near(g.integers(-3, 4, cols) * 400),                            # most too far below the maximum to count
            np.where(j % 5 == 0, -np.inf, near(g.integers(-6, 6, cols))),   # with masks
            np.where(j % 7 == 0, np.finfo(np.float32).min, near(g.integers(-6, 6, cols)))]
    return torch.from_numpy(np.stack(rows).astype(np.float32))


@pytest.mark.parametrize("scale", [1.0, 0.75, 1e6])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("cols", [5, 64, 2000, 5003, 33001, 70003, 131072, 262147])
def test_either_side_of_the_largest_exponent(cols, sign, scale):
    # the lowest masks times a scale above 1 are -infinity in binary32: such a product is a mask as well
    x = rows_around(cols, sign, scale, cols)
    g = torch.Generator().manual_seed(cols)
    tok = torch.randint(0, cols, (len(x),), generator=g)
    top = min(cols, 5)
    check_forward(x, tok, scale, top)
    check_forward(x, tok, scale, 0, cols + 3, 1)
    check_forward(x[[0, 2, 6]], tok[:3], scale, top)


@pytest.mark.parametrize("scale", [1.0, 1e6])
@pytest.mark.parametrize("sign", [1, -1])
def test_many_rows(sign, scale):
    """As many rows as take the kernels of full launches (512 workgroups and more), of lengths of each."""
    for cols, rows in ((700, 600), (6000, 600), (17000, 520)):
        x = rows_around(cols, sign, scale, rows).repeat(rows // 14 + 1, 1)[:rows]
        check_forward(x, torch.arange(rows) % cols, scale)
