"""The 8-bit states' rounding as the reference defines it (the GPU's is the same bit for bit): its mean over all random
numbers."""
import numpy as np

import train_ref as R


def test_mean_over_all_random_numbers():
    """Low by 0 to 2^-16 of the codes' distance, 2^-17 on average, for m and v, where codes are normal and where not."""
    g = np.random.Generator(np.random.PCG64(3))
    lacks = []
    for which, top, small in (("m", 448.0, 2.0 ** -9), ("v", 61440.0, 2.0 ** -17)):
        for size in (1.0, 0.01, small * 3.3):
            x = np.float32(size * (1 + g.random()))
            n = 1 << 16
            # pairs in groups of their own: the value, and one that sets the scale to 1
            both = np.zeros((n, 32), np.float32)
            both[:, 0], both[:, 1] = x, top
            r = np.zeros((n, 32), np.int64)
            r[:, 0] = np.arange(n)
            buf = R.write_state(both.ravel(), r.ravel(), which)
            got = R.read_state(buf, 32 * n, which).reshape(n, 32)[:, 0]
            low, high = got.min(), got.max()
            assert low <= x <= high
            gap = high - low
            lack = (x - got.mean()) / gap if gap else 0.0
            assert 0 <= lack < 2.0 ** -16
            lacks.append(lack)
    assert 2.0 ** -18 < np.mean(lacks) < 2.0 ** -16
