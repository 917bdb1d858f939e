"""The norms' backward pass with infinities in its rows, and the norms at every shape that their kernels
are made for, against the plain 64-bit reference (layer_ref.py)."""
import gc

import numpy as np
import pytest
import torch

import layer_ref as R
import sharded_fsdp_flatten_amd as F
from gpu_util import dev
from test_gpu_layer import T, close, f64, given_stats, norm_inputs, normal, run_backward

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _free():
    F.load()
    yield
    gc.collect()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [2, 40, 256, 700, 1280, 1283, 2500, 5003, 12288])
def test_norm_backward_infinities_are_those_of_the_formula(cols, t, kind):
    """An infinite gradient, or input, in a row's first or last column: infinities and NaN where the formula
    has them and nowhere else, whether or not the width leaves lanes idle, and no trace in other rows."""
    rows = 12
    x, w, _ = norm_inputs(cols, rows, cols, t, t)
    dy = normal(50, rows, cols, scale=0.1).to(T[t]).to(dev())
    mean, rstd = given_stats(x, kind)
    inf = float("inf")
    dy[1, 0], dy[3, cols - 1] = inf, -inf
    x[5, 0], x[7, cols - 1] = -inf, inf
    dx, dw, db, _ = run_backward(dy, x, w, mean, rstd, kind, t)
    with np.errstate(all="ignore"):
        r = R.norm_grads(f64(dy), f64(x), f64(w), None, f64(mean), f64(rstd), kind, t)
    for got, want, e, what in ((dx, r["dx"], r["edx"], "dx"), (dw, r["dw"], r["edw"], "dw"), (db, r["db"], r["edb"], "db")):
        finite = np.isfinite(want)
        assert np.array_equal(f64(got)[~finite], want[~finite], equal_nan=True), what
        close(got, want, np.where(finite, e, 0), what)
    fine = [i for i in range(rows) if i not in (1, 3, 5, 7)]
    assert torch.isfinite(dx[fine]).all()
