"""The norms' backward pass with infinities in its rows, and the norms at every shape that their kernels
are made for, against the plain 64-bit reference (layer_ref.py)."""
import gc

import numpy as np
import pytest
import torch

import layer_ref as R
import sharded_fsdp_flatten_amd as F
from gpu_util import dev
from test_gpu_layer import EPS, Guarded, T, close, f64, given_stats, norm_inputs, normal, run_backward, stats

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


# ---------------------------------------------------------------------------
# every shape of the kernels over rows in registers
# ---------------------------------------------------------------------------
# Widths that fill a shape's last vector, end inside it, and lie at the shapes' ends.
WIDTHS = [8, 100, 203, 256, 512, 507, 520, 765, 768, 1000, 1021, 1024, 1030, 1533, 1536, 1540, 1600, 2045, 2048, 2051, 2504, 2501,
          4000, 4093, 4096, 4104, 6141, 6144, 6152, 8189, 8192, 8200, 9003, 10240, 10243, 12280, 12285, 12289, 14336, 16381, 16384]


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("cols", WIDTHS)
def test_norm_forward_shapes(cols, t):
    """Four rows and one more (a wave's rows share a workgroup), plain, and with residual, sum and
    checkpoint; parameters of either type."""
    rows = 5
    x, w, b = norm_inputs(cols, rows, cols, t, t)
    res = normal(9, rows, cols).to(T[t]).to(dev())
    for kind, pt, residual in (("layer", "bf16", None), ("rms", "f32", res), ("layer", "f32", res), ("rms", "bf16", None)):
        w2, b2 = w.to(T[pt]), b.to(T[pt])
        y, s = Guarded(rows, cols, T[t]), Guarded(rows, cols, T[t])
        mean, rstd = stats(rows)
        q = F.Ckpt.empty(rows, cols, "e4m3" if kind == "layer" else "int8", device=dev())
        F.fsdp_norm_forward(x, w2, b2, y.t, mean, rstd, kind=kind, eps=EPS, residual=residual, ckpt=q,
                            sum=None if residual is None else s.t)
        held = x if residual is None else (x.float() + residual.float()).to(T[t])
        assert residual is None or torch.equal(s.t, held)
        r = R.norm(f64(held), f64(w2), f64(b2), kind, EPS, t)
        close(y.t, r["y"], r["ey"], "y")
        close(rstd, r["rstd"], r["erstd"], "rstd")
        assert kind == "rms" or close(mean, r["mean"], r["emean"], "mean") is None
        assert y.around_is_untouched() and s.around_is_untouched()
        back = torch.empty_like(x)
        F.fsdp_ckpt_unpack(q, back)
        assert np.array_equal(f64(back), R.ckpt(f64(held), q.format)[0])


def threads_of_a_row(cols):
    """Threads and vectors that the backward pass gives a row."""
    nq = -(-cols // 4)
    if nq <= 64:
        return 64, 1
    threads = 64
    while threads < 1024 and nq > 3 * threads:
        threads *= 2
    return threads, -(-nq // threads)


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("cols", WIDTHS)
def test_norm_backward_shapes(cols, t):
    """From the tensor and both checkpoints, with and without a residual gradient, with the output again and
    without; more rows than workgroups, so that some take two rows and some three."""
    rows = 150 * max(1, 512 // threads_of_a_row(cols)[0]) + 3
    x, w, b = norm_inputs(cols, rows, cols, t, t)
    dy = normal(50, rows, cols, scale=0.1).to(T[t]).to(dev())
    dres = normal(51, rows, cols, scale=0.1).to(T[t]).to(dev())
    for i, (src, res, again) in enumerate((("tensor", None, False), ("tensor", dres, True), ("e4m3", None, True),
                                           ("e4m3", dres, False), ("int8", None, False), ("int8", dres, True))):
        kind = ("layer", "rms")[i // 2 % 2]
        mean, rstd = given_stats(x, kind)
        held, source = f64(x), x
        if src != "tensor":
            source = F.Ckpt.empty(rows, cols, src, device=dev())
            F.fsdp_ckpt_pack(x, source)
            back = torch.empty_like(x)
            F.fsdp_ckpt_unpack(source, back)
            held = f64(back)
        dx, dw, db, y = run_backward(dy, source, w, mean, rstd, kind, t, dres=res, b=b if again else None, again=again)
        r = R.norm_grads(f64(dy), held, f64(w), f64(b) if again else None, f64(mean), f64(rstd), kind, t,
                         None if res is None else f64(res))
        close(dx, r["dx"], r["edx"], "dx")
        close(dw, r["dw"], r["edw"], "dw")
        close(db, r["db"], r["edb"], "db")
        if again:
            close(y, r["y"], r["ey"], "y")
