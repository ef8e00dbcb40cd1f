"""The norm's backward at widths that are not a multiple of 8, with more rows than CTAs (so that the next
row is on its way while one is computed), in every instance of that kernel: up to 4, 8 and 32 columns
a thread.  Bounds: tests/test_rms_norm_gpu.py."""
import numpy as np
import pytest

from selective_state_space_56_b200 import ops
from tests import layer_ref as ref
from tests.test_rms_norm_gpu import REL, n64, problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("types", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")], ids=str)
@pytest.mark.parametrize("rows,dim", [(1300, 101), (1300, 2047), (1300, 2049), (700, 3001), (700, 4095), (700, 4097),
                                      (700, 5001), (700, 9001), (320, 16383)])
def test_backward_of_odd_widths(cuda_ok, rows, dim, types):
    xt, rt = types
    p = problem(rows, dim, xt, rt, seed=dim)
    g = ops.add_rms_norm_bwd(p["dout"], p["residual"], p["weight"], p["dres"])
    d, v, w = n64(p["dout"]), n64(p["residual"]), n64(p["weight"])
    dv, dw = ref.rms_norm_backward(d, v, w, n64(p["dres"]), 1e-5)
    _, rstd = ref.rms_norm(v, w, 1e-5)
    xhat = v * rstd
    mag = rstd * (np.abs(d * w) + np.abs(xhat) * np.mean(np.abs(d * w * xhat), -1, keepdims=True))
    tol = 2 * REL * mag + 2 * ref.U * np.abs(dv)
    ref.check(n64(g["dx"]), dv, tol + ref.half_step(xt, dv), "dx")
    ref.check(n64(g["dresidual"]), dv, tol + ref.half_step(rt, dv), "dresidual")
    ref.check(n64(g["dweight"]), dw, (REL + (rows + 64) * ref.U) * np.abs(d * xhat).sum(0), "dweight")
