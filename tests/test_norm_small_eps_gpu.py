"""Norm to e4m3 where the row's factor 1 / sqrt(mean + eps) is large: rows of zeros (padding) and of
tiny values with an eps below 1e-12."""
import numpy as np
import pytest
import torch

from selective_state_space_56_b200 import ops
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dim", [128, 272, 2560])
@pytest.mark.parametrize("eps", [1e-6, 1e-12, 1e-20, 1e-30])
def test_rows_of_zeros_and_of_tiny_values(cuda_ok, eps, dim):
    g = torch.Generator().manual_seed(dim)
    x = torch.randn(6, dim, generator=g)
    x[1] = 0.0
    x[2] *= 1e-7
    x[3, :64] = 0.0
    # far below sqrt(eps): the squares vanish beside eps, so the outputs are x / sqrt(eps) weight
    x[4] *= 1e-16
    x[5] *= 1e-36
    w = 1 + 0.1 * torch.randn(dim, generator=g)
    w[64:128] = 0.0  # row 3's first group is zero without the row being zero
    q, s, _ = ops.add_rms_norm_fp8(x.to(DEV), w.to(DEV), eps=eps)
    q, s = q.float().double().cpu().numpy(), s.double().cpu().numpy()
    assert np.isfinite(q).all() and np.isfinite(s).all() and (s > 0).all()
    assert (q[1] == 0).all() and (q[3, :128] == 0).all()
    # The sum of squares passes up to 64 fp32 additions and the squares' underflow (below 2^-149 each)
    # changes it by less than 1e-42 against eps; the factor and the products add six roundings: 2^-18
    # relative in all.  An output lies within half a step of e4m3 (2^-4, or 2^-10 below 2^-6), scaled.
    out, _ = ref.rms_norm(x.double().numpy(), w.double().numpy(), float(np.float32(eps)))
    scale = s[:, np.arange(dim) // 128]
    half = np.maximum(np.abs(q) * 2.0 ** -4, 2.0 ** -10)
    ref.check(q * scale, out, half * scale + 2.0 ** -16 * np.abs(out) + 1e-33, "out")
