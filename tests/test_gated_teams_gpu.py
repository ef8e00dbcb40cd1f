"""Rows of the gated recurrence walked by clusters of 4 to 16 CTAs, in both element types, forward and
backward, against the fp64 recurrence (bounds: tests/layer_ref.py)."""
import pytest

from tests.test_gated_scan_gpu import compare, problem

# (rows, L): clusters of (forward, backward) CTAs
CASES = [(25, 33001),  # 16, 11
         (40, 28700),  # 14, 7
         (60, 18500),  # 9, 4
         (120, 9001),  # 4, 2
         (4, 34000),   # 16, 16
         (400, 2100)]  # 1, 1: several warps of one CTA


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,L", CASES)
def test_clusters(cuda_ok, rows, L, dtype):
    z, decay = rows != 40, rows in (60, 4)
    compare(problem(1, rows, L, dtype, decay, z=z, seed=rows), dtype, decay, checkpoints=rows != 25)
