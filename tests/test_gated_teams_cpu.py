"""How many warps and CTAs walk a row of the gated recurrence: the rule's bounds, and that the sizes of
the GPU tests reach what they are meant to."""
import pytest

from selective_state_space_56_b200 import build as s6build
from selective_state_space_56_b200 import ops
from tests.test_gated_teams_gpu import CASES


@pytest.fixture(scope="module", autouse=True)
def built():
    s6build.build()


@pytest.mark.parametrize("backward", [False, True])
def test_bounds(backward):
    for rows in (1, 2, 3, 20, 75, 148, 149, 300, 700, 1184, 1185, 2400, 100000):
        for L in (0, 1, 249, 250, 513, 5003, 33001, 524287):
            warps, ctas = ops.diag_gated_team(1, rows, L, backward)
            chunks = max(1, (L + 7 + 255) // 256)
            assert 1 <= warps <= 8 and 1 <= ctas <= 16 and warps <= chunks
            assert ctas == 1 or warps == 8  # a cluster of whole CTAs
            assert (ctas - 1) * warps < chunks  # no CTA without a chunk
            if rows > 8 * 148:
                assert (warps, ctas) == (1, 1)
            if ctas > 1:  # all rows at once
                assert rows * ctas * warps <= 148 * (16 if backward else 32)


def test_refusals():
    for dims in ((0, 3, 8), (2, 0, 8), (2, 3, -1)):
        with pytest.raises(ops.MambaError):
            ops.diag_gated_team(*dims)


def test_the_gpu_cases_reach_every_kind_of_cluster():
    forward = {ops.diag_gated_team(1, rows, L)[1] for rows, L in CASES}
    backward = {ops.diag_gated_team(1, rows, L, True)[1] for rows, L in CASES}
    assert {1, 4, 9, 14, 16} <= forward and {1, 4, 7, 11, 16} <= backward
