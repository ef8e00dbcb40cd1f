"""A CTA of a team that gave up a wait arrives at its barrier no more (its phase may be incomplete, and
a phase takes one arrival).  Checked on the source: the wait runs out only where a CTA of a running
cluster stands still for a second, which is nothing to bring about on a GPU."""
import os

from selective_state_space_56_b200 import build as s6build


def test_arrivals_and_hand_overs_end_with_the_wait_that_gave_up():
    text = open(os.path.join(s6build.CSRC, "gated_scan.cu")).read()
    body = text[text.index("float team_round("):]
    body = body[:body.index("\n}\n")]
    start = body.index("if (alive) {")
    indent = start - body.rindex("\n", 0, start) - 1
    block = body[start:body.index("\n" + " " * indent + "}", start)]
    for what in ("mbar_arrive_expect_tx(", "hand_over(", "mbar_wait_bounded("):
        assert body.count(what) == 1 and what in block, what
    assert "alive = false;" in block
