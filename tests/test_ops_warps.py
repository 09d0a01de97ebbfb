"""A bounded wait that runs out ends whole warps: what one lane sees, the time or the abort flag, has to decide for all 32
before the next warp-wide instruction.  Read from the sources, since no test makes these waits run out on a GPU."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "log_domain_sinkhorn_updates_b200", "csrc")


def _without_single_lane_blocks(text):
    """The code that whole warps run: blocks of `if (lane == 0)` and `if (lead)` are one lane's."""
    for guard in ("if (lane == 0) {", "if (lead) {"):
        while guard in text:
            start = text.index(guard)
            at, depth = start + len(guard), 1
            while depth:
                depth += {"{": 1, "}": -1}.get(text[at], 0)
                at += 1
            text = text[:start] + text[at:]
    return text


@pytest.mark.parametrize("name", ["fs_xattn_tc.cu", "fs_xattn_grad_tc.cu", "fs_xent_tc.cu"])
def test_a_warp_decides_together(name):
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    found = 0
    for statement in re.split(r"[;{}]", _without_single_lane_blocks(text)):
        statement = " ".join(statement.split())
        if statement == "const bool aborted = *abort_flag":  # counts as a read of the flag where it is used
            continue
        reads = re.findall(r"mbar_wait_\w+\(|\*abort_flag\b(?! = )|\baborted\b", statement)
        if not reads or "reinterpret_cast" in statement:
            continue
        if re.fullmatch(r"mbar_wait_\w+\(.*\)", statement):  # its result decides nothing
            continue
        found += 1
        assert "warp_all(" in statement and statement.index("warp_all(") < statement.index(reads[0]), statement
    assert found >= 3
