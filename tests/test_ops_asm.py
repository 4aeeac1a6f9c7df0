"""Copies, barriers and waits written as inline PTX carry a "memory" clobber: without
one the compiler may move an ordinary load of shared memory across them, since
`asm volatile` alone is ordered with other volatile accesses only."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_delta_rule_varlen_gb300", "csrc")
ORDERING = re.compile(r"cp\.async|mbarrier\.|griddepcontrol|barrier\.cluster|\bbar\.(sync|red)|fence\.|tcgen05\.(commit|wait|fence)")


def statements(text):
    """The texts of the asm statements, whole."""
    text = re.sub(r"//[^\n]*", "", text)
    for m in re.finditer(r"\basm\s*(volatile)?\s*\(", text):
        depth, i, quoted = 1, m.end(), False
        while depth:
            c = text[i]
            if c == '"' and text[i - 1] != "\\":
                quoted = not quoted
            elif not quoted:
                depth += (c == "(") - (c == ")")
            i += 1
        yield text[m.start():i]


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))),
                         ids=os.path.basename)
def test_ordering_statements_clobber_memory(path):
    with open(path) as f:
        found = [s for s in statements(f.read()) if ORDERING.search(s)]
    for s in found:
        assert '"memory"' in s and "volatile" in s, s


def test_the_helpers_are_seen():
    with open(os.path.join(CSRC, "gdr_common.cuh")) as f:
        text = f.read()
    ring = [s for s in statements(text) if "cp.async" in s]
    assert sum("wait_group" in s for s in ring) >= 1 and sum("commit_group" in s for s in ring) >= 1
