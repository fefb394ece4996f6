"""Who issues the tensor-core and tile-copy instructions: never a lane picked by its
number, only one that elect.sync picked (read from the sources, no GPU)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "fine_tuning_gb300", "csrc")
ISSUES = re.compile(r"\b(umma_\w+|mma_\w+|tma_load_2d|tma_prefetch_2d|load_tile|load_box)\s*[<(]")


def guarded(text, test):
    """The statements under every `if` whose condition matches `test`."""
    for m in re.finditer(r"\bif \(", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[i], 0)
            i += 1
        if not test.search(text[m.end():i - 1]):
            continue
        rest = text[i:].lstrip()
        if not rest.startswith("{"):
            yield rest[:rest.index(";") + 1]
            continue
        depth = 0
        for j, c in enumerate(rest):
            depth += {"{": 1, "}": -1}.get(c, 0)
            if depth == 0:
                yield rest[:j]
                break


FILES = [f for f in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))) if "tcgen05" in open(f).read()]


@pytest.mark.parametrize("name", [os.path.basename(f) for f in FILES])
def test_no_issue_under_a_test_of_the_lane_number(name):
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    for body in guarded(text, re.compile(r"\blane == 0\b|threadIdx\.x == 0\b")):
        found = ISSUES.search(body)
        assert not found, f"{name}: {found.group(0)} under a test of the lane number"


def test_the_elections_are_seen():
    """The scan finds the guarded issues it is meant for."""
    text = open(os.path.join(CSRC, "tc_gemm.cuh")).read()
    bodies = list(guarded(text, re.compile(r"\belect_one\(\)")))
    assert sum(bool(ISSUES.search(b)) for b in bodies) == 2
