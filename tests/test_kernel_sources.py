"""Rules of the kernels' sources that no run can show (CPU)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "paged_kv_cache_476_b200", "csrc")
ISSUE = r"(mma_ss|mma_ts|tc_commit)\("


def _guards(text):
    """The condition of the `if` around every tcgen05 product and commit: the nearest one
    above that names a single thread."""
    found = []
    for m in re.finditer(ISSUE, text):
        before = text[:m.start()]
        who = [(before.rfind(g), g) for g in ("elect_one()", "lane == 0")]
        found.append((m.group(1), max(who)[1], before.count("\n") + 1))
    return found


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*.cu"))), ids=os.path.basename)
def test_products_and_commits_are_one_threads(path):
    """A commit covers the products of the thread that executes it, and which lane
    elect.sync picks is not said: a file issues both under the one or the other."""
    with open(path) as f:
        guards = _guards(f.read())
    assert len({g for _, g, _ in guards}) <= 1, [g for g in guards if g[1] == "lane == 0"]
