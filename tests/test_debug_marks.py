"""The debug build's index checks in the sources: every mark has a number of its own and can fail (no
condition that a template flag alone makes true), and every kernel file of the operators has marks."""
import glob
import os
import re

from recurrent_state_memory_b200 import build

MARK = re.compile(r"GDR_(?:AND_)?INB\(((?:[^()]|\((?:[^()]|\([^()]*\))*\))*),\s*(\d+)\)")


def _marks():
    found = []
    for path in sorted(glob.glob(os.path.join(build.CSRC, "*.cuh"))):
        found += [(os.path.basename(path), *m) for m in MARK.findall(open(path).read())]
    return found


def test_marks_have_numbers_of_their_own():
    sites = [site for _, _, site in _marks()]
    assert len(sites) > 40 and len(sites) == len(set(sites))


def test_marks_can_fail():
    for file, condition, site in _marks():
        first = condition.strip().lstrip("(").split("||")[0].split("&&")[0].strip()
        assert first not in ("SHIFT", "VEC", "FEW", "true", "1"), (file, site, condition)


def test_loads_stores_and_partial_sums_are_marked():
    count = {f: sum(1 for g, _, _ in _marks() if g == f) for f in ("norm.cuh", "beam.cuh", "scan.cuh")}
    assert count["norm.cuh"] >= 12 and count["beam.cuh"] >= 7 and count["scan.cuh"] >= 6
