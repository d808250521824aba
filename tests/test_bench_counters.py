"""The kept traffic counters are reported while the kernels are the ones they were taken on:
the sources that decide that are all that the measured kernels are built from."""
import json
import os
import re
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import bench  # noqa: E402

CSRC = os.path.join(ROOT, "float8_quantization_moe_amd", "csrc")


def included(name, seen=()):
    """`name` and the device headers it includes, theirs too (internal.hpp declares host functions only)."""
    names = {name}
    for h in re.findall(r'#include "(\w+\.hpp)"', open(os.path.join(CSRC, name)).read()):
        if h != "internal.hpp" and h not in names and h not in seen:
            names |= included(h, tuple(names) + tuple(seen))
    return names


def test_every_source_of_the_measured_kernels_counts():
    kernels = [f for f in bench.COUNTER_SOURCES if f.endswith(".hip")]
    assert set().union(*(included(f) for f in kernels)) == set(bench.COUNTER_SOURCES)


def test_the_kept_counters_name_these_sources():
    kept = json.load(open(bench.TRAFFIC_FILE))
    assert kept["source_files"] == bench.COUNTER_SOURCES
    assert len({k["source_sha256"] for k in kept["kernels"].values()}) == 1
