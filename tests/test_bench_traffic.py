"""The bench's DRAM traffic figures: each is tied to the sources of the kernel that it was captured on."""
import os
import re

import pytest

import bench

CSRC = os.path.join(bench.ROOT, "weight_only_int4_fp32_b200", "csrc")


def included(name, seen=()):
    """`name` and every header of this directory that it includes, directly or through another."""
    with open(os.path.join(CSRC, name)) as f:
        heads = [h for h in re.findall(r'#include "([^"]+)"', f.read()) if os.path.exists(os.path.join(CSRC, h))]
    out = {name, *seen}
    for h in heads:
        if h not in out:
            out |= included(h, out)
    return out


@pytest.mark.parametrize("workload", sorted(bench.TRAFFIC))
def test_the_hashed_sources_are_all_that_the_kernel_includes(workload):
    sources = bench.TRAFFIC[workload]["sources"]
    need = set().union(*(included(n) for n in sources))
    assert need == set(sources)


@pytest.mark.parametrize("workload", sorted(bench.TRAFFIC))
def test_a_figure_is_given_only_for_the_sources_it_was_captured_on(workload, monkeypatch):
    t = bench.TRAFFIC[workload]
    now = bench.kernel_sources_sha(t["sources"])
    monkeypatch.setitem(bench.TRAFFIC, workload, {**t, "sha256": now})
    assert bench.traffic_for(workload) == t["bytes"]
    monkeypatch.setitem(bench.TRAFFIC, workload, {**t, "sha256": "0" * 64})
    assert bench.traffic_for(workload) is None
