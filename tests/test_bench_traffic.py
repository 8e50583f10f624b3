"""The committed DRAM-traffic summaries that the benchmark's roofline line reports:
they are of the kernels as they stand, and cover all the sources that those are
made of."""
import os
import re

import pytest

import bench
import workloads


def _included(path):
    """The headers of this repository that a source includes, by way of others too."""
    found, todo = set(), [path]
    while todo:
        p = todo.pop()
        if p in found:
            continue
        found.add(p)
        with open(os.path.join(bench.ROOT, p)) as f:
            todo += [os.path.dirname(p) + "/" + h for h in re.findall(r'#include "([^"]+[.]cuh)"', f.read())]
    return found


@pytest.mark.parametrize("name", sorted(bench.TRAFFIC_FILES))
def test_a_summary_covers_all_sources_of_its_kernel(name):
    sources = bench.TRAFFIC_FILES[name][1]
    assert _included(sources[0]) == set(sources)


@pytest.mark.parametrize("name", sorted(bench.TRAFFIC_FILES))
def test_a_summary_is_of_the_kernel_as_it_stands(name):
    wl = workloads.WORKLOADS[name]
    traffic, need = bench.profiled_traffic(wl), bench.algorithmic_bytes(wl)
    assert traffic is not None, "captured on other sources: capture it again (the command stands in the file)"
    assert 0.98 * need <= traffic < 1.1 * need       # (a little of what is written may stay in L2)
