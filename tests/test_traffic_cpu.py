"""The DRAM figures that the benchmark's line reports are of the sources as they are."""

import os

import pytest

import bench

LINES = [x.split() for x in open(os.path.join(bench.ROOT, "profiles", "traffic.txt"))
         if x.strip() and not x.startswith("#")]


@pytest.mark.parametrize("line", LINES, ids=lambda x: x[0])
def test_figures_are_of_these_sources(line):
    """A change to a timed kernel or to what it includes needs its capture again (the commands are at
    the file's top); what only other operators use stands in headers of theirs."""
    kernel, workload, figure, sources = line
    assert bench.source_hash(kernel) == sources
    assert bench.workload_traffic(workload)[kernel] == int(figure)


def test_every_timed_kernel_has_a_figure():
    assert {x[0].split("<")[0] for x in LINES} == set(bench.KERNEL_SOURCES)
