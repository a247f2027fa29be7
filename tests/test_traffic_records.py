"""The committed HBM traffic of the grouped GEMMs belongs to the sources as they are: bench.py reports no traffic
from a summary of other sources, so an edit of those has to take the summaries again."""
import os

import pytest

import bench
from workloads import configs

RECORDED = [n for n in sorted(configs.WORKLOADS) if os.path.exists(bench.pmc_summary_path(n))]


def test_the_headline_workload_has_a_record():
    assert len(RECORDED) >= 14 and "mixtral_t512" in RECORDED


@pytest.mark.parametrize("name", RECORDED)
def test_traffic_was_measured_on_these_sources(name):
    w = configs.WORKLOADS[name]
    traffic = bench.measured_traffic(name)
    assert traffic is not None, "take the FETCH_SIZE and WRITE_SIZE runs named in the summary again"
    # gate+up reads two weight matrices of each active expert, k of them at the least, once at the least
    size = {"f32": 4, "bf16": 2}[w.dtype] if w.weights == "dtype" else 1
    assert traffic >= 0.99 * 2 * w.d * w.F * size * min(w.k, w.E)
