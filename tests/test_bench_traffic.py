"""The DRAM-traffic captures that the benchmark reports belong to the kernels'
present sources."""
import json

import pytest

from tests.test_bench_model import _bench


def _captures():
    with open(_bench().TRAFFIC_FILE) as f:
        return {k: e for k, e in json.load(f).items() if isinstance(e, dict)}


@pytest.mark.parametrize("workload", sorted(_captures()))
def test_capture_is_of_the_present_sources(workload):
    bench = _bench()
    value, note = bench.traffic_entry(_captures()[workload]["kernel"], workload)
    assert note is None and value > 0
