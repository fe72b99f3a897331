"""DRAM traffic records of the kernels: the bench reports one only while the sources that it was captured
on have not changed, so a change to them takes its record along or leaves a header alone."""
import importlib.util
import json
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
RECORDS = json.load(open(os.path.join(ROOT, "profiles", "traffic.json")))["records"]


@pytest.fixture(scope="module")
def bench():
    spec = importlib.util.spec_from_file_location("_q8_bench_records", os.path.join(ROOT, "bench.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("name", sorted(RECORDS))
def test_a_record_is_of_the_current_sources(bench, name):
    assert bench.recorded_traffic(name) == RECORDS[name]["dram_bytes_per_launch"]
