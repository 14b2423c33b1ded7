"""The line that bench.py prints is short; the other workloads' figures are kept apart."""
import json

import bench


def test_the_line_is_the_headline():
    modes = {f"workload_{i}_exact": {"ms": 1.0, "rep_ms": [1.0] * 3, "context": "x" * 200} for i in range(40)}
    rows = [{"workload": f"w{i}", "GFLOP/s": 1.0} for i in range(28)]
    line = {"metric": "GFLOP/s", "value": 1.5, "cpu_baseline": {"value": 2.0, "per_workload": rows}, "modes": modes}
    short, details = bench.split_line(line)
    assert short == {"metric": "GFLOP/s", "value": 1.5, "cpu_baseline": {"value": 2.0}}
    assert details == {"modes": modes, "cpu_per_workload": rows}
    assert line["modes"] is modes and line["cpu_baseline"]["per_workload"] is rows  # the argument stays as it is
    assert json.loads(json.dumps(short)) == short


def test_a_line_without_other_workloads_stays():
    line = {"metric": "GFLOP/s", "value": 1.5, "cpu_baseline": {"value": 2.0}}
    assert bench.split_line(line) == (line, None)


def test_the_metrics_workloads_are_in_the_line():
    one = {"ms": 1.0, "GFLOP/s": 2.0, "roofline_frac": 0.5, "rep_ms": [1.0] * 3}
    line = {"metric": "GFLOP/s", "modes": {n: one for n in bench.IN_LINE + ("another",)}}
    short, details = bench.split_line(line)
    assert short["modes"] == {n: {"ms": 1.0, "GFLOP/s": 2.0, "roofline_frac": 0.5} for n in bench.IN_LINE}
    assert details["modes"] == line["modes"]
