"""The benchmark's line on stdout stays short enough to be read from the end of a log: the figures of the other
workloads go to stderr."""

import json

import bench


def test_one_short_line(capsys):
    figures = {"GB/s": 1 / 3, "us": 2 / 3, "frac_of_peak": 1 / 7, "launches": 1, "steady_us": 1 / 9}
    line = {"metric": bench.METRIC, "value": 6400.123456789, "config": {"workload": bench.WORKLOAD},
            "workloads": {f"workload {i}": figures for i in range(100)}}
    bench.emit(line)
    out, err = capsys.readouterr()
    assert len(out.splitlines()) == 1 and len(out) < 1000
    got = json.loads(out)
    assert got == {k: v for k, v in line.items() if k != "workloads"}
    assert json.loads(err) == {"workloads": line["workloads"]}
    assert "workloads" in line


def test_a_line_without_workloads_is_alone(capsys):
    bench.emit({"value": 1})
    assert capsys.readouterr() == ('{"value": 1}\n', "")
