"""What the bench prints (CPU)."""
import json

import bench


def test_one_short_line(capfd):
    """One JSON line on standard output with the headline and what explains it; the long records on standard error, none lost."""
    short = {"metric": "m", "value": 1.5, "e2e": {"value": 1.25}, "clocks": {"sm_mhz": 2070}, "gamma_sweep": None}
    long = {k: {"x": [0.123456789] * 400} for k in bench.LONG}
    bench.emit({**short, **long})
    out, err = capfd.readouterr()
    assert out.count("\n") == 1 and out.endswith("\n") and len(out) < 1000
    assert json.loads(out) == short
    got = {}
    for line in err.strip().split("\n"):
        got.update(json.loads(line))
    assert got == long


def test_a_result_without_them(capfd):
    bench.emit({"impl": "reference", "value": 2.0, "workloads": None})
    out, err = capfd.readouterr()
    assert json.loads(out) == {"impl": "reference", "value": 2.0} and err == ""
