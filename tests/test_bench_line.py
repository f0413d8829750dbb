"""The benchmark's line: what goes to stdout and what beside it."""
import json

import bench


def test_tables_and_notes_go_beside_the_line():
    line = {"metric": "m", "value": 2.5, "config": {"workload": "w"},
            "roofline": {"frac": 1.0, "bytes": "requested", "traffic_source": "file"},
            "e2e": {"value": 2.0, "h2d_bytes_per_step": 8, "path": "forward"},
            "e2e_eager": {"value": 1.0, "note": "one by one"}, "cpu_baseline": None,
            "layer_breakdown": {"engines": [1] * 5000}, "stack_check": None, "best_engine": None,
            "tables": {"v3": [2] * 5000}}
    kept = json.dumps(line)
    short, extras = bench.split_line(line)
    assert json.dumps(line) == kept                      # the caller's dicts stay
    assert short == {"metric": "m", "value": 2.5, "config": {"workload": "w"},
                     "roofline": {"frac": 1.0}, "e2e": {"value": 2.0, "h2d_bytes_per_step": 8},
                     "e2e_eager": {"value": 1.0}, "cpu_baseline": None}
    assert extras["tables"] == line["tables"] and extras["e2e.path"] == "forward"
    assert extras["roofline.bytes"] == "requested" and "cpu_baseline.single_thread" not in extras
    line["cpu_baseline"] = {"value": 3.0, "sample": "s", "single_thread": {"value": 1.0}}
    short, extras = bench.split_line(line)
    assert short["cpu_baseline"] == {"value": 3.0, "sample": "s"}
    assert extras["cpu_baseline.single_thread"] == {"value": 1.0}
