"""bench.py --layer: one JSON line whose metric is the one that its value is of."""

import argparse
import json

import pytest

import bench

pytestmark = pytest.mark.gpu


def test_the_layer_s_line(capsys):
    bench.layer_main(argparse.Namespace(steps=2, warmup=1))
    lines = capsys.readouterr().out.strip().splitlines()
    r = json.loads(lines[-1])
    assert len(lines) == 1 and r["unit"] == "tokens/s" and r["metric"].startswith("tokens/s") and r["metric"] != bench.METRIC
    assert r["value"] == pytest.approx(r["config"]["tokens"] / (r["ms_per_step"] * 1e-3), rel=1e-4)
    assert r["ms_per_step"] == pytest.approx(sum(k["ms"] for k in r["kernels"]), rel=1e-3)
    assert all(k["roofline"]["achieved"] > 0 for k in r["kernels"])


def test_the_lookup_reads_a_row_once(capsys):
    """Its bytes are 83.9 MB written and the rows that tokens name, under half of 8192 with a text's frequencies; counted for
    each token they would exceed the memory's rate."""
    bench.layer_main(argparse.Namespace(steps=2, warmup=1))
    k = json.loads(capsys.readouterr().out.strip().splitlines()[-1])["kernels"][0]
    assert k["kernel"] == "embedding lookup"
    assert 84e6 < k["roofline"]["achieved"] * 1e9 * k["ms"] * 1e-3 < 127e6
