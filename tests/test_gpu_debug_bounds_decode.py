"""The bounds-checked build on the speculative decoding calls: the release build's bits on valid
inputs, FLIDE_ERR_BOUNDS with the site on a corrupted index (each build in a child process)."""
import json
import os
import subprocess
import sys

import numpy as np
import pytest

from tree_forked_decision_b200 import flide

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def _child(mode, out_dir, debug):
    env = dict(os.environ, FLIDE_DEBUG_BOUNDS="1" if debug else "0")
    out = subprocess.run([sys.executable, os.path.join(HERE, "_debug_bounds_decode_cases.py"), mode, out_dir], env=env,
                         capture_output=True, text=True, timeout=600)
    assert out.returncode == 0, out.stderr[-3000:]


def test_debug_build_matches_release_build(tmp_path):
    got = {}
    for name, debug in (("release", False), ("debug", True)):
        (tmp_path / name).mkdir()
        _child("run", str(tmp_path / name), debug)
        got[name] = (json.loads((tmp_path / name / "result.json").read_text()), np.load(tmp_path / name / "arrays.npz"))
    assert got["release"][0].pop("debug_bounds") == 0 and got["debug"][0].pop("debug_bounds") == 1
    assert got["release"][0] == got["debug"][0] and not any(got["debug"][0].values())
    a, b = got["release"][1], got["debug"][1]
    assert sorted(a.files) == sorted(b.files)
    for k in a.files:
        assert np.array_equal(a[k], b[k], equal_nan=True), k


def test_debug_build_reports_a_corrupted_index(tmp_path):
    _child("corrupt", str(tmp_path), True)
    res = json.loads((tmp_path / "corrupt.json").read_text())
    sites = {"ancestor": (804,), "token": (701,), "range": (802,)}
    for tag, (status, site, value, planted) in res.items():
        assert status == flide.ERR_BOUNDS and site in sites[tag] and value == planted, (tag, res[tag])
