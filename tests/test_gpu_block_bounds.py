"""The residual block's operators on the bounds-checked build of the library: no kernel reads or writes outside its
tensors (tests/block_bounds_cases.py, in a process of its own)."""

import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_route_stays_inside_its_tensors():
    from einsum_device_side_gb300 import build
    lib = build.build(variant="debug")
    env = dict(os.environ, TROP_LIBRARY="debug")
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "block_bounds_cases.py")], env=env, cwd=ROOT,
                       capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0, r.stderr[-3000:]
    got = json.loads(r.stdout.strip().splitlines()[-1])
    assert got["library"] == lib and got["cases"] >= 1000
    assert got["wrong"] == [], got["wrong"]
    assert got["report"] is not None and got["report"]["count"] == 0, got["report"]
