"""What the operator calls would launch, found in a child process (launch_grid_child.py)."""

import json
import os
import shutil
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


def grids(calls, tmp_path, cap=None):
    """[(status, message, [[grid x, grid y, threads], ...])] of the calls; cap: QKNORM_MAX_GRID."""
    if shutil.which("gcc") is None:
        pytest.skip("no C compiler")
    lib = str(tmp_path / "launch_record.so")
    subprocess.run(["gcc", "-shared", "-fPIC", "-Wall", "-Werror", os.path.join(HERE, "c", "launch_record.c"), "-o",
                    lib], check=True)
    env = {k: v for k, v in os.environ.items() if k != "QKNORM_MAX_GRID"}
    if cap:
        env["QKNORM_MAX_GRID"] = str(cap)
    res = subprocess.run([sys.executable, os.path.join(HERE, "launch_grid_child.py"), lib], env=env, text=True,
                         input=json.dumps(calls), capture_output=True, timeout=120)
    assert res.returncode == 0, res.stderr
    return [tuple(r) for r in json.loads(res.stdout)]
