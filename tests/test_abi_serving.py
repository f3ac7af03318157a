"""The serving calls refuse bad arguments on the host.  The checks (tests/abi_serving_checks.py) hand the entry points
invented device addresses, so they run in a child process that sees no GPU."""

import os
import subprocess
import sys

from conftest import ROOT


def test_serving_calls_refuse_before_any_device_access():
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider",
                        os.path.join(ROOT, "tests", "abi_serving_checks.py")],
                       env=env, cwd=ROOT, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, (r.stdout[-4000:] + r.stderr[-2000:])
    assert " passed" in r.stdout and "failed" not in r.stdout
