"""The beam and eviction calls refuse bad arguments on the host, and their binding what would change on its way to the
library.  The checks of tests/abi_keep_checks.py hand the entry points invented device addresses, so they run in a child
process that sees no GPU."""

import os
import subprocess
import sys

import pytest

from conftest import ROOT


def test_beam_and_eviction_calls_refuse_before_any_device_access():
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider",
                        os.path.join(ROOT, "tests", "abi_keep_checks.py")],
                       env=env, cwd=ROOT, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, (r.stdout[-4000:] + r.stderr[-2000:])
    assert " passed" in r.stdout and "failed" not in r.stdout


@pytest.fixture(scope="module")
def binding():
    import __graft_entry__
    __graft_entry__.build()
    from tree_speculative_decoding_spec_gb300 import _binding
    return _binding


@pytest.mark.parametrize("x", [1 << 31, (1 << 32) + 4, -(1 << 32), 0.5, float("nan"), float("inf")])
def test_numbers_that_would_change_on_the_way_are_refused(binding, x):
    with pytest.raises(ValueError, match="budget"):
        binding._whole(x, "budget")


def test_whole_numbers_pass(binding):
    assert [binding._whole(x, "K") for x in (0, 4, 4.0, -1, (1 << 31) - 1)] == [0, 4, 4, -1, (1 << 31) - 1]
