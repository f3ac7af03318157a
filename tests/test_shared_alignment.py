"""Shared memory that is read in wider units than its elements says so where it is declared."""

import glob
import os
import re

from conftest import ROOT

CSRC = os.path.join(ROOT, "tree_speculative_decoding_spec_gb300", "csrc")


def test_arrays_read_sixteen_bytes_at_a_time_are_aligned():
    """Every static shared array whose address goes through a cast to a 16-byte vector is declared with that alignment."""
    seen = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        text = open(path).read()
        for m in re.finditer(r"^\s*__shared__ (.*?)(\w+)\[", text, re.M):
            kind, name = m.group(1).split()[-1], m.group(2)
            cast = re.search(r"reinterpret_cast<(?:const )?(?:float4|uint4|int4|ulonglong2)\s*\*>\(\s*&?%s\b" % name, text)
            if cast and kind not in ("float4", "uint4", "int4", "ulonglong2"):
                seen += 1
                assert "__align__(16)" in m.group(0), f"{os.path.basename(path)}: {m.group(0).strip()} is read by {cast.group(0)}"
    assert seen >= 2
