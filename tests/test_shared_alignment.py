"""Shared arrays of floats that kernels access 16 bytes at a time say so: without it a
compiler may place them on any multiple of 4."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "dual_window_attention_b200", "csrc")


def test_vector_accesses_of_shared_arrays_are_aligned():
    seen = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cuh"))):
        with open(path) as f:
            source = f.read()
        for m in re.finditer(r"__shared__ (__align__\(\d+\) )?float (\w+)\[", source):
            if re.search(r"float4\s*\*>\(&" + m[2] + r"\[", source):
                seen += 1
                assert m[1] == "__align__(16) ", (os.path.basename(path), m[2])
    assert seen  # the array of paged_decode.cuh
