"""The library holds the variants of the paged kernel of few rows that calls reach, and
no others (names of the built library; nothing is launched)."""
import re
import subprocess

from dual_window_attention_b200 import build


def test_variants_of_the_kernel_of_few_rows():
    names = subprocess.run(["nm", "-C", build.build()], check=True, capture_output=True, text=True).stdout
    held = set(re.findall(r" W void ttcd::paged_decode_kernel<(\d+), (\d+), (\d+)>", names))
    # (head_dim, rows, tiles in flight): 16 rows have one in flight, 8 rows two, or one
    # where that holds more CTAs on an SM (not at head_dim 32)
    want = {(32, 8, 2), (64, 8, 2), (128, 8, 2), (64, 8, 1), (128, 8, 1), (32, 16, 1), (64, 16, 1), (128, 16, 1)}
    assert held == {tuple(map(str, x)) for x in want}
