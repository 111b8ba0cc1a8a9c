"""Which kernel a dense product goes to, as the GPU tests' sizes take for granted (no GPU)."""
import os
import re

from conftest import ROOT
from test_gpu_linear_tiles import LARGE, SMALL, many


def test_sizes_of_the_tile_tests_are_the_tiles():
    with open(os.path.join(ROOT, "block_scaled_precision_mxfp8_amd", "csrc", "fp8_tiles.hip")) as f:
        rule = re.search(r"ragged == kDense && \(a\.m <= (\d+) \|\| \(int64_t\)\(\(a\.m \+ 63\) / 64\) \* a\.n <= (\d+)\)", f.read())
    assert rule and (int(rule[1]), int(rule[2])) == (64, 16384), "the rule has changed: choose the tests' sizes by the new one"
    assert many(*SMALL) and many(*LARGE)
