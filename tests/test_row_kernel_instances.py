"""The row kernels of layer norm that the library holds are those that some call reaches: rows by
their number of octets (groups of eight channels), with and without edge channels, few rows or many."""
import re
import shutil
import subprocess

import pytest

from speech_encoder_depthwise_b200 import build

# (octets up to, threads per row, octets per thread)
FEW = [(16, 16, 1), (32, 32, 1), (64, 32, 2), (128, 64, 2), (192, 64, 3), (256, 128, 2), (384, 128, 3), (512, 256, 2),
       (768, 256, 3), (1024, 256, 4)]
LONG = [(192, 64, 3), (256, 64, 4), (384, 128, 3), (512, 128, 4), (768, 256, 3), (1024, 256, 4)]
MANY = [(48, 16, 3), (64, 16, 4), (80, 16, 5), (96, 32, 3), (128, 32, 4)] + LONG
BWD = [(32, 16, 2), (64, 32, 2), (96, 32, 3), (128, 32, 4)] + LONG
TABLES = {
    ("fwd", "float", "false"): [(8, 8, 1)] + FEW,
    ("fwd", "float", "true"): FEW,
    ("fwd", "16", "false"): [(8, 8, 1), (16, 8, 2), (24, 8, 3), (32, 8, 4)] + FEW + MANY,
    ("fwd", "16", "true"): [(16, 16, 1), (32, 16, 2)] + FEW + MANY,
    ("bwd", "float", "false"): [(8, 8, 1), (16, 8, 2)] + BWD,
    ("bwd", "float", "true"): [(16, 16, 1)] + BWD,
}
TABLES["bwd", "16", "false"], TABLES["bwd", "16", "true"] = TABLES["bwd", "float", "false"], TABLES["bwd", "float", "true"]


@pytest.mark.skipif(shutil.which("nm") is None, reason="needs nm")
def test_instances_are_those_that_calls_reach():
    names = subprocess.run(["nm", "-C", build.build()], capture_output=True, text=True, check=True).stdout
    held = set(re.findall(r" \w void dwk::\w+::layernorm_(fwd|bwd)_rows_kernel<(\w+), (\d+), (\d+), (true|false), (\d)>\(",
                          names))
    reached = {(way, t, str(threads), str(octets), edges, mode)
               for (way, kind, edges), rows in TABLES.items() for t in (["float"] if kind == "float" else
                                                                        ["__nv_bfloat16", "__half"])
               for _, threads, octets in rows for mode in "012"}
    assert held == reached
