"""CPU: no kernel source has a TMA load with cluster multicast (jobs on several GPUs run the same library)."""
import glob
import os
import re

from conftest import ROOT


def test_no_source_has_a_multicast_load():
    paths = glob.glob(os.path.join(ROOT, "quantized_moe_gb300", "csrc", "*.cu*")) + glob.glob(os.path.join(ROOT, "include", "*.h"))
    assert paths
    for path in paths:
        text = re.sub(r'"\s*"', "", open(path).read())  # (string literals that follow each other are one)
        for load in re.findall(r"cp\.async\.bulk[^;]*", text):
            assert "multicast" not in load, path
