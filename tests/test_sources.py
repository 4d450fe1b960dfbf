"""What the kernels' sources may not hold."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "nvfp4_weight_only_02_gb300", "csrc")


def test_no_multicast_copies():
    """Ranks of a job on several GPUs run this library too: no copy goes to several CTAs at once.  (A commit that arrives
    at the barriers of both CTAs of a pair is none.)"""
    files = glob.glob(os.path.join(CSRC, "*"))
    assert files
    for path in files:
        for text in re.findall(r'"\s*cp\.async\.bulk[^;]*;', open(path).read()):
            assert ".multicast" not in text, path
