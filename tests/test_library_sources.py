"""What the kernels' sources may not hold. The library is one file for programs on one GPU and on
several (the sharded head, the replicas of the benchmark): none of its copies goes to more than
one CTA."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "nvfp4_draft_head_gb300", "csrc")
FILES = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")))


def code(path):
    """The file without its comments."""
    with open(path) as f:
        text = f.read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", " ", text, flags=re.S)


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_no_copy_to_several_ctas(path):
    for ptx in re.findall(r"cp\.async\.bulk[\w.:]*", code(path)):
        assert "multicast" not in ptx, ptx
