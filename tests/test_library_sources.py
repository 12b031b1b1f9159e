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


def kernels(text):
    """(name, parameters, body) of the file's kernels."""
    for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\([^{;]*?\)\s+)?(\w+)\s*\(", text):
        ends, depth, at = [], 1, m.end()
        for opening, closing in ("()", "{}"):
            while depth:
                depth += {opening: 1, closing: -1}.get(text[at], 0)
                at += 1
            ends.append(at)
            at = text.index("{", at) + 1 if opening == "(" else at
            depth = 1
        yield m[1], text[m.end():ends[0] - 1], text[ends[0]:ends[1]]


def test_kernels_that_start_early_read_with_ordinary_loads():
    """A kernel that calls programmatic_wait() starts while the one before it still writes. Loads that
    promise data which nobody writes during the kernel (__ldg, pointers to const that are
    __restrict__) may go before that wait or past it to stale data: there they are for the scales of
    a weight alone, which no kernel of a call writes."""
    seen = []
    for path in FILES:
        text = code(path)
        for name, parameters, body in kernels(text):
            if "programmatic_wait()" not in body:
                continue
            seen.append(name)
            for p in parameters.split(","):
                assert not ("const" in p and "__restrict__" in p), (os.path.basename(path), name, p.strip())
        if "programmatic_wait()" in text or os.path.basename(path) == "dh_fp8_blocks.cuh":
            for pointer in re.findall(r"__ldg\(\s*(?:reinterpret_cast<[^>]*>\()?\s*([\w.]+)", text):
                assert pointer == "sw", (os.path.basename(path), pointer)
    # the draft step's kernel starts early too, and reads the head before its wait: the hidden states are not the head
    text = code(os.path.join(CSRC, "dh_gemv_mma.cuh"))
    assert set(re.findall(r"__ldg\(\s*(?:reinterpret_cast<[^>]*>\()?\s*([\w.]+)", text)) <= {"a.scale", "a.idx"}
    assert {"product_kernel", "few_kernel", "quantize_kernel", "join_kernel", "rows_kernel", "sum_kernel", "rest_kernel"} <= set(seen)
