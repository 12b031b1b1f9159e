"""The first cross entropy of a process is a captured one: its error word is there, outlives the
graph, and tells what a replay met."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

START = """
import torch
import nvfp4_draft_head_gb300 as dh
h, W = torch.randn((300, 64), device="cuda").bfloat16(), torch.randn((1001, 64), device="cuda").bfloat16()
t = torch.randint(0, 1001, (300,), device="cuda", dtype=torch.int32)
graph = torch.cuda.CUDAGraph()
"""

# captured and replayed; then the graph goes, with the memory that it holds
STEP = START + """
with torch.cuda.graph(graph):
    out = dh.linear_cross_entropy(h, W, t)
assert all(dh._error_words.values()) and len(dh._error_words) == 1
graph.replay()
assert dh.linear_cross_entropy_device_error() == 0
want = [x.clone() for x in out]
assert all(torch.equal(a, b) for a, b in zip(dh.linear_cross_entropy(h, W, t), want))
del graph, out
torch.cuda.empty_cache()
assert all(torch.equal(a, b) for a, b in zip(dh.linear_cross_entropy(h, W, t), want))
assert dh.linear_cross_entropy_device_error() == 0
print("done")
"""

# a replay whose waits run out (a role of the kernel's warps does nothing)
PROBE = START + """
with torch.cuda.graph(graph):
    dh.linear_cross_entropy_wait_probe(h, W, t, 1, 16)
for _ in range(2):
    graph.replay()
    assert dh.linear_cross_entropy_device_error() == dh.DH_DEVERR_TIMEOUT
assert dh.linear_cross_entropy_device_error() == 0
print("done")
"""


@pytest.mark.parametrize("program", [STEP, PROBE], ids=["step", "wait"])
def test_first_call_is_captured(program):
    assert torch.cuda.is_available(), "GPU test needs a CUDA device"
    from nvfp4_draft_head_gb300 import build
    build.build()
    r = subprocess.run([sys.executable, "-c", program], capture_output=True, text=True, cwd=ROOT, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "done", r.stdout + r.stderr
