"""First calls of the operators from several threads at once (each finds out what a
launch needs to know of the device)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import threading
import torch
import nvfp4_draft_head_gb300 as dh
z = torch.randn((300, 4001), device="cuda")
ids, val = torch.randint(0, 4001, (300, 8), device="cuda", dtype=torch.int32), torch.randn((300, 8), device="cuda")
x = torch.randn((300, 64), device="cuda")
mm = dh.NVFP4Matmul.from_weight(torch.randn((1088, 64), device="cuda").bfloat16())
torch.cuda.synchronize()
start, out = threading.Barrier(8), [None] * 8
def call(i):
    start.wait()
    out[i] = [dh.token_logprobs(z, top_k=5).top_ids, *dh.distill_topk(z, ids, val), *dh.distill_topk_forward(z, ids, val), mm(x)]
threads = [threading.Thread(target=call, args=(i,)) for i in range(8)]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
assert all(torch.equal(a, b) for o in out for a, b in zip(o, out[0], strict=True))
print("equal")
"""


def test_first_calls_at_once():
    from nvfp4_draft_head_gb300 import build
    build.build()
    r = subprocess.run([sys.executable, "-c", PROGRAM], capture_output=True, text=True, cwd=ROOT, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "equal", r.stdout + r.stderr
