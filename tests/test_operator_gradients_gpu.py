"""The operators without a gradient refuse inputs that require one."""
import pytest
import torch

import nvfp4_draft_head_gb300 as dh
from test_matmul_gpu import weight

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU test needs a CUDA device"
    from nvfp4_draft_head_gb300 import build
    build.build()


def test_inputs_that_require_a_gradient():
    mm = dh.NVFP4Matmul(*weight(64, 32, 1)[:3])
    x = torch.randn((5, 32), device="cuda", requires_grad=True)
    z = torch.randn((5, 64), device="cuda", requires_grad=True)
    y, r = mm(x.detach()), dh.token_logprobs(z.detach(), top_k=3)
    side = torch.cuda.Stream()
    for call in (lambda: mm(x), lambda: mm(x * 2), lambda: mm(x, stream=side), lambda: dh.token_logprobs(z),
                 lambda: dh.token_logprobs(z * 2, top_k=3), lambda: dh.token_logprobs(z, stream=side)):
        with pytest.raises(ValueError, match="gradient"):
            call()
    with torch.no_grad():
        assert torch.equal(mm(x), y)
        assert all(torch.equal(a, b) for a, b in zip(dh.token_logprobs(z, top_k=3)[1:], r[1:]))
    # the explicit loss and gradient take such logits: the gradient is their result
    ids = torch.zeros((5, 1), dtype=torch.int32, device="cuda")
    loss, dz = dh.distill_topk(z, ids, torch.zeros((5, 1), device="cuda"))
    z.backward(dz)
    assert torch.equal(z.grad, dz) and not loss.requires_grad
