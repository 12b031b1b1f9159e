"""What autograd gets from DistillTopK, and what it is refused."""
import pytest
import torch

import nvfp4_draft_head_gb300 as dh
from test_rows_gpu import close, rand_rows, ref_distill, teacher

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU test needs a CUDA device"
    from nvfp4_draft_head_gb300 import build
    build.build()


def test_second_derivatives_are_refused():
    """The gradient's graph is refused, not missing: a penalty on the gradient beside
    another term of the loss must not lose its derivative without a word."""
    z = rand_rows(5, 70, torch.float32, 1).requires_grad_()
    ids, val = teacher(z.detach(), 6, 2)
    (dz,) = torch.autograd.grad(dh.DistillTopK.apply(z, ids, val).sum(), z, create_graph=True)
    ref = ref_distill(z.detach(), ids, val, 1.0, None, None)
    close(dz.detach(), ref[2], ref[3] + 1e-6, "gradient")
    with pytest.raises(RuntimeError, match="differentiable once"):
        ((dz * dz).sum() + z.square().sum()).backward()
    scale = torch.ones((), device="cuda", requires_grad=True)
    (dz,) = torch.autograd.grad((dh.DistillTopK.apply(z, ids, val) * scale).sum(), z, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiable once"):
        torch.autograd.grad(dz.sum() + scale, scale)
