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


@pytest.mark.parametrize("logits_too", [False, True])
def test_gradient_of_the_row_weights(logits_too):
    """loss_m is linear in w_m: its derivative is the row's loss at weight 1, for a
    row of weight 0 too. Tolerance: that of the loss, times the upstream gradient."""
    M, n, K, t = 40, 1031, 9, 1.5
    z = rand_rows(M, n, torch.float32, 3)
    ids, val = teacher(z, K, 4)
    ids[7] = -1                                  # no entry in use: nothing depends on this weight
    w = torch.rand(M, generator=torch.Generator("cuda").manual_seed(5), device="cuda")
    w[3] = 0.0
    up = torch.rand(M, generator=torch.Generator("cuda").manual_seed(6), device="cuda")
    z.requires_grad_(logits_too)
    w.requires_grad_()
    loss = dh.DistillTopK.apply(z, ids, val, t, w)
    (loss * up).sum().backward()
    base, tol = ref_distill(z.detach(), ids, val, t, None, None)[:2]
    close(w.grad, base * up, tol * up + 1e-6 * (base * up).abs(), "weights")
    assert w.grad[7] == 0 and loss[3] == 0
    if logits_too:
        ref = ref_distill(z.detach(), ids, val, t, w.detach() * up, None)
        close(z.grad, ref[2], ref[3] + 1e-6, "logits")


def test_a_gradient_for_the_teacher_is_refused():
    z = rand_rows(5, 70, torch.float32, 1).requires_grad_()
    ids, val = teacher(z.detach(), 6, 2)
    val.requires_grad_()
    with pytest.raises(RuntimeError, match="teacher"):
        dh.DistillTopK.apply(z, ids, val).sum().backward()
    (dz,) = torch.autograd.grad(dh.DistillTopK.apply(z, ids, val).sum(), z)   # the logits' alone, and the loss alone
    ref = ref_distill(z.detach(), ids, val.detach(), 1.0, None, None)
    close(dz, ref[2], ref[3] + 1e-6, "logits")
    with torch.no_grad():
        close(dh.DistillTopK.apply(z, ids, val), ref[0], ref[1], "loss")
    z.grad = None   # (the refused pass had reached the logits)
    dh.DistillTopK.apply(z, ids, val.detach()).sum().backward()
    assert torch.equal(z.grad, dz)
