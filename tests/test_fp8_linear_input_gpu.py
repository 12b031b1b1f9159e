"""FP8BlockLinear, a frozen layer, does not keep its input: the storage goes with its last user, and
it may be changed in place before the backward pass; its gradient is refused a derivative."""
import pytest
import torch

import nvfp4_draft_head_gb300 as dh

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def layer():
    from nvfp4_draft_head_gb300 import build
    build.build()
    g = torch.Generator("cuda").manual_seed(1)
    return dh.FP8BlockMatmul.from_weight((torch.randn((272, 400), generator=g, device="cuda") * 0.05).bfloat16())


def leaf():
    return torch.randn((150, 400), generator=torch.Generator("cuda").manual_seed(2), device="cuda", requires_grad=True)


def test_the_input_is_released(layer):
    w = leaf()
    x = w * 2.0
    layer(x.detach())                       # (what a first call allocates for good)
    size = x.untyped_storage().nbytes()
    y = dh.FP8BlockLinear.apply(x, layer)
    before = torch.cuda.memory_allocated()
    del x
    assert before - torch.cuda.memory_allocated() >= size
    y.sum().backward()
    ones = torch.ones((150, 272), device="cuda").bfloat16()
    assert torch.equal(w.grad, 2.0 * layer.input_gradient(ones, out_dtype=torch.float32))


def test_the_input_may_be_changed_in_place(layer):
    w = leaf()
    x = w * 2.0
    y = dh.FP8BlockLinear.apply(x, layer)
    want = layer(x.detach().clone())
    x.add_(1.0)                             # a residual sum
    assert torch.equal(y, want)
    (y.float().sum() + x.sum()).backward()
    ones = torch.ones((150, 272), device="cuda").bfloat16()
    assert torch.equal(w.grad, (layer.input_gradient(ones, out_dtype=torch.float32) + 1.0) * 2.0)


def test_a_second_derivative_is_refused(layer):
    for square in (False, True):            # with a constant gradient, and one that depends on x
        x = leaf()
        y = dh.FP8BlockLinear.apply(x, layer, torch.float32)
        (dx,) = torch.autograd.grad(y.square().sum() if square else y.sum(), x, create_graph=True)
        with pytest.raises(RuntimeError, match="differentiable once"):
            (dx.square().sum() + x.square().sum()).backward()
        assert x.grad is None
        y = dh.FP8BlockLinear.apply(x, layer, torch.float32)
        (dx,) = torch.autograd.grad(y.square().sum() if square else y.sum(), x, create_graph=True)
        with pytest.raises(RuntimeError, match="differentiable once"):
            torch.autograd.grad(dx.sum(), x)
