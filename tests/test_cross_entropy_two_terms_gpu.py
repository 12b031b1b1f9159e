"""Gradients of the vocabulary cross entropy from g in two 16-bit terms, at the caller's choice.

What is left is the results' own rounding: at most u (half a step of the type), uniform, so u /
sqrt(3) in the relative 2-norm where all mantissas were 1 and less otherwise. 32-bit sums and g's second
rounding, u^2, are far below. Nothing is said of one term: the error that it adds is sum dg h over sum g
h, which for dW of many tokens may be anything from as much again down to nothing, as |dg| <= u |g| are
independent and the terms of the sum below are not. Elementwise: the tolerances of
test_cross_entropy_gpu."""
import pytest
import torch

import nvfp4_draft_head_gb300 as dh
from test_cross_entropy_gpu import make, near, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from nvfp4_draft_head_gb300 import build
    build.build()


def off(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


# pairs with one row block and more; a last round in parts; several pieces of 2,048 head rows, which one
# term would have in one of 5,120
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,N,K", [(129, 700, 136), (300, 513, 1032), (1000, 5000, 264), (1250, 8000, 2056), (52_000, 5003, 64)])
def test_two_terms(T, N, K, dtype):
    s = make(T, N, K, dtype)
    out, tol, _ = reference(s)
    loss, dx, dw = dh.linear_cross_entropy(**s, two_terms=True)
    assert torch.equal(loss, dh.linear_cross_entropy(**s)[0])
    u = torch.finfo(dtype).eps / 2
    for got, k in ((dx, "dhidden"), (dw, "dhead")):
        near(got, out[k], tol[k], k)
        assert off(got, out[k]) <= u / 3 ** 0.5
        assert off(got, out[k]) <= 1.03 * off(out[k].to(dtype), out[k])
    _, lse, rest = dh.linear_cross_entropy_forward(**s)
    a = (s["hidden"], s["head"], s["tokens"], lse, s["weights"], rest, s["row_of"])
    both = dh.linear_cross_entropy_backward(*a, two_terms=True)
    assert torch.equal(both[0], dx) and torch.equal(both[1], dw)
    assert torch.equal(dh.linear_cross_entropy_backward(*a, dhead=False, two_terms=True)[0], dx)
    assert torch.equal(dh.linear_cross_entropy_backward(*a, dhidden=False, two_terms=True)[1], dw)
    h, W = s["hidden"].clone().requires_grad_(), s["head"].clone().requires_grad_()
    dh.LinearCrossEntropy.apply(h, W, s["tokens"], s["weights"], s["row_of"], True).sum().backward()
    assert torch.equal(h.grad, dx) and torch.equal(W.grad, dw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for r, w in zip(dh.linear_cross_entropy(**s, stream=side, two_terms=True), (loss, dx, dw)):
        side.synchronize()
        assert torch.equal(r, w)
    assert dh.linear_cross_entropy_device_error() == 0


@pytest.mark.parametrize("T", [1, 128])
def test_few_tokens_have_them_anyway(T):
    s = make(T, 300, 72, torch.bfloat16)
    for a, b in zip(dh.linear_cross_entropy(**s, two_terms=True), dh.linear_cross_entropy(**s)):
        assert torch.equal(a, b)


def test_rows_that_are_left_out_and_not_finite():
    s = make(300, 500, 136, torch.bfloat16)
    _, _, live = reference(s)
    want = dh.linear_cross_entropy(**s, two_terms=True)
    junk = s["hidden"].clone()
    junk[~live] = float("nan")
    for a, b in zip(dh.linear_cross_entropy(**{**s, "hidden": junk}, two_terms=True), want):
        assert torch.equal(a, b)
    bad = s["hidden"].clone()
    first = live.nonzero()[0, 0]
    bad[first, 3] = float("inf")
    loss, dx, dw = dh.linear_cross_entropy(**{**s, "hidden": bad}, two_terms=True)
    others = torch.arange(300, device="cuda") != first
    assert loss[first].isnan() and dx[first].isnan().all() and dw.isnan().any() and torch.equal(dx[others], want[1][others])
