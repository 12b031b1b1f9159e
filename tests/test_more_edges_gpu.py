"""Calls at the edges of what the quantisers, the FP8 block-scaled product and the vocabulary cross
entropy document: answered, or refused before anything is launched."""
import pytest
import torch

import nvfp4_draft_head_gb300 as dh

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from nvfp4_draft_head_gb300 import build
    build.build()


def rand(shape, seed=1, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=torch.Generator(DEV).manual_seed(seed), device=DEV) * scale).to(dtype)


@pytest.mark.parametrize("quantise", [dh.fp8_quantize_blocks, dh.fp8_quantize_rows, dh.nvfp4_quantize_rows])
def test_ids_that_are_not_contiguous_are_refused(quantise):
    W = rand((256, 256))
    ids = torch.arange(128, dtype=torch.int32, device=DEV)
    for bad in (ids[::2], ids[:1].expand(64)):
        with pytest.raises(ValueError, match="contiguous"):
            quantise(W, bad)
        with pytest.raises(ValueError, match="contiguous"):
            quantise(W, bad, stream=torch.cuda.Stream())
    quantise(W, ids[::2].contiguous())


def test_sizes_past_32_bits_are_refused():
    """More tokens than the library's integers hold (one row of them, cut, would be computed)."""
    mm = dh.FP8BlockMatmul.from_weight(rand((1, 16)))
    dy = torch.empty((2 ** 32 + 1, 1), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(dh.DraftHeadError, match="shape"):
        mm.input_gradient(dy)
    del dy
    x = torch.empty((2 ** 24 + 1, 16), dtype=torch.bfloat16, device=DEV)
    for call in (mm, mm.forward, lambda t: mm.wait_probe(t, 1, 16)):
        with pytest.raises(dh.DraftHeadError, match="shape"):
            call(x)
    for shape in ((2 ** 24 + 1, 16), (1, 2 ** 20 + 16)):
        with pytest.raises(dh.DraftHeadError, match="shape"):
            dh.FP8BlockMatmul(torch.empty(shape, dtype=torch.uint8, device=DEV), torch.empty((-(-shape[0] // 128), -(-shape[1] // 128)), device=DEV))


@pytest.mark.parametrize("sliced", [False, True])
def test_no_tokens_with_given_results(sliced):
    """Empty tensors have no address of their own to tell them apart by."""
    def none(dtype):
        return torch.empty((4, 64), dtype=dtype, device=DEV)[:0] if sliced else torch.empty((0, 64), dtype=dtype, device=DEV)

    head, tokens = rand((40, 64)), torch.empty(0, dtype=torch.int32, device=DEV)
    h, dx, dw = none(torch.bfloat16), none(torch.bfloat16), torch.full((40, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    loss, got_dx, got_dw = dh.linear_cross_entropy(h, head, tokens, dhidden=dx, dhead=dw)
    assert loss.shape == (0,) and got_dx is dx and got_dw is dw and not dw.any()
    dw.fill_(3.0)
    lse = torch.empty(0, device=DEV)
    got_dx, got_dw = dh.linear_cross_entropy_backward(h, head, tokens, lse, dhidden=dx, dhead=dw)
    assert got_dx is dx and got_dw is dw and not dw.any()
    with pytest.raises(ValueError, match="gradient of"):
        dh.linear_cross_entropy(h, head, tokens, dhead=head)
    mm = dh.FP8BlockMatmul.from_weight(rand((64, 64)))
    assert mm(h, dx) is dx and mm.input_gradient(h, dx) is dx


@pytest.mark.parametrize("T", [60, 200])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_rows_that_are_left_out_have_any_gradient_of_their_loss(T, bad):
    """Rows of weight 0 and tokens without a row: what comes back to their losses (0 / 0 of an empty
    count, say) reaches nothing."""
    h, head = rand((T, 64)).requires_grad_(), rand((300, 64), 2, 0.1).requires_grad_()
    tokens = torch.arange(T, dtype=torch.int32, device=DEV)
    weights = torch.rand(T, generator=torch.Generator(DEV).manual_seed(3), device=DEV) + 0.5
    weights[::3] = 0.0
    tokens[1::3] = -100
    up = torch.ones(T, device=DEV)
    loss = dh.LinearCrossEntropy.apply(h, head, tokens, weights)
    want = torch.autograd.grad(loss, (h, head), up, retain_graph=True)
    up[::3] = up[1::3] = bad
    got = torch.autograd.grad(loss, (h, head), up)
    assert all(torch.equal(a, b) and b.isfinite().all() for a, b in zip(got, want))
    assert not got[0][::3].any() and not got[0][1::3].any() and got[0][2::3].any()


@pytest.mark.parametrize("T,N", [(3, 40), (100, 700), (300, 700)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_a_row_whose_logits_are_all_minus_infinity(T, N, dtype):
    """An infinity times head rows of one sign: no logit is NaN, and the loss, lse and dh are all the same,
    in a row that is left out its lse."""
    h, head = rand((T, 64), dtype=dtype), rand((N, 64), 2, 0.1, dtype)
    head[:, 5] = -head[:, 5].abs() - 0.01
    tokens = torch.arange(T, dtype=torch.int32, device=DEV) % N
    want = dh.linear_cross_entropy_forward(h, head, tokens)
    h[1, 5] = h[2, 5] = float("inf")
    tokens[2] = -100
    loss, lse, rest = dh.linear_cross_entropy_forward(h, head, tokens)
    assert loss[1].isnan() and loss[2] == 0.0 and lse[1:3].isnan().all()
    others = [i for i in range(T) if i not in (1, 2)]
    assert torch.equal(loss[others], want[0][others]) and torch.equal(lse[others], want[1][others])
    both, dx, dw = dh.linear_cross_entropy(h, head, tokens)
    assert both[1].isnan() and both[2] == 0.0 and dx[1].isnan().all() and not dx[2].any() and dw.isnan().any()
    assert dx[others].isfinite().all()
    dx, _ = dh.linear_cross_entropy_backward(h, head, tokens, lse, rest=rest, dhead=False)
    assert dx[1].isnan().all() and not dx[2].any() and dx[others].isfinite().all()
