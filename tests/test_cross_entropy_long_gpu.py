"""Gradients of the vocabulary cross entropy over long contractions: sums whose terms all have one
sign, where an error that does not average out can be told from roundings that do.

A tensor-core sum is truncated by at most 2^-23 of itself at each of its instructions (16 elements of
the contraction). Summed for c steps of 64 elements at a time, in between added in 32 bits, a mean of
relative errors keeps at most 4 c 2^-23; with 32 steps at most, as here required, 2^-16. What rounds
to nearest averages out: the results' own rounding and g's, each at most u, half a step of the type,
uniform over values that spread over many steps: a standard deviation of at most sqrt(2 / 3) u per
element, six of which over the square root of their number are allowed.
"""
import pytest
import torch

import nvfp4_draft_head_gb300 as dh

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from nvfp4_draft_head_gb300 import build
    build.build()


def make(T, N, K, spread, dtype=torch.float16):
    """Positive hidden states and head rows; every token is row 0, which is zeros: the other rows' weights
    in g are positive, and row 0 adds nothing to dh."""
    g = torch.Generator(DEV).manual_seed(T + N + K)
    h = (torch.rand((T, K), generator=g, device=DEV) + 0.25).to(dtype)
    head = (torch.rand((N, K), generator=g, device=DEV) * spread + 0.01).to(dtype)
    head[0] = 0.0
    weights = torch.rand(T, generator=g, device=DEV) + 0.5
    return h, head, torch.zeros(T, dtype=torch.int32, device=DEV), weights


def mean_error(got, want):
    d = (got.double() - want) / want
    u = torch.finfo(got.dtype).eps / 2
    tol = 2.0 ** -16 + 6 * (2 / 3) ** 0.5 * u / d.numel() ** 0.5
    assert d.mean().abs() <= tol, (d.mean().item(), tol)


@pytest.mark.parametrize("T,N,K", [(1_100_000, 1000, 16), (131_072, 2048, 64), (20_000, 700, 512)])
def test_head_gradient_of_many_tokens(T, N, K):
    h, head, tokens, weights = make(T, N, K, 2.0 / K ** 0.5)
    weights *= 4.0 / T ** 0.5        # (sums that float16 holds)
    _, _, dw = dh.linear_cross_entropy(h, head, tokens, weights)
    want = torch.zeros((N, K), dtype=torch.float64, device=DEV)
    for r in range(0, T, 100_000):
        x = h[r:r + 100_000].double()
        want += (torch.softmax(x @ head.double().t(), 1) * weights[r:r + 100_000, None]).t() @ x
    mean_error(dw[1:], want[1:])
    assert dh.linear_cross_entropy_device_error() == 0


@pytest.mark.parametrize("T,N,K", [(40, 400_000, 256), (300, 400_000, 256), (1000, 64_026, 520)])
def test_hidden_gradient_over_a_large_vocabulary(T, N, K):
    h, head, tokens, weights = make(T, N, K, 2.0 / K ** 0.5)
    _, dx, _ = dh.linear_cross_entropy(h, head, tokens, weights)
    p = torch.softmax(h.double() @ head.double().t(), 1) * weights[:, None]
    mean_error(dx, p @ head.double())
    assert dh.linear_cross_entropy_device_error() == 0
