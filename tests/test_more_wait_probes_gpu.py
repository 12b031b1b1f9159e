"""Bounded waits of the products on tensor maps: a role of the kernel's warps that does nothing
makes the others give up, and the kernel ends in order (one CTA, a pair of CTAs, a cluster)."""
import pytest
import torch

import nvfp4_draft_head_gb300 as dh

pytestmark = pytest.mark.gpu
PRODUCER, ISSUER, EPILOGUE = range(3)


@pytest.fixture(scope="module", autouse=True)
def built():
    from nvfp4_draft_head_gb300 import build
    build.build()


def rand(shape, seed, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda") * scale).bfloat16()


# (M, N, K): few tokens with steps in the ring and more, in a cluster (48 rows leave SMs idle) and
# alone; many, in narrow tiles (parts of six steps for four accumulators), in wide ones two by two
# and in wide ones alone
SIZES = {"one step": (3, 70, 128), "a cluster": (5, 48, 8192), "alone": (5, 20000, 2048), "quantised before": (16, 19500, 2560),
         "narrow tiles": (300, 1000, 4096), "wide tiles": (2000, 4608, 1040), "wide tiles alone": (300, 12700, 1040)}


@pytest.mark.parametrize("size,role", [(s, r) for s in SIZES for r in (PRODUCER, ISSUER, EPILOGUE) if r != EPILOGUE or s != "one step"])
def test_product(size, role):
    M, N, K = SIZES[size]
    mm = dh.FP8BlockMatmul.from_weight(rand((N, K), 1, 0.02))
    x = rand((M, K), 2)
    want = mm(x)
    assert mm.device_error() == 0
    mm.wait_probe(x, role, 16)
    assert mm.device_error() == dh.DH_DEVERR_TIMEOUT
    assert mm.device_error() == 0
    assert torch.equal(mm(x), want) and mm.device_error() == 0


# (T, N, K): single CTAs and pairs; less than a ring of steps, and more than two accumulators
@pytest.mark.parametrize("role", [PRODUCER, ISSUER, EPILOGUE])
@pytest.mark.parametrize("T,N,K", [(20, 300, 64), (128, 1000, 2560), (300, 300, 64), (300, 1000, 2560), (700, 20000, 256)])
def test_loss(T, N, K, role):
    if role == EPILOGUE and N == 300:
        pytest.skip("one accumulator: nobody waits for the results")
    h, W, t = rand((T, K), 1), rand((N, K), 2, 0.1), torch.arange(T, device="cuda", dtype=torch.int32) % N
    want = dh.linear_cross_entropy(h, W, t)
    assert dh.linear_cross_entropy_device_error() == 0
    dh.linear_cross_entropy_wait_probe(h, W, t, role, 16)
    assert dh.linear_cross_entropy_device_error() == dh.DH_DEVERR_TIMEOUT
    assert dh.linear_cross_entropy_device_error() == 0
    for a, b in zip(dh.linear_cross_entropy(h, W, t), want):
        assert torch.equal(a, b)
    assert dh.linear_cross_entropy_device_error() == 0
