"""Logits rows past one per CTA. The row kernels are persistent (some 456 CTAs on 152
SMs): with more rows, a CTA takes its second and third row with the ring already
running into them, the buffers of two rows in turn, ids fetched ahead and the last
row's end still open. References, tolerances and inputs as in test_rows_gpu.py."""
import pytest
import torch

import nvfp4_draft_head_gb300 as dh
from test_rows_gpu import NEG, TYPES, check_distill, check_logprobs, close, rand_rows, ref_distill, ref_stats, teacher

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU test needs a CUDA device"
    from nvfp4_draft_head_gb300 import build
    build.build()


def spoil(z):
    """Rows that leave the common path, scattered over the CTAs' turns: masked throughout,
    at the type's lowest value, of equal values, half masked, with a NaN."""
    M, n = z.shape
    z[5::61] = NEG
    z[7::67] = float(torch.finfo(z.dtype).min)
    z[9::71] = 0.5
    z[11::73, ::2] = NEG
    z[13::301, n // 2] = float("nan")
    return z


# rows, columns, columns of padding after a row, offset of the first row: odd strides give
# every row another offset from a 16-byte boundary
SHAPES = [(1400, 1, 0, 0), (1399, 37, 2, 1), (1400, 300, 0, 0), (1111, 1031, 4, 3), (1000, 4001, 0, 0), (950, 9001, 7, 1)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("M, n, pad, offset", SHAPES)
@pytest.mark.parametrize("spoilt", [False, True])
def test_logprobs(dtype, M, n, pad, offset, spoilt):
    z = rand_rows(M, n, TYPES[dtype], n, n + pad, offset)
    if spoilt:
        spoil(z)
    tokens = torch.randint(-1, n + 1, (M, 3), generator=torch.Generator("cuda").manual_seed(1), device="cuda", dtype=torch.int32)
    for k in (0, 1, 20, 128):
        check_logprobs(z, tokens, k, t=1.25)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("M, n, pad, offset", SHAPES)
@pytest.mark.parametrize("K", [5, 300])
def test_distillation(dtype, M, n, pad, offset, K):
    """Loss and gradient (in place too), loss alone, gradient from the normaliser."""
    z = spoil(rand_rows(M, n, TYPES[dtype], n, n + pad, offset))
    ids, val = teacher(z, K, 2)
    ids[17::79, : K // 2] = ids[17::79, :1]          # one column named many times
    ids[19::83] = -1                                 # no entry in use
    val[23::89, 1:] = NEG
    w = torch.rand(M, generator=torch.Generator("cuda").manual_seed(3), device="cuda") + 0.25
    w[2::97] = 0.0
    check_distill(z, ids, val, t=1.5, w=w)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_backward_in_place(dtype):
    M, n = 1399, 1031
    z = rand_rows(M, n, TYPES[dtype], 3, n + 2, 1)
    ids, val = teacher(z, 12, 2)
    lse = dh.distill_topk_forward(z, ids, val)[1]
    want = dh.distill_topk_backward(z, ids, val, lse)
    ref = ref_distill(z, ids, val, 1.0, None, None)
    q = ref_stats(z, 1.0)
    close(want, ref[2], ref[3] + (2e-5 + 3e-7 * ref[4].abs())[:, None] * q[2] / q[3], "backward")
    got = dh.distill_topk_backward(z, ids, val, lse, dlogits=z)
    assert got.data_ptr() == z.data_ptr() and torch.equal(got, want)


@pytest.mark.parametrize("M, n", [(150, 200_003), (330, 130_001)])
def test_several_rows_per_cluster(M, n):
    """Long rows of 32 bits, shared by clusters of CTAs that take more than one."""
    z = spoil(rand_rows(M, n, torch.float32, 1, n + 1, 1))
    tokens = torch.randint(-1, n + 1, (M, 2), generator=torch.Generator("cuda").manual_seed(1), device="cuda", dtype=torch.int32)
    check_logprobs(z, tokens, 20)
    ids, val = teacher(z, 20, 2)
    check_distill(z, ids, val, t=1.75)   # (below 1 the normaliser of a row at the lowest value is past fp32)


@pytest.mark.parametrize("M, n", [(3, 64_026), (700, 501)])
@pytest.mark.parametrize("G", [256, 257, 900])
def test_more_tokens_than_threads(M, n, G):
    z = rand_rows(M, n, torch.bfloat16, G)
    V = n + 700
    row_of = torch.randint(-1, n, (V,), generator=torch.Generator("cuda").manual_seed(2), device="cuda", dtype=torch.int32)
    tokens = torch.randint(-2, V + 2, (M, G), generator=torch.Generator("cuda").manual_seed(1), device="cuda", dtype=torch.int32)
    check_logprobs(z, tokens, 3, row_of=row_of)
    check_logprobs(z, tokens, 0)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("t", [4.3e-39, 1e-30, 1e30, 3e38])
def test_ends_of_the_temperatures_range(dtype, t):
    """Rows whose largest logit is 0, so that the normaliser stays within 32 bits."""
    for M, n in ((3, 700), (600, 1031), (2, 30_000)):
        z = rand_rows(M, n, TYPES[dtype], n)
        z -= z.amax(1, keepdim=True)
        check_logprobs(z, z.argmax(1).int(), 9, t=t)
