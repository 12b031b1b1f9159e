"""The gradient from a kept normaliser on rows far from zero, where fp32 no longer
holds the normaliser's logarithm of the sum.

Tolerance: that of the fused gradient (test_rows_gpu.py), and on q the rounding of a
normaliser below 1,024 in magnitude, at most half its spacing 2^-14 there (3.1e-5), with the
exponent's own (|x| 2^-23): in all 2e-5 + 5e-5 of q."""
import pytest
import torch

import nvfp4_draft_head_gb300 as dh
from test_rows_gpu import NEG, TYPES, close, rand_rows, ref_distill, ref_stats, teacher

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU test needs a CUDA device"
    from nvfp4_draft_head_gb300 import build
    build.build()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("M, n", [(9, 50), (9, 30_011), (1200, 700), (40, 200_003)])
@pytest.mark.parametrize("t", [1.0, 0.5, 3.0])
def test_rows_far_from_zero(dtype, M, n, t):
    T = TYPES[dtype]
    z = rand_rows(M, n, T, n)
    low = float(torch.finfo(T).min)
    z[0::9] = low                                      # every column at the type's lowest value
    z[1::9, 1:] = low
    z[2::9] = (z[2::9].float() + 3000.0).to(T)
    z[3::9] = (z[3::9].float() * 100.0 - 20000.0).to(T)
    z[4::9, ::3] = NEG
    z[4::9, 1::3] = low
    z[4::9, 2::3] = low
    z[5::9] = NEG
    z[6::9] = -low                                     # and at the largest
    z[7::9, n // 2] = float("nan")
    ids, val = teacher(z.float().nan_to_num(0.0).clamp(-50, 50), 6, 1)
    ids[4::9, 0] = 1
    w = torch.rand(M, generator=torch.Generator("cuda").manual_seed(2), device="cuda") + 0.5
    ref = ref_distill(z, ids, val, t, w, None)
    _, _, e, S = ref_stats(z, t)
    tol = ref[3] + (w.double() * t * 7e-5)[:, None] * (e / S).nan_to_num(0)
    loss, lse = dh.distill_topk_forward(z, ids, val, temperature=t, weights=w)
    close(dh.distill_topk_backward(z, ids, val, lse, w, temperature=t), ref[2], tol, "backward")
    leaf = z.clone().requires_grad_()
    dh.DistillTopK.apply(leaf, ids, val, t, w).sum().backward()
    close(leaf.grad, ref[2], tol, "autograd")
    # in place, rows that are summed again among them
    want = dh.distill_topk_backward(z, ids, val, lse, w, temperature=t)
    got = dh.distill_topk_backward(z, ids, val, lse, w, temperature=t, dlogits=z)
    assert torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("t", [1e-38, 1e-20, 1e20, 1e37])
def test_ends_of_the_temperatures_range(dtype, t):
    """The normaliser is ordinary, its product with t is not. (At 1e-38 and 1e-20 the
    logits are scaled with t, so that the probabilities are ordinary too.)"""
    z = rand_rows(7, 901, TYPES[dtype], 4)
    ids, val = teacher(z, 5, 1)
    if t < 1:
        z, val = (z.float() * t).to(z.dtype), val * t
    ref = ref_distill(z, ids, val, t, None, None)
    _, _, e, S = ref_stats(z, t)
    _, lse = dh.distill_topk_forward(z, ids, val, temperature=t)
    got = dh.distill_topk_backward(z, ids, val, lse, temperature=t)
    # (results below the normal range are rounded to its spacing there, or flushed)
    close(got, ref[2], ref[3] + t * 7e-5 * e / S + 2.0 ** -126, "backward")
