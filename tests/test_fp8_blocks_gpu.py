"""FP8 product with a scale per block of 128 (and its gradient in the input) against a plain
implementation in 64 bits.

The quantiser's decisions are fp32 (IEEE division) and compared by their result: the reference
quantises with the same recipe in torch. After it, products of codes are exact; a block's sum of
128 has 127 additions, each off by at most 2^-23 of the magnitudes summed (truncation
included), the scales' product and the multiply-add into the B blocks' sum by 2^-24 each:
  |error| <= (130 + B) 2^-23 sum |x'| |w'| + u |y|,
u half a step of y's type (bf16 2^-8, f16 2^-11, f32 2^-24); f16 results below its range add one
subnormal step.
"""
import pytest
import torch

import nvfp4_draft_head_gb300 as dh

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, HF, F = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from nvfp4_draft_head_gb300 import build
    build.build()


def blocks(x, rows):
    r, c = x.shape
    x = torch.nn.functional.pad(x, (0, -c % 128, 0, -r % rows))
    return x.view(x.shape[0] // rows, rows, x.shape[1] // 128, 128)


def quantise(x, rows):
    """(codes, scales, values in 64 bits) of x, one scale per rows x 128."""
    b = blocks(x.float(), rows)
    amax = b.abs().amax((1, 3), keepdim=True)
    s = torch.clamp(amax, min=1e-12) / torch.full_like(amax, 448.0)
    s = torch.where(torch.isfinite(amax), s, torch.full_like(s, float("nan")))
    q = torch.clamp(b / s, -448.0, 448.0).to(torch.float8_e4m3fn)
    v = (q.double() * s.double()).reshape(b.shape[0] * rows, -1)[:x.shape[0], :x.shape[1]]
    return q.reshape(b.shape[0] * rows, -1)[:x.shape[0], :x.shape[1]], s[:, 0, :, 0], v


def weight(N, K, seed=0, decades=True):
    g = torch.Generator(DEV).manual_seed(seed + 3 * N + K)
    w = torch.randn((N, K), generator=g, device=DEV) * 0.02
    if decades:   # blocks of very different scales
        w *= (10.0 ** (torch.arange(-(-K // 128), device=DEV) % 5 - 2)).repeat_interleave(128)[:K]
        w *= (3.0 ** (torch.arange(-(-N // 128), device=DEV) % 3 - 1)).repeat_interleave(128)[:N, None]
    return w.bfloat16()


def rows(M, width, dtype, seed=0, ld=None, offset=0):
    g = torch.Generator(DEV).manual_seed(seed + 11 * M + width)
    ld = width if ld is None else ld
    buf = torch.full((M * ld + offset + 16,), float("nan"), dtype=dtype, device=DEV)
    x = torch.as_strided(buf, (M, width), (ld, 1), offset)
    x.copy_(torch.randn((M, width), generator=g, device=DEV) * (1 + 9 * (torch.arange(width, device=DEV) % 37 == 0)))
    return x


def check(y, xv, wv, width):
    want, mag = xv @ wv, xv.abs() @ wv.abs()
    u = torch.finfo(y.dtype).eps / 2
    tol = (130 + -(-width // 128)) * 2.0 ** -23 * mag + u * want.abs() + (2.0 ** -24 if y.dtype == HF else 1e-38)
    bad = ~((y.double() - want).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {((y.double() - want).abs() / tol).nan_to_num(9e9).max().item():.3g}, " \
                          f"first at {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("N,K", [(1, 16), (64, 128), (127, 144), (130, 512), (257, 1040), (4608, 2560)])
def test_weight_blocks(N, K):
    W = weight(N + 7, K)
    idx = torch.randperm(N + 7, device=DEV)[:N].to(torch.int32)
    q, s = dh.fp8_quantize_blocks(W, idx)
    rq, rs, _ = quantise(W[idx.long()], 128)
    assert torch.equal(q, rq.view(torch.uint8)) and torch.equal(s, rs)
    q, s = dh.fp8_quantize_blocks(W[:N])
    rq, rs, _ = quantise(W[:N], 128)
    assert torch.equal(q, rq.view(torch.uint8)) and torch.equal(s, rs)


def test_weight_of_zeros_and_an_id_out_of_range():
    W = torch.zeros((130, 256), dtype=BF, device=DEV)
    q, s = dh.fp8_quantize_blocks(W)
    assert not q.any() and torch.equal(s, torch.full_like(s, float(torch.tensor(1e-12) / torch.tensor(448.0))))
    with pytest.raises(RuntimeError, match="dh_idx"):
        dh.fp8_quantize_blocks(W, torch.tensor([0, 130], dtype=torch.int32, device=DEV))


SIZES = [(1, 1, 16), (1, 4608, 2560), (2, 130, 144), (5, 64, 4096), (16, 2560, 5120), (17, 257, 272), (33, 1000, 512), (64, 515, 1040), (100, 4000, 256),
         (129, 255, 128), (256, 256, 2560), (300, 1023, 2320), (517, 4608, 2560)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("tx,ty", [(BF, BF), (HF, F), (F, HF)])
def test_forward(M, N, K, tx, ty):
    q, s, wv = quantise(weight(N, K), 128)
    mm = dh.FP8BlockMatmul(q.contiguous(), s.contiguous())
    x = rows(M, K, tx)
    y = mm(x, out_dtype=ty)
    check(y, quantise(x, 1)[2], wv.t(), K)
    assert torch.equal(mm(x, out_dtype=ty), y)
    assert mm.device_error() == 0


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("tx,ty", [(BF, BF), (F, F), (HF, HF)])
def test_input_gradient(M, N, K, tx, ty):
    q, s, wv = quantise(weight(N, K), 128)
    mm = dh.FP8BlockMatmul(q.contiguous(), s.contiguous())
    dy = rows(M, N, tx)
    dx = mm.input_gradient(dy, out_dtype=ty)
    check(dx, quantise(dy, 1)[2], wv, N)
    assert torch.equal(mm.input_gradient(dy, out_dtype=ty), dx)
    assert mm.device_error() == 0
