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


def layer(N, K, seed=0):
    q, s, wv = quantise(weight(N, K, seed), 128)
    return dh.FP8BlockMatmul(q.contiguous(), s.contiguous()), wv


@pytest.mark.parametrize("M", [3, 40, 140])
@pytest.mark.parametrize("tx,ld,offset", [(BF, 272, 0), (BF, 273, 1), (HF, 300, 4), (F, 259, 3), (F, 264, 2)])
@pytest.mark.parametrize("ty,ldy,at", [(BF, 512, 0), (BF, 131, 1), (HF, 134, 2), (F, 133, 1), (F, 136, 4)])
def test_strides_and_given_results(M, tx, ld, offset, ty, ldy, at):
    N, K = 130, 256
    mm, wv = layer(N, K)
    x = rows(M, K, tx, ld=ld, offset=offset)
    buf = torch.full((M * ldy + at + 8,), 7.0, dtype=ty, device=DEV)
    y = torch.as_strided(buf, (M, N), (ldy, 1), at)
    assert mm(x, y) is y
    check(y, quantise(x, 1)[2], wv.t(), K)
    assert torch.equal(mm(x.contiguous(), out_dtype=ty), y)
    torch.as_strided(buf, (M, N), (ldy, 1), at).fill_(7.0)
    assert (buf == 7).all(), "something beside the rows was written"
    dx = torch.full((M, K + 3), 7.0, dtype=ty, device=DEV)
    mm.input_gradient(y.fill_(0.5), dx[:, :K])
    assert (dx[:, K:] == 7).all()
    assert torch.equal(dx[:, :K], mm.input_gradient(y.contiguous(), out_dtype=ty))


@pytest.mark.parametrize("M", [2, 33, 150])
def test_rows_that_are_not_finite_and_zeros(M):
    mm, wv = layer(300, 400)
    x = rows(M, 400, F)
    want = mm(x, out_dtype=F)
    x[0] = 0.0
    x[1, 399] = float("nan") if M != 33 else float("-inf")
    y = mm(x, out_dtype=F)
    assert y[1].isnan().all() and not y[0].any()
    assert torch.equal(y[2:], want[2:])
    dy = rows(M, 300, F)
    want = mm.input_gradient(dy, out_dtype=F)
    dy[0] = 1e-30                                     # below the smallest scale: zeros
    dy[1, 0] = float("inf")
    dx = mm.input_gradient(dy, out_dtype=F)
    assert dx[1].isnan().all() and dx[0].abs().max() <= 1e-12 and torch.equal(dx[2:], want[2:])


@pytest.mark.parametrize("M", [4, 40, 300])
@pytest.mark.parametrize("tx", [F, HF, BF])
def test_codes_at_ties(M, tx):
    """The activations' codes themselves, through a weight of ones on the diagonal: each result
    is a code times its scale, one product in 32 bits. Values at the ties between codes and next
    to them, over all of E4M3's binades."""
    K = 256
    eye = torch.zeros((K, K), dtype=torch.uint8, device=DEV)
    eye.fill_diagonal_(0x38)                          # 1.0
    mm = dh.FP8BlockMatmul(eye, torch.ones((2, 2), device=DEV))
    g = torch.Generator(DEV).manual_seed(M)
    amax = (torch.rand((M, 2, 1), generator=g, device=DEV) + 1.0) * 10.0 ** torch.randint(-3, 3, (M, 2, 1), generator=g, device=DEV)
    s = amax.to(tx).float() / torch.full_like(amax, 448.0)
    ties = torch.randint(1, 32, (M, 2, 128), generator=g, device=DEV) * 2.0 ** torch.randint(-10, 4, (M, 2, 128), generator=g, device=DEV)
    x = s * ties.float()
    x = (x.view(torch.int32) + torch.randint(-2, 3, x.shape, generator=g, device=DEV, dtype=torch.int32)).view(F)
    x *= torch.where(torch.rand(x.shape, generator=g, device=DEV) < 0.5, -1.0, 1.0)
    x[:, :, 5:6] = amax
    x = x.reshape(M, K).to(tx)
    codes, scales, _ = quantise(x, 1)
    y = mm(x, out_dtype=F)
    assert torch.equal(y, codes.float() * scales.repeat_interleave(128, 1)), (y / scales.repeat_interleave(128, 1) != codes.float()).nonzero()[:4].tolist()


def test_a_row_of_the_weight():
    """The gradient of one output feature is its row of the weight (1 is a code times a scale, to
    fp32's rounding), the output of one input feature its column."""
    mm, wv = layer(300, 400)
    one = torch.eye(300, device=DEV)[[0, 127, 128, 299]].contiguous()
    dx = mm.input_gradient(one, out_dtype=F)
    assert ((dx.double() - wv[[0, 127, 128, 299]]).abs() <= 2.0 ** -21 * wv[[0, 127, 128, 299]].abs()).all()
    one = torch.eye(400, device=DEV)[[0, 128, 399]].contiguous()
    y = mm(one, out_dtype=F)
    assert ((y.double() - wv[:, [0, 128, 399]].t()).abs() <= 2.0 ** -21 * wv[:, [0, 128, 399]].t().abs()).all()


@pytest.mark.parametrize("M,N,K", [(5, 19500, 8192), (16, 6000, 8192), (1, 70000, 256), (16, 19500, 2560), (33, 16000, 2560), (24, 1504, 1536)])
def test_few_tokens_on_many_tiles(M, N, K):
    """Clusters that exchange their sums for tile after tile."""
    mm, wv = layer(N, K)
    x = rows(M, K, BF)
    y = mm(x)
    check(y, quantise(x, 1)[2], wv.t(), K)
    for _ in range(3):
        assert torch.equal(mm(x), y)
    assert mm.device_error() == 0


@pytest.mark.parametrize("M,N,K,grad", [(200, 9000, 272, True), (150, 130, 6000, False), (129, 64026, 256, True), (16, 48, 70000, False),
                                        (100, 40000, 256, True), (20, 48, 30000, False)])
def test_long_contractions(M, N, K, grad):
    K = K // 16 * 16
    mm, wv = layer(N, K)
    x = rows(M, N if grad else K, BF)
    y = mm.input_gradient(x, out_dtype=F) if grad else mm(x, out_dtype=F)
    check(y, quantise(x, 1)[2], wv if grad else wv.t(), x.shape[1])


# wide tiles: one by one (three row blocks, which two by two would take a second round), two by two,
# and with an odd last row block; a round of whole tiles and the rest in parts of the contraction
@pytest.mark.parametrize("M,out,width", [(300, 12640, 272), (2000, 4608, 528), (1100, 4592, 272), (1000, 5104, 4000)])
@pytest.mark.parametrize("grad", [False, True])
def test_wide_tiles(M, out, width, grad):
    mm, wv = layer(*((width, out) if grad else (out, width)))
    x = rows(M, width, BF)
    check(mm.input_gradient(x, out_dtype=F) if grad else mm(x, out_dtype=F), quantise(x, 1)[2], wv if grad else wv.t(), width)


def test_no_tokens_and_float8_codes():
    q, s, wv = quantise(weight(64, 128), 128)
    mm = dh.FP8BlockMatmul(q.contiguous(), s.contiguous())
    raw = dh.FP8BlockMatmul(q.contiguous().view(torch.uint8), s.contiguous())
    x = rows(9, 128, BF)
    assert torch.equal(mm(x), raw(x))
    assert mm(x[:0]).shape == (0, 64) and mm.input_gradient(rows(1, 64, F)[:0]).shape == (0, 128)


def test_refusals():
    q, s, _ = quantise(weight(64, 128), 128)
    q, s = q.contiguous(), s.contiguous()
    mm = dh.FP8BlockMatmul(q, s)
    x = rows(4, 128, BF)
    for bad in (lambda: dh.FP8BlockMatmul(q.float(), s), lambda: dh.FP8BlockMatmul(q.t(), s), lambda: dh.FP8BlockMatmul(q, s.double()),
                lambda: dh.FP8BlockMatmul(q, s.expand(2, 1)), lambda: dh.FP8BlockMatmul(q.cpu(), s), lambda: mm(x[:, :112]), lambda: mm(x.t()),
                lambda: mm(x.double()), lambda: mm(x.cpu()), lambda: mm(x[0]), lambda: mm(x, out_dtype=torch.float64),
                lambda: mm(x, torch.empty((4, 65), device=DEV)), lambda: mm(x, torch.empty((64, 4), device=DEV).t()),
                lambda: mm.input_gradient(x), lambda: mm(x.float().requires_grad_()), lambda: mm.input_gradient(rows(4, 64, F).requires_grad_()),
                lambda: mm(x[:1].expand(4, 128)), lambda: mm(x, x[:, :64]), lambda: dh.fp8_quantize_blocks(weight(64, 128).float())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: dh.FP8BlockMatmul(q[:, :120].contiguous(), s), lambda: dh.FP8BlockMatmul(q[:0], s[:0]),
                lambda: dh.fp8_quantize_blocks(weight(64, 136))):
        with pytest.raises(dh.DraftHeadError):
            bad()
    assert mm(x).shape == (4, 64)


@pytest.mark.parametrize("M", [1, 300])
def test_offsets_past_32_bits_in_the_weight(M):
    N, K = 840_000, 2560
    q = torch.randint(0, 0x78, (N, K), dtype=torch.uint8, device=DEV)
    s = torch.rand((N // 128 + 1, 20), device=DEV) + 0.1
    mm = dh.FP8BlockMatmul(q, s)
    x = rows(M, K, BF)
    y = mm(x)
    for r in (0, 512_000, N - 1000):
        wv = q[r:r + 1000].view(torch.float8_e4m3fn).double() * s.double()[torch.arange(r, r + 1000, device=DEV) // 128].repeat_interleave(128, 1)
        check(y[:, r:r + 1000], quantise(x, 1)[2], wv.t(), K)


def test_offsets_past_32_bits_in_the_results():
    M, N, K = 40_000, 60_003, 16
    mm, wv = layer(N, K)
    x = rows(M, K, BF)
    y = mm(x)
    for r in (0, 35_700, M - 100):      # 35,700 x 60,003 is about 2^31
        check(y[r:r + 100], quantise(x[r:r + 100], 1)[2], wv.t(), K)


@pytest.mark.parametrize("M", [1, 16, 40, 200])
def test_graphs(M):
    mm, _ = layer(600, 2000)
    a, b = rows(M, 2000, BF), rows(M, 2000, BF, seed=9)
    want = [(mm(t), mm.input_gradient(mm(t))) for t in (a, b)]
    x = a.clone()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = mm(x)
            out = (y, mm.input_gradient(y))
        graphs.append((g, out))
    for i, t in ((0, a), (1, b), (0, a)):
        x.copy_(t)
        for g, _ in graphs:
            g.replay()
        for _, out in graphs:
            assert torch.equal(out[0], want[i][0]) and torch.equal(out[1], want[i][1])


def test_autograd():
    mm, wv = layer(300, 400)
    for M, tx in ((5, F), (150, BF)):
        x = rows(M, 400, tx).requires_grad_()
        y = dh.FP8BlockLinear.apply(x, mm, F)
        assert torch.equal(y, mm(x.detach(), out_dtype=F))
        up = rows(M, 300, F)
        (dx,) = torch.autograd.grad(y, x, up, create_graph=True)
        assert dx.dtype == tx and torch.equal(dx, mm.input_gradient(up, out_dtype=tx))
        with pytest.raises(RuntimeError, match="differentiable once"):
            (dx.float().square().sum() + x.float().sum()).backward()
        dh.FP8BlockLinear.apply(x, mm, F).sum().backward()          # an expanded gradient
        assert torch.equal(x.grad, mm.input_gradient(torch.ones((M, 300), device=DEV), out_dtype=tx))
        assert not dh.FP8BlockLinear.apply(x.detach(), mm).requires_grad
