"""The many-token NVFP4 product against the formula in 64 bits.

The activations' quantiser is defined in fp32 and checked bit for bit through
weights that pick single inputs. Products of codes and scales are exact; each of
the K / 64 instructions adds into the 32-bit accumulator, within 2^-22 of the
magnitudes it has summed, so |dy| <= (K / 64 + 1) 2^-22 sum |x' w'|, and y's type
rounds once (unit roundoff 2^-8, 2^-11, 2^-24) after a 32-bit scaling (two of 2^-24)."""
import numpy as np
import pytest
import torch

import nvfp4_draft_head_gb300 as dh
import oracle

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
E4M3 = np.array([(m / 8 * 2.0 ** -6) if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)])[:127]


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU test needs a CUDA device"
    from nvfp4_draft_head_gb300 import build
    build.build()


def nearest(v, grid):
    """Index of the nearest grid value, ties to the even index, saturating."""
    v = v.astype(np.float64)
    i = np.clip(np.searchsorted(grid, v), 1, len(grid) - 1)
    lo, hi = v - grid[i - 1], grid[i] - v
    return np.where(lo < hi, i - 1, np.where(lo > hi, i, i - 1 + (i - 1) % 2))


def quantized(x):
    """The activations' values (float64) by the recipe: decisions in fp32."""
    f = np.float32
    x = x.float().cpu().numpy()
    M, K = x.shape
    g = np.maximum(np.abs(x).max(1), f(1e-12)) / f(2688)
    b = np.abs(x).reshape(M, K // 16, 16)
    s = E4M3[nearest(b.max(2) / (f(6) * g)[:, None], E4M3)].astype(f)
    d = s * g[:, None]
    with np.errstate(divide="ignore", invalid="ignore"):
        a = np.where(d[..., None] == 0, f(0), b / d[..., None])
    v = np.copysign(GRID[nearest(a, GRID)], x.reshape(b.shape)) * s[..., None]
    return v.reshape(M, K).astype(np.float64) * g.astype(np.float64)[:, None]


def weight(N, K, seed):
    """Random codes and scales, and the values they stand for (without the global scale)."""
    rng = np.random.default_rng(seed)
    code = rng.integers(0, 16, (N, K), dtype=np.uint8)
    sf = rng.integers(0x28, 0x50, (N, K // 16), dtype=np.uint8)
    w = np.where(code & 8, -1.0, 1.0) * GRID[code & 7] * np.repeat(E4M3[sf], 16, axis=1)
    q = code[:, 0::2] | (code[:, 1::2] << 4)
    g = np.float32(rng.uniform(1e-4, 1e-3))
    return torch.from_numpy(q).cuda(), torch.from_numpy(sf).cuda(), torch.tensor([g], device="cuda"), w * np.float64(g)


def check(mm, x, w, out_dtype, y=None):
    got = mm(x, y, out_dtype=out_dtype)
    xq = quantized(x)
    xd, wd = torch.from_numpy(xq).cuda(), torch.from_numpy(w).cuda()
    ref, mag = xd @ wd.t(), xd.abs() @ wd.t().abs()
    tol = (mm.K / 64 + 1) * 2.0 ** -22 * mag + (EPS[got.dtype] + 2.0 ** -23) * ref.abs()
    if got.dtype == torch.float16:
        tol += 2.0 ** -25
        ref = ref.clamp(-1e6, 1e6)
    assert mm.device_error() == 0
    fin = ref.abs() < (65504.0 if got.dtype == torch.float16 else 1e38)
    err = (got.double() - ref).abs()
    assert (err <= tol)[fin].all(), float((err - tol)[fin].max())
    return got


def rand_x(M, K, dtype, seed, ld=None, offset=0):
    ld = ld or K
    buf = torch.full((offset + M * ld,), 5.0, dtype=dtype, device="cuda")
    x = torch.as_strided(buf, (M, K), (ld, 1), offset)
    v = torch.randn((M, K), generator=torch.Generator("cuda").manual_seed(seed), device="cuda")
    v[:, 3::41] *= 20
    return x.copy_(v)


@pytest.mark.parametrize("K", [16, 48, 256, 272, 1040, 2560])
@pytest.mark.parametrize("N", [64, 128, 320, 1088])
def test_shapes(N, K):
    q, sf, g, w = weight(N, K, N + K)
    mm = dh.NVFP4Matmul(q, sf, g)
    for i, M in enumerate([1, 7, 128, 129, 333]):
        name = ["bf16", "f16", "f32"][i % 3]
        check(mm, rand_x(M, K, TYPES[name], i), w, TYPES[["f32", "bf16", "f16"][i % 3]])


@pytest.mark.parametrize("xt", list(TYPES))
@pytest.mark.parametrize("yt", list(TYPES))
def test_types_and_strides(xt, yt):
    N, K, M = 192, 528, 150
    q, sf, g, w = weight(N, K, 5)
    mm = dh.NVFP4Matmul(q, sf, g)
    a = check(mm, rand_x(M, K, TYPES[xt], 1), w, TYPES[yt])
    for ld, offset, ldy, offy in ((K + 8, 0, N + 8, 0), (K + 1, 1, N + 3, 1), (K + 16, 4, N + 64, 4)):
        x = rand_x(M, K, TYPES[xt], 1, ld, offset)
        buf = torch.full((offy + M * ldy,), 9.0, dtype=TYPES[yt], device="cuda")
        y = torch.as_strided(buf, (M, N), (ldy, 1), offy)
        assert torch.equal(check(mm, x, w, TYPES[yt], y), a)
        pad = torch.as_strided(buf, (M - 1, ldy - N), (ldy, 1), offy + N)
        assert (pad == 9.0).all() and (buf[:offy] == 9.0).all()


def test_larger_products_and_several_tiles_per_sm():
    q, sf, g, w = weight(20032, 512, 3)
    mm = dh.NVFP4Matmul(q, sf, g)
    check(mm, rand_x(1500, 512, torch.bfloat16, 2), w, torch.bfloat16)
    check(mm, rand_x(700, 512, torch.bfloat16, 3), w, torch.float32)


def one_hot(K):
    """NVFP4 weight whose row n picks input n: code 1.0, scale 1.0."""
    code = np.zeros((K, K), dtype=np.uint8)
    code[np.arange(K), np.arange(K)] = 2
    sf = np.full((K, K // 16), 0x38, dtype=np.uint8)
    q = torch.from_numpy(code[:, 0::2] | (code[:, 1::2] << 4)).cuda()
    return dh.NVFP4Matmul(q, torch.from_numpy(sf).cuda(), torch.ones(1, device="cuda"))


def test_quantiser_bit_exact():
    K = 512
    mm = one_hot(K)
    rng = np.random.default_rng(1)
    rows = [rng.standard_normal(K) * 10.0 ** e for e in (-30, -13, -8, -3, 0, 3, 20)]
    rows += [np.zeros(K), np.full(K, 1e-14), rng.integers(-96, 97, K) / 16.0,          # zero, below the floor, ties
             rng.standard_normal(K) * np.exp(rng.uniform(-20, 0, K)), np.repeat(2.0 ** -np.arange(32), 16) * 6.0]
    x = torch.from_numpy(np.stack(rows).astype(np.float32)).cuda()
    for dtype in (torch.float32, torch.bfloat16):
        xt = x.to(dtype)
        y = mm(xt, out_dtype=torch.float32)
        ref = torch.from_numpy(quantized(xt)).cuda().float()
        assert torch.equal(y, ref), (y - ref).abs().max()
    xh = x[2:6].half()
    assert torch.equal(mm(xh, out_dtype=torch.float32), torch.from_numpy(quantized(xh)).cuda().float())


def test_rows_that_are_not_finite_stay_alone():
    K, N = 256, 128
    q, sf, g, w = weight(N, K, 8)
    mm = dh.NVFP4Matmul(q, sf, g)
    x = rand_x(6, K, torch.bfloat16, 1)
    clean = mm(x, out_dtype=torch.float32)
    x[1, 7], x[2, 255], x[4, 0] = float("nan"), float("inf"), float("-inf")
    y = mm(x, out_dtype=torch.float32)
    assert y[[1, 2, 4]].isnan().all() and torch.equal(y[[0, 3, 5]], clean[[0, 3, 5]])
    # a token's result does not depend on the batch around it
    assert torch.equal(mm(x[3:4], out_dtype=torch.float32), clean[3:4])


def test_matches_the_head_built_from_bf16_rows():
    V, K = 4096, 256
    W = (torch.randn((V, K), generator=torch.Generator("cuda").manual_seed(1), device="cuda") * 0.02).bfloat16()
    keep = np.zeros(V, np.uint8)
    keep[np.random.default_rng(0).permutation(V)[:1000]] = 1
    idx, n = dh.draft_head_build_index(keep)
    idx = torch.from_numpy(idx).cuda()
    mm = dh.NVFP4Matmul.from_weight(W, idx)
    qo, so, go = oracle.nvfp4_quantize(W.cpu().view(torch.int16).numpy().view(np.uint16), idx.cpu().numpy())
    code = np.stack([qo & 15, qo >> 4], -1).reshape(len(idx), K)
    w = np.where(code & 8, -1.0, 1.0) * GRID[code & 7] * np.repeat(E4M3[so], 16, axis=1) * np.float64(np.asarray(go).reshape(-1)[0])
    check(mm, rand_x(40, K, torch.bfloat16, 4), w, torch.float32)


def test_streams_graphs_and_repeats():
    N, K, M = 2560, 1024, 300
    q, sf, g, w = weight(N, K, 2)
    mm = dh.NVFP4Matmul(q, sf, g)
    x = rand_x(M, K, torch.bfloat16, 6)
    a = check(mm, x, w, torch.bfloat16)
    for _ in range(4):
        assert torch.equal(mm(x), a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = mm(x, stream=s)
    s.synchronize()
    assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = mm(x)
    x.copy_(x.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(c, a.flip(0))


def test_refusals():
    q, sf, g, _ = weight(64, 32, 1)
    mm = dh.NVFP4Matmul(q, sf, g)
    assert mm(torch.empty((0, 32), device="cuda")).shape == (0, 64)
    for bad in (torch.zeros((2, 48), device="cuda"), torch.zeros((2, 32)), torch.zeros((2, 32), device="cuda").double(),
                torch.zeros(32, device="cuda"), torch.zeros((32, 2), device="cuda").t(), torch.zeros((1, 32), device="cuda").expand(2, 32)):
        with pytest.raises(ValueError):
            mm(bad)
    x = torch.zeros((2, 32), device="cuda")
    with pytest.raises(ValueError):
        mm(x, out_dtype=torch.float64)
    with pytest.raises(ValueError):
        mm(x, torch.zeros((2, 63), device="cuda"))
    for args in ((q[:, :15], sf, g), (q, sf[:, :1], g), (q, sf, torch.ones(2, device="cuda")), (q.int(), sf, g), (q.cpu(), sf, g)):
        with pytest.raises(ValueError):
            dh.NVFP4Matmul(*args)
    with pytest.raises(dh.DraftHeadError):
        dh.NVFP4Matmul(*weight(96, 32, 1)[:3])   # N % 64 != 0


@pytest.mark.parametrize("M, N, K, yt, ldy", [
    (600, 29440, 272, "bf16", 0), (513, 29504, 48, "f32", 0), (640, 29632, 1040, "f16", 0),
    (129, 87808, 16, "bf16", 0), (600, 29440, 528, "bf16", 29443)])
def test_many_tiles(M, N, K, yt, ldy):
    """Products of several rounds of the largest tiles, with ragged last tiles in
    both directions; a token's result is that of a call of its own."""
    q, sf, g, w = weight(N, K, M)
    mm = dh.NVFP4Matmul(q, sf, g)
    x = rand_x(M, K, torch.bfloat16, 3)
    y = torch.empty((M, ldy), dtype=TYPES[yt], device="cuda")[:, :N] if ldy else None
    got = check(mm, x, w, TYPES[yt], y)
    for rows in (slice(0, 3), slice(M - 2, M)):
        assert torch.equal(mm(x[rows], out_dtype=TYPES[yt]), got[rows])
