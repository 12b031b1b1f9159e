"""Token log-probabilities and distillation against plain formulas in 64 bits.

Tolerances (derived, not fitted). A probability term 2^((z - m) c) carries the
rounding of its exponent (two roundings of |x| <= 40: 40 * 2^-23 * ln 2 ~ 3.3e-6)
and the exponential's own (2^-22); a thread adds at most a few hundred terms in
sequence (each addition 2^-24 of the partial sum), the rest is a tree: the sum S
is within 2e-5 of itself, and ln S within 2e-5. A log-probability adds the
rounding of (z - max) / t, three of 2^-24, relative: 2e-5 + 5e-7 |log p|. The
entropy's second term is a mean of |(z - max) / t| with the relative error of S.
Whole numbers (ids) are exact: the kernel orders the logits themselves."""
import math

import pytest
import torch

import nvfp4_draft_head_gb300 as dh

pytestmark = pytest.mark.gpu

NEG = float("-inf")
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
# unit roundoffs: 8, 11 and 24 significant bits
EPS = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU test needs a CUDA device"
    from nvfp4_draft_head_gb300 import build
    build.build()


def rand_rows(M, n, dtype, seed, ld=None, offset=0, scale=3.0):
    """[M, n] logits inside a larger buffer: row stride ld, first element `offset` in."""
    ld = n if ld is None else ld
    g = torch.Generator("cuda").manual_seed(seed)
    buf = torch.full((offset + M * ld,), 99.0, dtype=dtype, device="cuda")
    z = torch.as_strided(buf, (M, n), (ld, 1), offset)
    z.copy_(torch.randn((M, n), generator=g, device="cuda") * scale)
    return z


def close(x, ref, tol, what=""):
    """Equal infinities and NaNs, and finite values within tol."""
    x, ref = x.double(), ref.double()
    tol = torch.as_tensor(tol, device=ref.device, dtype=torch.float64).expand_as(ref)
    assert torch.equal(x.isnan(), ref.isnan()), f"{what}: NaNs differ"
    inf = ref.isinf() & ~ref.isnan()
    assert torch.equal(x[inf], ref[inf]) and not x[~inf & ~ref.isnan()].isinf().any(), f"{what}: infinities differ"
    fin = ref.isfinite()
    bad = (x - ref).abs()[fin] > tol[fin]
    assert not bad.any(), f"{what}: {int(bad.sum())} off, worst {float(((x - ref).abs()[fin] - tol[fin]).max()):.3g} past"


def columns(ids, n, row_of):
    ids = ids.long()
    if row_of is not None:
        ok = (ids >= 0) & (ids < row_of.numel())
        ids = torch.where(ok, row_of[ids.clamp(0, row_of.numel() - 1)].long(), -1)
    return ids.clamp(0, n - 1), (ids >= 0) & (ids < n)


def ref_stats(z, t):
    z = z.double()
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == NEG, 0.0, m)
    d = (z - m) / t
    e = d.exp()
    return m, d, e, e.sum(-1, keepdim=True)


def check_logprobs(z, tokens, k, t=1.0, idx=None, row_of=None, **kw):
    r = dh.token_logprobs(z, tokens, top_k=k, temperature=t, idx=idx, row_of=row_of, **kw)
    torch.cuda.synchronize()
    M, n = z.shape
    m, d, e, S = ref_stats(z, t)
    empty = S == 0
    close(r.lse, torch.where(empty, NEG, m / t + S.log())[:, 0], 2e-5 + 5e-7 * (m / t).abs()[:, 0].nan_to_num(0, 0, 0), "lse")
    mean = (torch.where(e == 0, 0.0, e * d)).sum(-1, keepdim=True) / S
    close(r.entropy, torch.where(empty, 0.0, S.log() - mean)[:, 0], (2e-5 * (2 + mean.abs()))[:, 0].nan_to_num(1), "entropy")
    if tokens is not None:
        tok = tokens.view(M, -1)
        col, there = columns(tok, n, row_of)
        ref = torch.where(there & ~empty, d.gather(1, col) - S.log(), NEG)
        assert r.logp.shape == tokens.shape
        close(r.logp.view(M, -1), ref.float(), 2e-5 + 5e-7 * ref.abs().nan_to_num(0, 0, 0), "logp")
    val, at = torch.sort(z.float(), dim=1, descending=True, stable=True)
    val, at = val[:, :k], at[:, :k]
    none = val == NEG
    ids = torch.where(none, -1, at.int() if idx is None else idx[at])
    top = torch.where(none, NEG, (val.double() - m) / t - S.log())
    pad = k - ids.shape[1]
    ids = torch.nn.functional.pad(ids, (0, pad), value=-1)
    top = torch.nn.functional.pad(top, (0, pad), value=NEG)
    assert torch.equal(r.top_ids, ids.int()), "top ids"
    close(r.top_logp, top.float(), 2e-5 + 5e-7 * top.abs().nan_to_num(0, 0, 0), "top logp")
    return r


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("n", [1, 2, 7, 9, 100, 1023, 1025, 4001, 20011, 64026])
def test_logprobs_sizes(dtype, n):
    for i, (M, k, extra, offset) in enumerate([(1, 5, 0, 0), (3, 20, 38, 0), (17, 128, 1, 3), (330, 1, 3, 1)]):
        z = rand_rows(M, n, TYPES[dtype], 10 * n + i, n + extra, offset)
        g = torch.Generator("cuda").manual_seed(i)
        tokens = torch.randint(-1, n + 1, (M, 2), generator=g, device="cuda", dtype=torch.int32)
        check_logprobs(z, tokens, k, t=[1.0, 0.7, 2.0, 1.3][i])


@pytest.mark.parametrize("M", [1, 2, 5, 40])
def test_logprobs_full_vocabulary_rows(M):
    z = rand_rows(M, 248_320, torch.float32, M)
    off = torch.rand(248_320, generator=torch.Generator("cuda").manual_seed(5), device="cuda") < 0.74
    z[:, off] = NEG
    check_logprobs(z, z.argmax(-1).int(), 20)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("n", [700, 4001, 30000, 200003])
def test_logprobs_masks_ties_and_orders(dtype, n):
    T = TYPES[dtype]
    rows = [
        torch.full((n,), NEG),                                    # nothing left
        torch.full((n,), float(torch.finfo(T).min)),              # all at the type's lowest value
        torch.full((n,), 1.5),                                    # all equal
        torch.linspace(-30, 30, n),                               # ascending
        torch.linspace(30, -30, n),                               # descending
        (torch.arange(n) % 3).float(),                            # three values
        torch.where(torch.arange(n) == n - 1, 2.0, NEG),          # one column left, the last
        torch.where(torch.arange(n) % 97 == 5, 0.25, NEG),        # few left, equal
        torch.where(torch.arange(n) % 512 == 9, torch.arange(n) / n + 8.0, torch.zeros(n)),   # large ones at one stride
        torch.where(torch.arange(n) % 4096 < 8, 5.0, -torch.ones(n)),
        torch.where(torch.arange(n) < 3, 0.0, float(torch.finfo(T).min) * torch.ones(n)),
        torch.where(torch.arange(n) % 2 == 0, 0.0, -0.0 * torch.ones(n)),
    ]
    z = torch.stack(rows).to("cuda").to(T)
    tokens = torch.tensor([[0, n - 1, n // 2]] * len(rows), dtype=torch.int32, device="cuda")
    for k in (1, 20, 128):
        check_logprobs(z, tokens, k)
    check_logprobs(z[:1], tokens[:1], 20)      # one row over several CTAs
    check_logprobs(z[2:3], tokens[:1], 128)
    check_logprobs(z[5:6], tokens[:1], 33, t=0.25)


@pytest.mark.parametrize("n", [50, 5000, 120000])
def test_logprobs_nan_and_infinity(n):
    z = rand_rows(6, n, torch.float32, 3)
    z[1, n // 3] = float("nan")
    z[2, n - 1] = float("inf")
    z[3, :] = float("nan")
    z[4, ::2] = NEG
    z[4, 1] = float("nan")
    z[5, [2, 7]] = float("inf")
    tokens = torch.tensor([[1, n - 1]] * 6, dtype=torch.int32, device="cuda")
    check_logprobs(z, tokens, 20)


def test_logprobs_large_magnitudes():
    for dtype, s in ((torch.float32, 1e30), (torch.float32, 3e38), (torch.float16, 2e4), (torch.bfloat16, 1e37)):
        z = (torch.rand((5, 3001), generator=torch.Generator("cuda").manual_seed(1), device="cuda") * 2 - 1) * s
        check_logprobs(z.to(dtype), None, 9)
    z = rand_rows(4, 5000, torch.float32, 8) + 1000.0
    r = dh.token_logprobs(z, None, top_k=3)
    m, d, e, S = ref_stats(z, 1.0)
    close(r.entropy, (S.log() - (e * d).sum(-1, keepdim=True) / S)[:, 0], 2e-4, "entropy far from zero")


def test_logprobs_ids_through_the_head_index():
    V, n = 9000, 3777
    kept = torch.randperm(V, generator=torch.Generator().manual_seed(2))[:n].sort().values
    idx = torch.cat([kept, kept[:1].expand((-n) % 64)]).int().cuda()
    row_of = dh.draft_head_row_map(idx, n, V)
    ref = torch.full((V,), -1, dtype=torch.int32)
    ref[kept] = torch.arange(n, dtype=torch.int32)
    assert torch.equal(row_of.cpu(), ref)
    z = rand_rows(9, idx.numel(), torch.bfloat16, 4)[:, :n]
    tokens = torch.tensor([int(kept[5]), int(kept[-1]), -3, V, V + 100, 2 ** 31 - 1,
                           int((ref < 0).nonzero()[0]), int(kept[0]), 0], dtype=torch.int32, device="cuda")
    check_logprobs(z, tokens, 20, idx=idx, row_of=row_of)


def test_logprobs_past_32_bit_offsets():
    M, n = 3, 1000
    ld = 2 ** 30 + 8     # the last row starts past 2^31 elements
    buf = torch.empty(2 * ld + n, dtype=torch.bfloat16, device="cuda")
    z = torch.as_strided(buf, (M, n), (ld, 1))
    z.copy_(torch.randn((M, n), generator=torch.Generator("cuda").manual_seed(3), device="cuda"))
    check_logprobs(z, None, 7)
    ids = torch.randint(0, n, (M, 1), device="cuda", dtype=torch.int32)
    loss, dz = dh.distill_topk(z, ids, torch.zeros((M, 1), device="cuda"), dlogits=z.clone())
    g = ref_stats(z, 1.0)
    close(dz, (g[2] / g[3]).scatter_add(1, ids.long(), -torch.ones((M, 1), device="cuda", dtype=torch.double)), 1e-2, "gradient")


def test_logprobs_repeat_streams_and_graphs():
    z = rand_rows(7, 64_026, torch.bfloat16, 5, 64_064)
    tokens = z.float().argmax(-1).int()
    a = check_logprobs(z, tokens, 20)
    for _ in range(3):
        b = dh.token_logprobs(z, tokens, top_k=20)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c = dh.token_logprobs(z, tokens, top_k=20, stream=s)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, c))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d = dh.token_logprobs(z, tokens, top_k=20)
    z.copy_(z.flip(1))
    graph.replay()
    torch.cuda.synchronize()
    e = dh.token_logprobs(z, tokens, top_k=20)
    assert all(torch.equal(x, y) for x, y in zip(d, e))


def test_empty_batches():
    z = torch.empty((0, 100), device="cuda")
    r = dh.token_logprobs(z, torch.empty((0, 2), dtype=torch.int32, device="cuda"), top_k=3)
    assert r.logp.shape == (0, 2) and r.top_ids.shape == (0, 3) and r.lse.shape == (0,)
    ids, val = torch.empty((0, 4), dtype=torch.int32, device="cuda"), torch.empty((0, 4), device="cuda")
    loss, dz = dh.distill_topk(z, ids, val)
    assert loss.shape == (0,) and dz.shape == (0, 100)


# ---------------------------------------------------------------- distillation --

def ref_distill(z, ids, val, t, w, row_of):
    n = z.shape[1]
    m, d, e, S = ref_stats(z, t)
    q = e / S
    col, there = columns(ids, n, row_of)
    zc = z.double().gather(1, col)
    v = val.double()
    w = torch.ones(z.shape[0], device="cuda", dtype=torch.double) if w is None else w.double()
    w = w[:, None]
    there = there & (zc != NEG) & (v != NEG) & (w != 0)
    some = there.any(-1, keepdim=True)
    _, dt, et, St = ref_stats(torch.where(there, v, NEG), t)
    p = torch.where(there, et / St, 0.0)
    diff = torch.where(p == 0, 0.0, dt - St.log() - ((zc - m) / t - S.log()))
    loss = torch.where(some, w * t * t * (p * diff).sum(-1, keepdim=True), 0.0)[:, 0]
    # an exponent's rounding, S and the teacher's sum: 2e-5 each; p and the difference of logarithms
    loss_tol = (w.abs() * t * t * (4e-5 + (p * (1e-6 * (d.gather(1, col).abs().nan_to_num(0, 0, 0) + dt.abs().nan_to_num(0, 0, 0))
                                                + 2e-5 * diff.abs())).sum(-1, keepdim=True)))[:, 0]
    psum = torch.zeros_like(q).scatter_add(1, col, p)
    grad = torch.where(some, w * t * (q - psum), 0.0)
    grad_tol = w.abs() * t * 2e-5 * (q.abs() + psum.abs()) + EPS[z.dtype] * grad.abs()
    grad_tol += 2.0 ** -25 if z.dtype == torch.float16 else 1e-37   # half the type's spacing near zero; flushed subnormals
    lse = torch.where(S == 0, NEG, m / t + S.log())[:, 0]
    return loss, loss_tol.nan_to_num(1.0), grad, grad_tol.nan_to_num(1.0), lse


def check_distill(z, ids, val, t=1.0, w=None, row_of=None):
    loss, loss_tol, grad, grad_tol, lse = ref_distill(z, ids, val, t, w, row_of)
    l, g = dh.distill_topk(z, ids, val, temperature=t, weights=w, row_of=row_of)
    torch.cuda.synchronize()
    close(l, loss, loss_tol, "loss")
    close(g, grad, grad_tol, "gradient")
    lf, lsef = dh.distill_topk_forward(z, ids, val, temperature=t, weights=w, row_of=row_of)
    assert torch.equal(lf.nan_to_num(7.0), l.nan_to_num(7.0))
    big = lse.abs().nan_to_num(0, 0, 0)
    close(lsef, lse, 2e-5 + 5e-7 * big, "lse")
    gb = dh.distill_topk_backward(z, ids, val, lsef, w, temperature=t, row_of=row_of)
    # q = e^(z/t - lse): lse is rounded to 32 bits (2^-24 |lse| in the exponent)
    extra = (w.double().abs() if w is not None else torch.ones_like(lse)) * t * (2e-5 + 3e-7 * big)
    close(gb, grad, grad_tol + extra[:, None] * (ref_stats(z, t)[2] / ref_stats(z, t)[3]).nan_to_num(0), "backward")
    # in place (in a copy at the same offset from a 16-byte boundary, which sets the order of the sums)
    M, n = z.shape
    whole = torch.empty(z.storage_offset() + M * z.stride(0) + n, dtype=z.dtype, device="cuda")
    buf = torch.as_strided(whole, (M, n), (z.stride(0), 1), z.storage_offset()).copy_(z)
    l2, g2 = dh.distill_topk(buf, ids, val, temperature=t, weights=w, row_of=row_of, dlogits=buf)
    assert g2.data_ptr() == buf.data_ptr() and torch.equal(g2.nan_to_num(7.0), g.nan_to_num(7.0)) and torch.equal(l2.nan_to_num(7.0), l.nan_to_num(7.0))
    return l, g


def teacher(z, K, seed):
    M, n = z.shape
    g = torch.Generator("cuda").manual_seed(seed)
    near = z.float().nan_to_num(-20.0, neginf=-20.0) + torch.randn((M, n), generator=g, device="cuda")
    k = min(K, n)
    val, ids = near.topk(k, dim=1)
    ids = torch.nn.functional.pad(ids, (0, K - k), value=-1).int()
    return ids.contiguous(), torch.nn.functional.pad(val, (0, K - k), value=NEG).contiguous()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("n", [1, 3, 8, 100, 1031, 4001, 64026])
def test_distill_sizes(dtype, n):
    for i, (M, K, extra, offset) in enumerate([(1, 1, 0, 0), (3, 20, 38, 0), (17, 128, 1, 3), (310, 7, 3, 1), (2, 512, 0, 0)]):
        z = rand_rows(M, n, TYPES[dtype], 100 * n + i, n + extra, offset)
        ids, val = teacher(z, K, i)
        w = torch.rand(M, generator=torch.Generator("cuda").manual_seed(i), device="cuda") + 0.25
        if M > 2:
            w[1] = 0.0
        check_distill(z, ids, val.to([torch.float32, torch.bfloat16, torch.float16][i % 3]), t=[1.0, 2.0, 0.5, 1.0, 4.0][i],
                      w=None if i == 0 else w)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [600, 30011, 248320])
def test_distill_masks(dtype, n):
    T = TYPES[dtype]
    z = rand_rows(8, n, T, n)
    z[0] = NEG                                             # student masked throughout
    z[1, ::2] = NEG
    z[2] = float(torch.finfo(T).min)
    z[3, 1:] = float(torch.finfo(T).min)
    ids, val = teacher(z, 16, 1)
    ids[1, :4] = torch.tensor([0, 2, 1, 3])                # two on masked columns
    val[4] = NEG                                           # teacher row masked throughout
    val[5, 3:] = NEG
    ids[6] = -1                                            # nothing on the student's vocabulary
    ids[7, 5:] = n + 3
    ids[5, 1] = ids[5, 0]                                  # one column named twice
    ids[3, 2:9] = ids[3, 2]
    check_distill(z, ids, val)
    check_distill(z, ids, val, t=2.0, w=torch.tensor([1, 2, .5, 1, 1, -1, 1, 3.0], device="cuda"))


def test_distill_nan_and_infinity():
    z = rand_rows(5, 3000, torch.float32, 3)
    ids, val = teacher(z, 8, 1)
    z[0, 77] = float("nan")
    z[1, 5] = float("inf")
    val[2, 3] = float("nan")
    w = torch.tensor([1.0, 1.0, 1.0, 0.0, 1.0], device="cuda")
    z[3] = float("nan")                                    # a row left out stays out
    l, g = check_distill(z, ids, val, w=w)
    assert l[3] == 0 and (g[3] == 0).all() and torch.isfinite(g[4]).all()


def test_distill_through_the_head_index_and_autograd():
    V, n, M, K = 5000, 1999, 21, 12
    kept = torch.randperm(V, generator=torch.Generator().manual_seed(2))[:n].sort().values.int().cuda()
    row_of = dh.draft_head_row_map(kept, n, V)
    z = rand_rows(M, n, torch.float32, 6).requires_grad_()
    ids = torch.stack([torch.randperm(V, generator=torch.Generator().manual_seed(i))[:K] for i in range(M)]).int().cuda()
    val = torch.randn((M, K), generator=torch.Generator("cuda").manual_seed(3), device="cuda") * 2
    w = torch.rand(M, generator=torch.Generator("cuda").manual_seed(4), device="cuda")
    check_distill(z.detach(), ids, val, t=1.5, w=w, row_of=row_of)
    up = torch.rand(M, generator=torch.Generator("cuda").manual_seed(5), device="cuda")
    loss = dh.DistillTopK.apply(z, ids, val, 1.5, w, row_of)
    (loss * up).sum().backward()
    ref = ref_distill(z.detach(), ids, val, 1.5, w * up, row_of)
    close(z.grad, ref[2], ref[3] + 1e-6, "autograd")


@pytest.mark.parametrize("t", [1.0, 2.0])
def test_distill_gradient_against_differences(t):
    """Central differences of the kernel's own loss along random sign vectors v,
    step h = 2^-4: the loss is off by at most 4e-5 t^2 (noise 4e-5 t^2 / h) and
    the third derivative of t^2 log-sum-exp(z / t) along |v| <= 1 is at most 1 / t."""
    M, n, K, h = 6, 50, 9, 2.0 ** -4
    z = rand_rows(M, n, torch.float32, 9)
    ids, val = teacher(z, K, 2)
    _, g = dh.distill_topk(z, ids, val, temperature=t)
    for s in range(5):
        v = torch.randint(0, 2, (M, n), generator=torch.Generator("cuda").manual_seed(s), device="cuda") * 2.0 - 1.0
        lp, lm = (dh.distill_topk_forward(z + x * h * v, ids, val, temperature=t)[0] for x in (1, -1))
        close((lp - lm) / (2 * h), (g * v).sum(1), 4e-5 * t * t / h + h * h / (6 * t) + 1e-4, "difference")


def test_distill_pads_are_left_alone_and_rows_repeat():
    M, n, ld = 9, 1001, 1040
    buf = torch.full((M, ld), 3.0, dtype=torch.bfloat16, device="cuda")
    z = rand_rows(M, n, torch.bfloat16, 1, 1008)
    ids, val = teacher(z, 8, 3)
    l, g = dh.distill_topk(z, ids, val, dlogits=buf[:, :n])
    assert (buf[:, n:] == 3.0).all() and g.data_ptr() == buf.data_ptr()
    l2, g2 = dh.distill_topk(z, ids, val)
    assert torch.equal(l, l2) and torch.equal(g, g2)
    # rows at another offset from a 16-byte boundary than the logits'
    odd = torch.full((M * 1013 + 1,), 3.0, dtype=torch.bfloat16, device="cuda")
    g3 = dh.distill_topk(z, ids, val, dlogits=torch.as_strided(odd, (M, n), (1013, 1), 1))[1]
    assert torch.equal(g, g3)


def test_refusals():
    z = torch.zeros((4, 64), device="cuda")
    ids, val = torch.zeros((4, 2), dtype=torch.int32, device="cuda"), torch.zeros((4, 2), device="cuda")
    for bad in (z.double(), z.cpu(), z[0], z.t(), z.expand(4, 64)[:, ::2], z[:1].expand(4, 64)):
        with pytest.raises(ValueError):
            dh.token_logprobs(bad)
    for kw in (dict(tokens=torch.zeros(4, device="cuda")), dict(tokens=torch.zeros(3, dtype=torch.int32, device="cuda")),
               dict(tokens=torch.zeros(4, dtype=torch.int64, device="cuda")), dict(top_k=129), dict(top_k=-1),
               dict(idx=torch.zeros(63, dtype=torch.int32, device="cuda")), dict(row_of=torch.zeros(9, device="cuda")),
               dict(tokens=torch.zeros(4, dtype=torch.int32))):
        with pytest.raises(ValueError):
            dh.token_logprobs(z, **kw)
    for t in (0.0, -1.0, math.nan, math.inf, 1e-45):
        with pytest.raises(dh.DraftHeadError) as e:
            dh.token_logprobs(z, temperature=t)
        assert e.value.status == dh.DH_ERR_ARG
    for args, kw in (((z, ids[:3], val), {}), ((z, ids, val[:, :1]), {}), ((z, ids.long(), val), {}),
                     ((z, ids, val.double()), {}), ((z, ids, val), dict(weights=torch.ones(3, device="cuda"))),
                     ((z, ids, val), dict(dlogits=torch.empty((4, 64), dtype=torch.bfloat16, device="cuda"))),
                     ((z, ids, val), dict(dlogits=torch.empty((4, 63), device="cuda"))),
                     ((z, ids.expand(4, 2)[:, :0], val[:, :0]), {})):
        with pytest.raises(ValueError):
            dh.distill_topk(*args, **kw)
    with pytest.raises(ValueError):
        dh.distill_topk_backward(z, ids, val, torch.zeros(3, device="cuda"))
