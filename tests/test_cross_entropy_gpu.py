"""Vocabulary cross entropy (loss, normaliser, gradients in the hidden states and the head
rows) against a plain implementation in 64 bits.

Tolerances. u is half a step of the inputs' type (bf16 2^-8, f16 2^-11). A logit is a sum of K
exact products, each addition off by at most 2^-23 of what is summed so far (truncation
included): dz <= K 2^-23 A, A = sum |h W|, the largest of a row for all of its columns. The
exponentials are off by 2^-21 (their argument's rounding at 30 or below included), the sums
of N of them, in runs of 8 and then pairwise-like joins, by at most 2^-17, the logarithm and
the additions after it by 2^-22 (1 + |lse| + |z|). So
  lse:  dz + 2^-16 + 2^-22 (1 + |lse|);   loss: |w| (2 dz + 2^-16 + 2^-22 (1 + |lse| + |z_y|)).
A gradient is a product with g, |g error| <= |w| p (2 dz + 2^-15 + 2^-23 |lse|) + u |g| (its
rounding; f16's scale keeps w in [2^14, 2^15), so its subnormals add at most 2^-25 2^-14 |w|max),
(bf16 has 32-bit floats' range: the exponential, and g scaled by a power of two above 1 / (2
|w|max), are zero below 2^-126, which adds at most 2^-126 (|w| + 2 |w|max)), summed with at
most 2^-23 of the sum of magnitudes per addition, and rounded once; up to 128 tokens have g in
two terms, u^2 in place of u |g|:
  |error| <= sum_n |g error| |W| + N 2^-23 sum |g| |W| + u |dh|, the same over tokens for dW.
In the 2-norm, where roundings are independent: those of g (as large, relative to the result,
as those of the result) and of the result, and half a step below the type's range for each:
  ||error|| <= 1.5 u ||dh|| + sqrt(elements) half the smallest number.
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


def make(T, N, K, dtype, seed=0, pad_h=0, pad_w=0, mapped=False, dead=True, lean=6.0, spread=0.05):
    g = torch.Generator(DEV).manual_seed(1000 * seed + T + 7 * N + 13 * K)
    buf_w = torch.full((N, K + pad_w), float("nan"), dtype=dtype, device=DEV)
    buf_w[:, :K] = torch.randn((N, K), generator=g, device=DEV) * spread
    head = buf_w[:, :K]
    rows = torch.randint(0, N, (T,), generator=g, device=DEV)
    h = torch.randn((T, K), generator=g, device=DEV)
    w = head[rows].float()
    h += lean * w / (w * w).sum(1, keepdim=True).clamp(min=1e-6) * torch.rand((T, 1), generator=g, device=DEV)
    buf_h = torch.full((T, K + pad_h), float("nan"), dtype=dtype, device=DEV)
    buf_h[:, :K] = h
    weights = torch.rand(T, generator=g, device=DEV) + 0.5
    tokens, row_of = rows.to(torch.int32), None
    if mapped:
        V = 2 * N + 5
        ids = torch.randperm(V, generator=g, device=DEV)[:N].sort().values.to(torch.int32)
        row_of = dh.draft_head_row_map(ids, N, V)
        tokens = ids[rows].contiguous()
    if dead:
        tokens[1::5] = -100
        weights[2::7] = 0.0
        if mapped:
            tokens[3::11] = 2 * N + 5
    return dict(hidden=buf_h[:, :K], head=head, tokens=tokens, weights=weights, row_of=row_of)


def reference(s, lse_given=None):
    h, W = s["hidden"].double(), s["head"].double()
    T, K = h.shape
    N = W.shape[0]
    u = torch.finfo(s["hidden"].dtype).eps / 2
    tok = s["tokens"].long()
    if s["row_of"] is not None:
        V = s["row_of"].numel()
        tok = torch.where((tok >= 0) & (tok < V), s["row_of"].long()[tok.clamp(0, V - 1)], torch.full_like(tok, -1))
    w = torch.ones(T, dtype=torch.float64, device=DEV) if s["weights"] is None else s["weights"].double()
    live = (tok >= 0) & (tok < N) & (w != 0)
    y = tok.clamp(0, N - 1)
    w = torch.where(live, w, torch.zeros_like(w))
    hl = torch.where(live[:, None], h, torch.zeros_like(h))
    z = h @ W.t()
    dz = (K * 2.0 ** -23) * (h.abs() @ W.abs().t()).amax(1)
    lse = torch.logsumexp(z, 1)
    zy = z.gather(1, y[:, None])[:, 0]
    out, tol = {}, {}
    out["lse"], tol["lse"] = lse, dz + 2.0 ** -16 + 2.0 ** -22 * (1 + lse.abs())
    out["loss"] = torch.where(live, w * (lse - zy), torch.zeros_like(w))
    tol["loss"] = torch.where(live, w.abs() * (2 * dz + 2.0 ** -16 + 2.0 ** -22 * (1 + lse.abs() + zy.abs())), torch.zeros_like(w))
    norm = lse if lse_given is None else lse_given.double()
    p = torch.exp(z - norm[:, None])
    g = p.scatter_add(1, y[:, None], -torch.ones_like(w)[:, None])
    g = torch.where(live[:, None], g * w[:, None], torch.zeros_like(g))
    p = torch.where(live[:, None], p, torch.zeros_like(p))
    small = (2.0 ** -39 if s["hidden"].dtype == torch.float16 else 2.0 ** -124) * w.abs().max()
    ge = (w.abs() * (2 * dz + 2.0 ** -15 + 2.0 ** -23 * lse.abs()))[:, None] * p + (u * u if T <= 128 else u) * g.abs() + small * live[:, None]
    ge = torch.where(live[:, None], ge, torch.zeros_like(ge))
    out["dhidden"], out["dhead"] = g @ W, g.t() @ hl
    tol["dhidden"] = ge @ W.abs() + N * 2.0 ** -23 * (g.abs() @ W.abs()) + u * out["dhidden"].abs()
    tol["dhead"] = ge.t() @ hl.abs() + T * 2.0 ** -23 * (g.abs().t() @ hl.abs()) + u * out["dhead"].abs()
    tiny = torch.finfo(s["hidden"].dtype).smallest_normal * torch.finfo(s["hidden"].dtype).eps
    for k in ("dhidden", "dhead"):
        tol[k] = tol[k] + tiny
    return out, tol, live


def near(got, want, tol, what):
    d = (got.double() - want).abs()
    bad = ~(d <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {(d / tol.clamp(min=1e-300)).nan_to_num(9e9).max().item():.3g} " \
                          f"times the tolerance, first at {bad.nonzero()[0].tolist()}"


def check(s, **more):
    out, tol, live = reference(s)
    loss, dx, dw = dh.linear_cross_entropy(**s)
    near(loss, out["loss"], tol["loss"], "loss")
    near(dx, out["dhidden"], tol["dhidden"], "dhidden")
    near(dw, out["dhead"], tol["dhead"], "dhead")
    # in the 2-norm the error is that of independent roundings: of g, and of the result
    info = torch.finfo(s["hidden"].dtype)
    least = info.smallest_normal * info.eps
    for got, k in ((dx, "dhidden"), (dw, "dhead")):
        if got.numel() >= 4096 and live.any():
            assert (got.double() - out[k]).norm() <= 0.75 * info.eps * out[k].norm() + got.numel() ** 0.5 * least / 2, k
    f_loss, lse, rest = dh.linear_cross_entropy_forward(**s)
    assert torch.equal(f_loss, loss)
    near(lse, out["lse"], tol["lse"], "lse")
    assert (rest.abs() <= 2.0 ** -24 * lse.abs() * 1.01 + 1e-38).all()
    bx, bw = dh.linear_cross_entropy_backward(s["hidden"], s["head"], s["tokens"], lse, s["weights"], rest, s["row_of"])
    assert torch.equal(bx, dx) and torch.equal(bw, dw)
    assert dh.linear_cross_entropy_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,N,K", [(1, 1, 8), (1, 2, 8), (2, 300, 64), (16, 4000, 256), (130, 257, 72), (257, 1000, 200), (300, 513, 1032),
                                   (1000, 255, 520), (129, 2561, 2560)])
def test_sizes(T, N, K, dtype):
    check(make(T, N, K, dtype))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("pad_h,pad_w,mapped", [(8, 0, False), (0, 24, True), (72, 8, True)])
def test_strides_and_maps(pad_h, pad_w, mapped, dtype):
    check(make(200, 700, 136, dtype, pad_h=pad_h, pad_w=pad_w, mapped=mapped))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_several_pieces_of_the_vocabulary(dtype):
    """131,072 tokens leave 2,048 head rows a piece: three of them, the last one ragged."""
    s = make(131072, 5003, 64, dtype, dead=False)
    assert dh.lib().draft_head_cross_entropy_workspace_bytes(131072, 5003, 64, dh.DH_CE_DHIDDEN) < 131072 * 5003 * 2
    out, tol, _ = reference(s)
    loss, dx, dw = dh.linear_cross_entropy(**s)
    near(loss, out["loss"], tol["loss"], "loss")
    near(dx, out["dhidden"], tol["dhidden"], "dhidden")
    near(dw, out["dhead"], tol["dhead"], "dhead")


@pytest.mark.parametrize("lean,spread", [(0.0, 0.0), (60.0, 0.05), (0.0, 4.0)])
def test_flat_sure_and_large_logits(lean, spread):
    """Equal logits; tokens that are all but certain; logits in the thousands (lse + rest)."""
    check(make(150, 600, 264, torch.bfloat16, lean=lean, spread=spread))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("scale", [1e-30, 1e-4, 1.0, -300.0])
def test_row_weights(dtype, scale):
    s = make(140, 300, 72, dtype)
    s["weights"] *= scale
    s["weights"][5::9] *= 1e-3     # far from the largest
    if dtype == torch.float16 and abs(scale) < 1e-6:
        s["weights"] *= 1e26       # f16 results hold no less
    check(s)
    s["weights"] = None
    check(s)


def test_rows_that_are_left_out():
    """Whatever the hidden states of padding rows hold, they touch nothing."""
    s = make(300, 500, 136, torch.bfloat16)
    want = dh.linear_cross_entropy(**s)
    _, _, live = reference(s)
    junk = s["hidden"].clone()
    junk[~live] = float("nan")
    junk[(~live).nonzero()[::2, 0]] = float("inf")
    got = dh.linear_cross_entropy(junk, *(s[k] for k in ("head", "tokens", "weights", "row_of")))
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert not want[0][~live].any() and not want[1][~live].any()
    # no row counts
    for kw in (dict(tokens=torch.full_like(s["tokens"], -100)), dict(weights=torch.zeros_like(s["weights"])),
               dict(tokens=torch.full_like(s["tokens"], 500)), dict(tokens=torch.full_like(s["tokens"], 2 ** 31 - 1))):
        loss, dx, dw = dh.linear_cross_entropy(**{**s, "hidden": junk, **kw})
        assert not loss.any() and not dx.any() and not dw.any()
        loss, lse, _ = dh.linear_cross_entropy_forward(**{**s, **kw})
        assert not loss.any() and torch.isfinite(lse).all()


def test_rows_that_are_not_finite():
    s = make(260, 300, 72, torch.bfloat16, dead=False)
    want = dh.linear_cross_entropy(**s)
    bad = s["hidden"].clone()
    bad[7, 3], bad[200, 0] = float("nan"), float("inf")
    loss, dx, dw = dh.linear_cross_entropy(bad, *(s[k] for k in ("head", "tokens", "weights", "row_of")))
    rest = [i for i in range(260) if i not in (7, 200)]
    assert loss[[7, 200]].isnan().all() and dx[[7, 200]].isnan().all() and dw.isnan().any()
    assert torch.equal(loss[rest], want[0][rest]) and torch.equal(dx[rest], want[1][rest])


def test_one_token_many_times_and_given_outputs():
    s = make(257, 40, 64, torch.float16, dead=False)
    s["tokens"][:] = 17
    check(s)
    want = dh.linear_cross_entropy(**s)
    dx = torch.full((257, 96), 3.0, dtype=torch.float16, device=DEV)
    dw = torch.full((42, 72), 3.0, dtype=torch.float16, device=DEV)
    got = dh.linear_cross_entropy(**s, dhidden=dx[:, 16:80], dhead=dw[1:41, :64])
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert (dx[:, :16] == 3).all() and (dx[:, 80:] == 3).all() and (dw[0] == 3).all() and (dw[41] == 3).all() and (dw[:, 64:] == 3).all()
    lse = dh.linear_cross_entropy_forward(**s)[1]
    a = (s["hidden"], s["head"], s["tokens"], lse, s["weights"])
    both = dh.linear_cross_entropy_backward(*a)
    assert dh.linear_cross_entropy_backward(*a, dhead=False)[1] is None and dh.linear_cross_entropy_backward(*a, dhidden=False)[0] is None
    assert torch.equal(dh.linear_cross_entropy_backward(*a, dhead=False)[0], both[0])
    assert torch.equal(dh.linear_cross_entropy_backward(*a, dhidden=False)[1], both[1])


def test_no_tokens():
    s = make(4, 40, 64, torch.bfloat16)
    e = {k: (v[:0] if k in ("hidden", "tokens", "weights") else v) for k, v in s.items()}
    loss, dx, dw = dh.linear_cross_entropy(**e)
    assert loss.shape == (0,) and dx.shape == (0, 64) and dw.shape == (40, 64) and not dw.any()
    assert all(t.shape == (0,) for t in dh.linear_cross_entropy_forward(**e))
    dx, dw = dh.linear_cross_entropy_backward(e["hidden"], e["head"], e["tokens"], loss, e["weights"])
    assert dx.shape == (0, 64) and not dw.any()


def test_refusals():
    s = make(6, 40, 64, torch.bfloat16)
    h, W, t, w = s["hidden"], s["head"], s["tokens"], s["weights"]
    for bad in (dict(hidden=h.float()), dict(hidden=h[:, ::2]), dict(hidden=h.half()), dict(head=W[:, :56]), dict(head=W.t()),
                dict(head=W[:0]), dict(tokens=t.long()), dict(tokens=t[:5]), dict(tokens=t.cpu()), dict(weights=w.double()), dict(weights=w[:5]),
                dict(row_of=t.float()), dict(dhidden=h.float()), dict(dhead=W[1:]), dict(dhidden=h.half()),
                dict(hidden=torch.zeros(6 * 64 + 1, dtype=h.dtype, device=DEV)[1:].view(6, 64)),
                dict(hidden=torch.zeros((6, 68), dtype=h.dtype, device=DEV)[:, :64])):
        with pytest.raises(ValueError):
            dh.linear_cross_entropy(**{**s, **bad})
    square = torch.empty((40, 64), dtype=h.dtype, device=DEV)
    for bad in (dict(hidden=h[:, :60].contiguous(), head=W[:, :60].contiguous()), dict(dhidden=h), dict(dhead=W),
                dict(dhidden=square[:6], dhead=square)):
        with pytest.raises((dh.DraftHeadError, ValueError)):
            dh.linear_cross_entropy(**{**s, **bad})
    torch.cuda.synchronize()


def test_offsets_past_32_bits_in_the_head():
    """2.15e9 elements of the head and of its gradient; the last rows are what is looked at."""
    N, K, T = 840_000, 2560, 20
    head = torch.empty((N, K), dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(DEV).manual_seed(3)
    for r in range(0, N, 40_000):
        head[r:r + 40_000] = torch.randn((min(40_000, N - r), K), generator=g, device=DEV) * 0.02
    rows = torch.cat([torch.arange(N - 10, N, device=DEV), torch.arange(0, N, N // 10, device=DEV)[:10]])
    h = (torch.randn((T, K), generator=g, device=DEV) + 8.0 * head[rows].float()).bfloat16()
    loss, lse, rest = dh.linear_cross_entropy_forward(h, head, rows.to(torch.int32))
    z = torch.cat([h.double() @ head[r:r + 40_000].double().t() for r in range(0, N, 40_000)], 1)
    want = torch.logsumexp(z, 1) - z.gather(1, rows[:, None])[:, 0]
    A = (h.double().abs() @ head[rows].double().abs().t()).amax(1) * 2     # (a bound: rows of the head are alike)
    near(loss, want, 2 * K * 2.0 ** -23 * A + 2.0 ** -15, "loss")
    dx, dw = dh.linear_cross_entropy_backward(h, head, rows.to(torch.int32), lse, rest=rest)
    p = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
    p[torch.arange(T, device=DEV), rows] -= 1.0
    del z
    u = 2.0 ** -8
    for r in (0, N // 2, N - 3000):
        q = p[:, r:r + 3000]
        ref = q.t() @ h.double()
        near(dw[r:r + 3000], ref, u * ref.abs() + 2 * u * (q.abs().t() @ h.double().abs()) + 1e-30, "dhead")
    dh_ref = sum(p[:, r:r + 40_000] @ head[r:r + 40_000].double() for r in range(0, N, 40_000))
    mag = sum(p[:, r:r + 40_000].abs() @ head[r:r + 40_000].double().abs() for r in range(0, N, 40_000))
    near(dx, dh_ref, u * dh_ref.abs() + 2 * u * mag, "dhidden")


def test_offsets_past_32_bits_in_the_piece():
    """1,100,000 tokens times 2,048 rows: 2.25e9 elements of g."""
    T, N, K = 1_100_000, 2048, 8
    s = make(T, N, K, torch.bfloat16, dead=False, spread=0.5)
    loss, dx, dw = dh.linear_cross_entropy(**s)
    total = torch.zeros((N, K), dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(total)
    u = 2.0 ** -8
    for r in range(0, T, 100_000):
        e = {k: (v[r:r + 100_000] if k in ("hidden", "tokens", "weights") else v) for k, v in s.items()}
        out, tol, _ = reference(e)
        near(loss[r:r + 100_000], out["loss"], tol["loss"], "loss")
        near(dx[r:r + 100_000], out["dhidden"], tol["dhidden"], "dhidden")
        total += out["dhead"]
        mag += tol["dhead"] / u      # of the order of sum |g| |h|
    near(dw, total, u * total.abs() + (u + T * 2.0 ** -23) * mag, "dhead")


def test_graphs():
    """Captured once, replayed on other inputs; two graphs at a time; the first call of a
    process's device word may be a captured one."""
    s, t = make(200, 700, 136, torch.bfloat16, mapped=True), make(200, 700, 136, torch.bfloat16, seed=5, mapped=True)
    both = lambda a: dh.linear_cross_entropy(**a)  # noqa: E731

    def split(a):
        loss, lse, rest = dh.linear_cross_entropy_forward(**a)
        return loss, *dh.linear_cross_entropy_backward(a["hidden"], a["head"], a["tokens"], lse, a["weights"], rest, a["row_of"])

    want = {id(a): both(a) for a in (s, t)}
    static = {k: v.clone() for k, v in s.items()}
    graphs = []
    for f in (both, split):
        g = torch.cuda.CUDAGraph()
        f(static)
        with torch.cuda.graph(g):
            out = f(static)
        graphs.append((g, out))
    for a in (s, t, s):
        for k in static:
            static[k].copy_(a[k])
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            for x, y in zip(out, want[id(a)]):
                assert torch.equal(x, y)
    assert dh.linear_cross_entropy_device_error() == 0


# ---------------------------------------------------------------- autograd --

@pytest.mark.parametrize("wants", [(True, True, True), (True, False, False), (False, True, False), (False, False, True)])
def test_autograd(wants):
    s = make(130, 257, 72, torch.bfloat16)
    up = torch.rand(130, generator=torch.Generator(DEV).manual_seed(2), device=DEV)
    h, W, w = s["hidden"].clone().requires_grad_(wants[0]), s["head"].clone().requires_grad_(wants[1]), s["weights"].clone().requires_grad_(wants[2])
    loss = dh.LinearCrossEntropy.apply(h, W, s["tokens"], w, s["row_of"])
    (loss * up).sum().backward()
    out, tol, live = reference({**s, "weights": s["weights"] * up})
    for x, k, i in ((h, "dhidden", 0), (W, "dhead", 1)):
        if wants[i]:
            near(x.grad, out[k], tol[k] * 1.01, k)
        else:
            assert x.grad is None
    if wants[2]:   # the row's loss at weight 1, for a row of weight 0 too
        one, t1, _ = reference({**s, "weights": None})
        near(w.grad, one["loss"] * up, t1["loss"] * up + 2.0 ** -22 * (one["loss"] * up).abs(), "weights")


def test_autograd_without_weights_and_twice():
    s = make(40, 64, 64, torch.float16, dead=False)
    h = s["hidden"].clone().requires_grad_()
    loss = dh.LinearCrossEntropy.apply(h, s["head"], s["tokens"])
    (dx,) = torch.autograd.grad(loss.mean(), h, create_graph=True)
    out, tol, _ = reference({**s, "weights": torch.full((40,), 1 / 40, device=DEV)})
    near(dx.detach(), out["dhidden"], tol["dhidden"] * 1.01, "dhidden")
    with pytest.raises(RuntimeError, match="differentiable once"):
        (dx.float().square().sum() + h.float().square().sum()).backward()


def test_against_differences():
    """Central differences of the loss, in steps that the type holds: off by d^2 / 6 times a
    third derivative, at most (max W - min W)^3 a token, and by the loss's own error over d."""
    T, N, K, d = 3, 50, 16, 2.0 ** -5
    s = make(T, N, K, torch.float16, dead=False, spread=0.3)
    s["hidden"] = (s["hidden"].float() * 32).round().div(32).half()
    out, tol, _ = reference(s)
    _, dx, _ = dh.linear_cross_entropy(**s)
    span = (s["head"].float().amax(0) - s["head"].float().amin(0))
    for k in range(K):
        f = []
        for sign in (1, -1):
            h = s["hidden"].clone()
            h[:, k] += sign * d
            f.append(dh.linear_cross_entropy_forward(**{**s, "hidden": h})[0].double())
        diff = (f[0] - f[1]) / (2 * d)
        near(dx[:, k], diff, s["weights"].double() * span[k].double() ** 3 * d * d / 6 + 2 * tol["loss"] / d + tol["dhidden"][:, k], f"feature {k}")
