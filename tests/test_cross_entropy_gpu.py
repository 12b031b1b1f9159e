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
summed with at most 2^-23 of the sum of magnitudes per addition, and rounded once:
  |error| <= sum_n |g error| |W| + N 2^-23 sum |g| |W| + u |dh|, the same over tokens for dW.
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
    small = 2.0 ** -39 * w.abs().max() if s["hidden"].dtype == torch.float16 else 0.0
    ge = (w.abs() * (2 * dz + 2.0 ** -15 + 2.0 ** -23 * lse.abs()))[:, None] * p + u * g.abs() + small * live[:, None]
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
    u = torch.finfo(s["hidden"].dtype).eps / 2
    for got, k in ((dx, "dhidden"), (dw, "dhead")):
        if got.numel() >= 4096 and live.any():
            assert (got.double() - out[k]).norm() <= 1.5 * u * out[k].norm(), k
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
