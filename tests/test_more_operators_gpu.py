"""The FP8 block-scaled product and the vocabulary cross entropy: together as in training a
draft head behind a frozen FP8 layer, beside pending work on other streams, on another current
device, called first from several threads, and with a role of a kernel idle."""
import os
import subprocess
import sys

import pytest
import torch

import nvfp4_draft_head_gb300 as dh
from test_operator_streams_gpu import beside_pending_work

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU test needs a CUDA device"
    from nvfp4_draft_head_gb300 import build
    build.build()


def rand(shape, seed, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda") * scale).to(dtype)


def test_training_a_head_behind_a_frozen_layer():
    """input -> FP8 layer (frozen) -> hidden states -> loss over the kept rows -> gradients of the
    head and, through the layer, of the input; the head after a step is quantised and drafts.
    The gradients are compared with the chain in 64 bits from the layer's own outputs: the loss's
    are off by a few roundings (2^-8 of the magnitudes summed), and the layer's by those and
    by its quantisation of them (2^-4 more)."""
    V, n, K, T = 3000, 1000, 256, 300
    keep = torch.zeros(V, dtype=torch.bool)
    keep[torch.randperm(V, generator=torch.Generator().manual_seed(1))[:n]] = True
    idx_host, nk = dh.draft_head_build_index(keep)
    idx = torch.from_numpy(idx_host).cuda()
    row_of = dh.draft_head_row_map(idx, nk, V)
    W = rand((V, K), 2, 0.05)
    rows = W[idx[:nk].long()].clone().requires_grad_()
    layer = dh.FP8BlockMatmul.from_weight(rand((K, K), 3, K ** -0.5))
    x = rand((T, K), 4).requires_grad_()
    tokens = torch.randint(0, V, (T,), generator=torch.Generator("cuda").manual_seed(5), device="cuda", dtype=torch.int32)
    weights = torch.full((T,), 1.0 / T, device="cuda")

    hidden = dh.FP8BlockLinear.apply(x, layer)
    loss = dh.LinearCrossEntropy.apply(hidden, rows, tokens, weights, row_of)
    loss.sum().backward()

    h, R = hidden.detach().double(), rows.detach().double()
    col = row_of[tokens.long()].long()
    live = (col >= 0).double() / T
    z = h @ R.t()
    g = torch.softmax(z, 1)
    g[torch.arange(T, device="cuda"), col.clamp(min=0)] -= 1.0
    g *= live[:, None]
    assert 0.2 < (col >= 0).float().mean() < 0.5 and not loss[col < 0].any()
    u = 2.0 ** -8
    assert ((rows.grad.double() - g.t() @ h).abs() <= 3 * u * (g.abs().t() @ h.abs()) + 1e-12).all()
    dh_ref = g @ R
    q = layer.q.view(torch.float8_e4m3fn).double() * layer.scale.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    mag = (g.abs() @ R.abs()) @ q.abs()
    assert ((x.grad.double() - dh_ref @ q).abs() <= (2.0 ** -4 + 4 * u) * mag + 1e-12).all()
    assert not x.grad[col < 0].any()

    W[idx[:nk].long()] = (rows.detach().float() - 0.5 * rows.grad.float()).bfloat16()
    head = dh.nvfp4_head(W, keep)
    ids = head.top_tokens(hidden.detach()[:4].contiguous())
    assert torch.isin(ids, idx[:nk]).all() and head.device_error() == 0 and layer.device_error() == 0
    scores = dh.token_logprobs(hidden.detach() @ rows.detach().t(), tokens, row_of=row_of)
    exact = torch.log_softmax(z, 1).gather(1, col.clamp(min=0)[:, None])[:, 0]
    assert (((-loss.detach() * T) - exact).abs()[col >= 0] <= 1e-4).all()
    assert ((scores.logp - exact).abs()[col >= 0] <= 0.05).all()      # (those logits are rounded to bfloat16)
    assert dh.linear_cross_entropy_device_error() == 0


@pytest.mark.parametrize("T", [40, 300])
def test_captured_training_step(T):
    """Forward and backward pass of both captured into one graph, with leaves of its own, and
    replayed on other inputs."""
    n, K = 1000, 256
    layer = dh.FP8BlockMatmul.from_weight(rand((K, K), 3, K ** -0.5))
    inputs = [(rand((T, K), 10 + i), rand((n, K), 20 + i, 0.1), (torch.arange(T, device="cuda", dtype=torch.int32) * (i + 3)) % n,
               torch.rand(T, generator=torch.Generator("cuda").manual_seed(i), device="cuda")) for i in range(2)]

    def step(x, rows, tokens, weights):
        loss = dh.LinearCrossEntropy.apply(dh.FP8BlockLinear.apply(x, layer), rows, tokens, weights, None)
        return (loss.detach(), *torch.autograd.grad(loss.sum(), (x, rows, weights)))

    def leaves(a):
        return tuple(t.clone().requires_grad_(t.is_floating_point()) for t in a)

    want = [step(*leaves(a)) for a in inputs]
    static = leaves(inputs[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*static)
    for i in (0, 1, 0):
        with torch.no_grad():
            for s, v in zip(static, inputs[i]):
                s.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want[i]):
            assert torch.equal(a, b)
    assert layer.device_error() == 0 and dh.linear_cross_entropy_device_error() == 0


# ----------------------------------------------------------------- streams --

def test_beside_pending_work():
    mm = dh.FP8BlockMatmul.from_weight(rand((1088, 528), 1, 0.02))
    L = dh.lib()
    for M in (3, 50, 150):
        x, dy = rand((M, 528), 2), rand((M, 1088), 3)
        beside_pending_work(lambda s: mm(x, stream=s), [L.fp8_block_matmul_workspace_bytes(M, 528, 1088)])
        beside_pending_work(lambda s: mm.input_gradient(dy, stream=s), [L.fp8_block_matmul_workspace_bytes(M, 1088, 528)])
    W = rand((1000, 528), 4, 0.02)
    beside_pending_work(lambda s: dh.fp8_quantize_blocks(W, stream=s), [4000, 1024])
    h, t = rand((150, 528), 5), torch.arange(150, device="cuda", dtype=torch.int32)
    lse = dh.linear_cross_entropy_forward(h, W, t)[1]
    nb = [L.draft_head_cross_entropy_workspace_bytes(150, 1000, 528, o) for o in (1, 6, 7)]
    beside_pending_work(lambda s: dh.linear_cross_entropy(h, W, t, stream=s), nb)
    beside_pending_work(lambda s: dh.linear_cross_entropy_forward(h, W, t, stream=s), nb)
    beside_pending_work(lambda s: dh.linear_cross_entropy_backward(h, W, t, lse, stream=s), nb)


def test_constructors_on_a_stream():
    W = rand((300, 528), 1, 0.02)
    q, s = dh.fp8_quantize_blocks(W)
    x = rand((20, 528), 2)
    want = dh.FP8BlockMatmul(q, s)(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a, b = dh.FP8BlockMatmul(q, s, stream=side), dh.FP8BlockMatmul.from_weight(W, stream=side)
    ya, yb = a(x, stream=side), b(x, stream=side)
    side.synchronize()
    assert torch.equal(ya, want) and torch.equal(yb, want)


def test_calls_at_once_on_two_streams():
    """Each call has its own workspace: results do not depend on what runs beside it."""
    mm = dh.FP8BlockMatmul.from_weight(rand((2560, 2560), 1, 0.02))
    W, t = rand((5000, 256), 2, 0.1), torch.randint(0, 5000, (400,), device="cuda", dtype=torch.int32)
    xs, hs = [rand((m, 2560), 10 + m) for m in (1, 16, 90, 300)], [rand((400, 256), 30 + i) for i in range(4)]
    want = [(mm(x), dh.linear_cross_entropy(h, W, t)) for x, h in zip(xs, hs)]
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    for _ in range(5):
        out = [(mm(x, stream=s), dh.linear_cross_entropy(h, W, t, stream=s)) for x, h, s in zip(xs, hs, streams)]
        torch.cuda.synchronize()
        for (y, c), (yw, cw) in zip(out, want):
            assert torch.equal(y, yw) and all(torch.equal(p, q) for p, q in zip(c, cw))


# ----------------------------------------------------------------- devices --

def test_tensors_of_another_device_are_refused(monkeypatch):
    W, x = rand((64, 32), 1), rand((4, 32), 2)
    q, s = dh.fp8_quantize_blocks(W)
    mm = dh.FP8BlockMatmul(q, s)
    t, lse, side = torch.zeros(4, device="cuda", dtype=torch.int32), torch.zeros(4, device="cuda"), torch.cuda.Stream()
    launched = []

    class Library:
        """Sizes are answered; a launch is noted instead."""
        def __getattr__(self, name):
            if name.endswith("_bytes"):
                return getattr(real, name)
            return lambda *args: launched.append(name) or dh.DH_OK

    real = dh.lib()
    monkeypatch.setattr(dh, "lib", lambda: Library())
    monkeypatch.setattr(dh, "_current_device", lambda: 1)
    for stream in (None, side):
        for call in (lambda: mm(x, stream=stream), lambda: mm.input_gradient(rand((4, 64), 3), stream=stream),
                     lambda: dh.FP8BlockMatmul(q, s, stream=stream), lambda: dh.FP8BlockMatmul.from_weight(W, stream=stream),
                     lambda: dh.fp8_quantize_blocks(W, stream=stream), lambda: dh.linear_cross_entropy(x, W, t, stream=stream),
                     lambda: dh.linear_cross_entropy_forward(x, W, t, stream=stream),
                     lambda: dh.linear_cross_entropy_backward(x, W, t, lse, stream=stream)):
            with pytest.raises(ValueError, match="cuda:0"):
                call()
    assert launched == []


PROGRAM = """
import threading
import torch
import nvfp4_draft_head_gb300 as dh
mm = dh.FP8BlockMatmul(torch.randint(0, 100, (1088, 272), device="cuda", dtype=torch.uint8), torch.rand((9, 3), device="cuda"))
xs = [torch.randn((m, 272), device="cuda") for m in (1, 40, 300)]
h, W = torch.randn((300, 64), device="cuda").bfloat16(), torch.randn((1001, 64), device="cuda").bfloat16()
t = torch.randint(0, 1001, (300,), device="cuda", dtype=torch.int32)
torch.cuda.synchronize()
start, out = threading.Barrier(8), [None] * 8
def call(i):
    start.wait()
    out[i] = [*(mm(x) for x in xs), *dh.linear_cross_entropy(h, W, t), *dh.linear_cross_entropy_forward(h, W, t)]
threads = [threading.Thread(target=call, args=(i,)) for i in range(8)]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
assert all(torch.equal(a, b) for o in out for a, b in zip(o, out[0], strict=True))
print("equal")
"""


def test_first_calls_at_once():
    r = subprocess.run([sys.executable, "-c", PROGRAM], capture_output=True, text=True, cwd=ROOT, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "equal", r.stdout + r.stderr
