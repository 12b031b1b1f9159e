"""The operators with which a draft head is trained and its FP8 layers run over many
tokens, as cases with real sizes, each in a plain form (elementary torch operations,
32 bits) and as a user calls it:

  fp8      hidden states times an FP8 (E4M3) weight with one scale per block of
           128 x 128, the hidden states quantised per token and 128 features: the
           layer's output, or the gradient in its input (the incoming gradient
           quantised per token and 128 of its own features);
  loss     softmax cross entropy of hidden states against a vocabulary given by its
           head rows, without logits in memory: the loss, the loss with its gradients
           in the hidden states and the head, or the gradients from a kept normaliser.

`own` selects the framework's kernels; `exact` gives the same outputs in 64 bits.
Sizes: the 2,560-wide drafter with its 248,320-id vocabulary of which 64,026 ids are
kept, the MTP block's linears, and the 4,000-id small head of width 256.
"""
import math

import numpy as np
import torch

own = False

V_TARGET = 248_320
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
NEG = float("-inf")


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # the qkv linear of the MTP block for one drafted token
        dict(name="fp8 qkv, 1 token", op="fp8", T=1, N=4608, K=2560, x="bf16", y="bf16", mode="forward"),
        # the fc linear (two hidden states concatenated) for sixteen concurrent drafts, results in 32 bits
        dict(name="fp8 fc, 16 tokens", op="fp8", T=16, N=2560, K=5120, x="bf16", y="f32", mode="forward"),
        # a short prompt of an odd length on a layer whose sizes divide into no tile
        dict(name="fp8 ragged, 333 tokens", op="fp8", T=333, N=4001, K=1040, x="f16", y="f16", mode="forward"),
        # draft logits of the tokens of one prompt
        dict(name="fp8 head, 100 tokens", op="fp8", T=100, N=64026, K=2560, x="bf16", y="f32", mode="forward"),
        # draft logits of a batch of sequences
        dict(name="fp8 head, 8192 tokens", op="fp8", T=8192, N=64026, K=2560, x="bf16", y="bf16", mode="forward"),
        # training through the frozen qkv linear: the gradient of its input
        dict(name="fp8 qkv gradient, 4096 tokens", op="fp8", T=4096, N=4608, K=2560, x="bf16", y="bf16", mode="gradient"),
        # a few tokens of the small head: loss and gradients
        dict(name="loss 16 x 4000", op="loss", T=16, N=4000, K=256, h="f16", mode="both", mapped=False, pad=0),
        # the loss of one sequence's end, head read once
        dict(name="loss forward 61 x 64026", op="loss", T=61, N=64026, K=2560, h="bf16", mode="forward", mapped=True, pad=0),
        # a validation pass: the loss alone
        dict(name="loss forward 4095 x 64026", op="loss", T=4095, N=64026, K=2560, h="bf16", mode="forward", mapped=True, pad=64),
        # one training step of the draft head: loss and both gradients
        dict(name="loss 4096 x 64026", op="loss", T=4096, N=64026, K=2560, h="bf16", mode="both", mapped=True, pad=0),
        # the full vocabulary, gradients from a kept normaliser, float16
        dict(name="loss backward 333 x 248320", op="loss", T=333, N=248320, K=2560, h="f16", mode="backward", mapped=False, pad=0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fp8", "loss"])
    if op == "fp8":
        n, k = _log_int(rng, 16, 64026), 16 * _log_int(rng, 4, 320)
        t = min(_log_int(rng, 1, 8192), 8192 * 64026 * 2560 // (n * k))
        return dict(op=op, T=t, N=n, K=k, x=rng.choice(["bf16", "f16", "f32"]), y=rng.choice(["bf16", "f16", "f32"]),
                    mode=rng.choice(["forward", "forward", "gradient"]))
    mapped = rng.random() < 0.5
    n, k = _log_int(rng, 2, 100_000 if mapped else V_TARGET), 16 * _log_int(rng, 4, 320)
    t = max(1, min(_log_int(rng, 1, 8192), 4096 * 64026 * 2560 // (n * k), 4096 * 64026 // n))
    return dict(op=op, T=t, N=n, K=k, h=rng.choice(["bf16", "f16"]), mode=rng.choice(["both", "both", "forward", "backward"]),
                mapped=mapped, pad=rng.choice([0, 0, 8, 64]))


def work(case):
    t, n, k = case["T"], case["N"], case["K"]
    if case["op"] == "fp8":
        x, y = (n, k) if case["mode"] == "gradient" else (k, n)
        scales = -(-n // 128) * -(-k // 128) * 4
        return {"bytes": t * x * BYTES[case["x"]] + n * k + scales + t * y * BYTES[case["y"]], "flops": 2 * t * n * k}
    read = 2 * (t * k + n * k) + 8 * t
    if case["mode"] == "forward":
        return {"bytes": read + 8 * t, "flops": 2 * t * n * k}
    # the logits (again, where the loss was an earlier call) and the two gradients, three products either way
    return {"bytes": 2 * read, "flops": 6 * t * n * k}


# ----------------------------------------------------------------- inputs --

def _gen(seed, salt):
    return torch.Generator("cuda").manual_seed(int(seed) * 1013 + salt)


def _scale(amax):
    """amax / 448 with the amax clamped below, as tensors on the device (IEEE divisions)."""
    return torch.clamp(amax, min=1e-12) / torch.full_like(amax, 448.0)


def _codes(x, s):
    """E4M3 codes of x under the scales s (broadcast over x)."""
    return torch.clamp(x / s, -448.0, 448.0).to(torch.float8_e4m3fn)


def _blocks(x, rows, cols):
    """x [R, C] padded with zeros to whole blocks, as [R / rows, rows, C / cols, cols]."""
    r, c = x.shape
    x = torch.nn.functional.pad(x, (0, -c % cols, 0, -r % rows))
    return x.view(x.shape[0] // rows, rows, x.shape[1] // cols, cols)


def _weight(case, seed):
    """An FP8 weight [N, K]: codes, block scales and the values they stand for."""
    n, k = case["N"], case["K"]
    w = torch.empty((n, k), device="cuda")
    w.normal_(0.0, 0.02, generator=_gen(seed, 1))
    w[:, :: 97] *= 20.0
    w[5 :: 301] *= 0.01
    b = _blocks(w.bfloat16().float(), 128, 128)
    s = _scale(b.abs().amax((1, 3)))
    q = _codes(b, s[:, None, :, None])
    w = (q.float() * s[:, None, :, None]).view(b.shape[0] * 128, -1)[:n, :k].contiguous()
    return q.view(torch.uint8).view(b.shape[0] * 128, -1)[:n, :k].contiguous(), s, w


def _rows(case, seed, width):
    """Rows of activations: normal, some channels far larger than the rest (a gradient: far smaller throughout)."""
    x = torch.empty((case["T"], width), device="cuda")
    x.normal_(0.0, 1.0, generator=_gen(seed, 2))
    x[:, 5 :: 211] *= 30.0
    if case["mode"] == "gradient":
        x *= 1e-3
    return x.to(DTYPES[case["x"]])


def _vocabulary(case, seed):
    """Target ids of the head's rows (ascending) and the row of every target id (-1: not kept)."""
    if not case["mapped"]:
        return None, None
    kept = torch.randperm(V_TARGET, generator=_gen(seed, 4), device="cuda")[:case["N"]].sort().values
    row_of = torch.full((V_TARGET,), -1, dtype=torch.int32, device="cuda")
    row_of[kept] = torch.arange(case["N"], dtype=torch.int32, device="cuda")
    return kept.to(torch.int32), row_of


def _training(case, seed):
    """Hidden states that lean towards their token's head row, the head, token ids (some not kept, some that stand
    for no token), row weights (padding rows 0)."""
    t, n, k = case["T"], case["N"], case["K"]
    gen, dtype = _gen(seed, 5), DTYPES[case["h"]]
    head = torch.empty((n, k), device="cuda")
    head.normal_(0.0, 0.02, generator=gen)
    head = head.to(dtype)
    rows = torch.randint(0, n, (t,), generator=gen, device="cuda")
    h = torch.empty((t, k), device="cuda")
    h.normal_(0.0, 1.0, generator=gen)
    h[:, 5 :: 211] *= 4.0
    w = head[rows].float()
    h += w * (torch.rand((t, 1), generator=gen, device="cuda") * 12.0) / (w * w).sum(1, keepdim=True)
    buf = torch.full((t, k + case["pad"]), 7.0, dtype=dtype, device="cuda")
    buf[:, :k] = h
    idx, row_of = _vocabulary(case, seed)
    tokens = idx[rows].clone() if idx is not None else rows.to(torch.int32)
    tokens[3::10] = -100
    if idx is not None:
        tokens[4::10] = torch.randint(0, V_TARGET, (t,), generator=gen, device="cuda", dtype=torch.int32)[4::10]
    weights = torch.rand(t, generator=gen, device="cuda") + 0.5
    weights[5::16] = 0.0
    return dict(case=case, hidden=buf[:, :k], head=head, tokens=tokens, row_of=row_of, weights=weights)


def prepare(case, seed):
    if case["op"] == "fp8":
        q, s, w = _weight(case, seed)
        st = dict(case=case, x=_rows(case, seed, case["N"] if case["mode"] == "gradient" else case["K"]), w=w)
        if own:   # the weight as a program holds it, in place of its values
            import nvfp4_draft_head_gb300 as dh
            st["mm"] = dh.FP8BlockMatmul(q, s)
            del st["w"]
        return st
    st = _training(case, seed)
    if case["mode"] == "backward":
        st["lse"] = torch.logsumexp((st["hidden"].float() @ st["head"].float().t()).double(), 1).float()
    if own:
        import nvfp4_draft_head_gb300 as dh
        st["dh"] = dh
    return st


# -------------------------------------------------------------------- run --

def run(st):
    return (_own if own else _plain)[st["case"]["op"]](st)


def _own_fp8(st):
    mm, dtype = st["mm"], DTYPES[st["case"]["y"]]
    return mm.input_gradient(st["x"], out_dtype=dtype) if st["case"]["mode"] == "gradient" else mm(st["x"], out_dtype=dtype)


def _own_loss(st):
    dh, mode = st["dh"], st["case"]["mode"]
    args = (st["hidden"], st["head"], st["tokens"])
    if mode == "forward":
        loss, lse, _ = dh.linear_cross_entropy_forward(*args, weights=st["weights"], row_of=st["row_of"])
        return dict(loss=loss, lse=lse)
    if mode == "backward":
        dhidden, dhead = dh.linear_cross_entropy_backward(*args, st["lse"], weights=st["weights"], row_of=st["row_of"])
        return dict(dhidden=dhidden, dhead=dhead)
    loss, dhidden, dhead = dh.linear_cross_entropy(*args, weights=st["weights"], row_of=st["row_of"])
    return dict(loss=loss, dhidden=dhidden, dhead=dhead)


_own = dict(fp8=_own_fp8, loss=_own_loss)


def _plain_fp8(st):
    x = st["x"].float()
    b = _blocks(x, 1, 128)
    s = _scale(b.abs().amax(-1, keepdim=True))
    v = (_codes(b, s).float() * s).view(x.shape[0], -1)[:, :x.shape[1]]
    w = st["w"]
    return (v @ (w if st["case"]["mode"] == "gradient" else w.t())).to(DTYPES[st["case"]["y"]])


def _plain_columns(st):
    """Head row of every token, and which tokens have one and count."""
    col, row_of, n = st["tokens"], st["row_of"], st["case"]["N"]
    if row_of is not None:
        there = (col >= 0) & (col < row_of.numel())
        col = torch.where(there, row_of[col.clamp(0, row_of.numel() - 1).long()], torch.full_like(col, -1))
    there = (col >= 0) & (col < n) & (st["weights"] != 0)
    return col.clamp(0, n - 1).long().unsqueeze(1), there.unsqueeze(1)


def _plain_loss(st):
    mode, dtype = st["case"]["mode"], st["hidden"].dtype
    h, head, w = st["hidden"].float(), st["head"].float(), st["weights"].unsqueeze(1)
    col, there = _plain_columns(st)
    z = h @ head.t()
    if mode == "backward":
        p = torch.exp(z - st["lse"].unsqueeze(1))
    else:
        m = z.amax(1, keepdim=True)
        p = torch.exp(z - m)
        s = p.sum(1, keepdim=True)
        log_s = torch.log(s)
        loss = torch.where(there, w * (log_s + (m - z.gather(1, col))), torch.zeros_like(w)).squeeze(1)
        if mode == "forward":
            return dict(loss=loss, lse=(m + log_s).squeeze(1))
        p /= s
    g = p.scatter_add(1, col, -torch.ones_like(w)) * torch.where(there, w, torch.zeros_like(w))
    out = dict(dhidden=(g @ head).to(dtype), dhead=(g.t() @ h).to(dtype))
    return out if mode == "backward" else dict(loss=loss, **out)


_plain = dict(fp8=_plain_fp8, loss=_plain_loss)


# ------------------------------------------------------------------ exact --

def _exact_fp8(case, seed):
    """The quantiser's decisions are defined in 32 bits (numpy float32); everything after them is in 64."""
    q, s, _ = _weight(case, seed)
    x = _rows(case, seed, case["N"] if case["mode"] == "gradient" else case["K"]).float().cpu().numpy()
    f = np.float32
    t, k = x.shape
    x = np.pad(x, ((0, 0), (0, -k % 128))).reshape(t, -1, 128)
    sx = np.maximum(np.abs(x).max(2, keepdims=True), f(1e-12)) / f(448)
    a = np.minimum(np.abs(x) / sx, f(448)).astype(np.float64)
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -30))), -6.0) - 3.0)   # E4M3's spacing around a
    v = np.copysign(np.rint(a / step) * step, x) * sx.astype(np.float64)
    v = torch.from_numpy(v.reshape(t, -1)[:, :k].copy()).cuda()
    grid = [(m / 8 * 2.0 ** -6) if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127]
    grid = torch.tensor(grid + [float("nan")] + [-g for g in grid] + [float("nan")], dtype=torch.float64, device="cuda")
    w = grid[q.long()] * s.double().repeat_interleave(128, 0).repeat_interleave(128, 1)[:case["N"], :case["K"]]
    return v @ (w if case["mode"] == "gradient" else w.t())


def _exact_loss(case, seed):
    st = _training(case, seed)
    mode = case["mode"]
    h, head = st["hidden"].double(), st["head"].double()
    given = None
    if mode == "backward":
        given = torch.logsumexp((st["hidden"].float() @ st["head"].float().t()).double(), 1).float().double()
    out = dict(loss=[], lse=[], dhidden=[])
    dhead = torch.zeros_like(head)
    for r in range(0, case["T"], 512):
        z = h[r:r + 512] @ head.t()
        lse = torch.logsumexp(z, 1) if given is None else given[r:r + 512]
        tok = st["tokens"][r:r + 512].long()
        if st["row_of"] is not None:
            tok = torch.where(tok < 0, tok, st["row_of"][tok.clamp(min=0)].long())
        w = st["weights"][r:r + 512].double().masked_fill(tok < 0, 0.0)
        tok = tok.clamp(min=0)
        at = torch.arange(tok.numel(), device="cuda")
        out["lse"].append(lse)
        out["loss"].append(w * (lse - z[at, tok]))
        if mode != "forward":
            g = (z - lse.unsqueeze(1)).exp_()
            g[at, tok] -= 1.0
            g *= w.unsqueeze(1)
            out["dhidden"].append(g @ head)
            dhead += g.t() @ h[r:r + 512]
    out = {k: torch.cat(v) for k, v in out.items() if v}
    out["dhead"] = dhead
    return {k: out[k] for k in dict(both=["loss", "dhidden", "dhead"], forward=["loss", "lse"],
                                    backward=["dhidden", "dhead"])[mode]}


def exact(case, seed):
    return dict(fp8=_exact_fp8, loss=_exact_loss)[case["op"]](case, seed)
