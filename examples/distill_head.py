"""Distil a drafter on the target's outputs and score it: the many-token operators together.

A stand-in target (a BF16 head over V ids) and a stand-in drafter (one linear layer
in front of the reduced-vocabulary NVFP4 head):

  teacher   token_logprobs on the target's logits: its top alternatives per token;
  student   NVFP4Matmul: the drafter's hidden states through the kept rows of the
            head, quantised once, for all tokens of the batch;
  loss      distill_topk: the loss and the gradient of the student's logits in one
            kernel, target ids mapped to the kept rows by draft_head_row_map;
  gradient  back through the kept BF16 rows (a plain library product; four-bit
            weights and activations are taken straight through) into the layer;
  scoring   token_logprobs of the target's tokens under the drafter.

Student and scores are those of the W4A4 product. A drafter that is served through the
W4A16 draft step samples from slightly other logits (see NVFP4Matmul): acceptance is
measured on DraftHead.compute_logits.

Run: python examples/distill_head.py [--steps N] (needs the GPU; sizes of the small
head: 16,384 ids, 4,000 kept, 256 wide).
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import nvfp4_draft_head_gb300 as dh  # noqa: E402
import synthetic as syn  # noqa: E402

TOKENS, TOP, RATE = 512, 32, 0.5


def main(steps: int = 30, quiet: bool = False):
    """Trains for `steps` steps; returns the mean loss of every step and, before and
    after, the share of tokens whose most likely id is the target's."""
    V, K = syn.TINY["V"], syn.TINY["K"]
    keep = syn.keep_mask(syn.SEED_KEEP_TINY, **{k: syn.TINY[k] for k in ("V", "n_kept", "forced")})
    W = torch.from_numpy(syn.head_bf16(syn.SEED_HEAD_TINY, V, K).view("int16")).cuda().view(torch.bfloat16)
    idx_host, n = dh.draft_head_build_index(keep)
    idx = torch.from_numpy(idx_host).cuda()
    head = dh.NVFP4Matmul.from_weight(W, idx)
    row_of = dh.draft_head_row_map(idx, n, V)
    kept = W[idx[:n].long()]

    gen = torch.Generator("cuda").manual_seed(7)
    mix = torch.randn((K, K), generator=gen, device="cuda") / K ** 0.5    # what the drafter has to learn
    layer = torch.eye(K, device="cuda")

    def batch(seed):
        x = torch.randn((TOKENS, K), generator=torch.Generator("cuda").manual_seed(seed), device="cuda").bfloat16()
        target = (x.float() @ mix).bfloat16() @ W.t() * 4
        teacher = dh.token_logprobs(target, top_k=TOP)
        return x, teacher.top_ids, teacher.top_logp

    def student(x):
        return head(x.float() @ layer * 4)[:, :n]     # the padding rows are left out

    def agreement(seed):
        x, ids, logp = batch(seed)
        r = dh.token_logprobs(student(x), ids[:, :1].contiguous(), top_k=1, idx=idx, row_of=row_of)
        known = row_of[ids[:, 0].long()] >= 0        # the target's token is in the draft vocabulary
        same = (r.top_ids[:, 0] == ids[:, 0])[known].float().mean().item()
        if not quiet:
            print(f"  target's token: first with the drafter in {same:.3f} of {int(known.sum())} tokens, "
                  f"mean log-probability {r.logp[known].mean().item():.3f}, entropy {r.entropy.mean().item():.3f}")
        return same

    before, losses = agreement(1), []
    weights = torch.full((TOKENS,), 1.0 / TOKENS, device="cuda")
    for step in range(steps):
        x, ids, logp = batch(100 + step)
        z = student(x)
        loss, dz = dh.distill_topk(z, ids, logp, weights=weights, row_of=row_of, dlogits=z)   # over the logits
        grad = x.float().t() @ (dz @ kept).float() * 4
        layer -= RATE * grad
        losses.append(loss.sum().item())
        if not quiet and step % 10 == 0:
            print(f"step {step}: loss {losses[-1]:.4f}")
    after = agreement(1)
    assert head.device_error() == 0
    return losses, before, after


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=30)
    main(ap.parse_args().steps)
