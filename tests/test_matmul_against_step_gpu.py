"""How far the many-token product (W4A4) is from the draft step (W4A16) on one head."""
import numpy as np
import pytest
import torch

import nvfp4_draft_head_gb300 as dh

pytestmark = pytest.mark.gpu


def test_four_bit_activations_change_logits_by_a_tenth_of_their_spread():
    """Rounding to E2M1 with the block's largest of 16 at 6 units: a unit is about 1.8 / 6
    = 0.3 standard deviations of a normal x, and steps are half a unit below 2 units
    (45 % of x), one unit up to 4 (32 %), two above (23 %). An error is a step / sqrt(12)
    in the mean square: sqrt(0.45 0.044^2 + 0.32 0.087^2 + 0.23 0.173^2) = 0.10. Errors of
    different x are independent, so the logits' differ by that share of their spread; the
    draft step's own rounding is below 1 %."""
    from nvfp4_draft_head_gb300 import build
    build.build()
    V, K = 6000, 256
    gen = torch.Generator("cuda").manual_seed(1)
    W = (torch.randn((V, K), generator=gen, device="cuda") * 0.02).bfloat16()
    keep = np.zeros(V, np.uint8)
    keep[np.random.default_rng(0).permutation(V)[:4096]] = 1
    idx_host, n = dh.draft_head_build_index(keep)
    idx = torch.from_numpy(idx_host).cuda()
    head, mm = dh.nvfp4_head(W, keep), dh.NVFP4Matmul.from_weight(W, idx)
    x = torch.randn((16, K), generator=gen, device="cuda").bfloat16()
    served = head.compute_logits(x)[:, idx[:n].long()]
    share = ((mm(x, out_dtype=torch.float32)[:, :n] - served).square().mean().sqrt() / served.std()).item()
    assert 0.07 < share < 0.13, share
