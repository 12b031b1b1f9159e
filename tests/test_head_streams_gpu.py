"""The draft head's entry points on a stream of the caller's choice while the caller's
own stream is busy (see test_operator_streams_gpu.py)."""
import numpy as np
import pytest
import torch

import nvfp4_draft_head_gb300 as dh
from test_operator_streams_gpu import beside_pending_work, built  # noqa: F401

pytestmark = pytest.mark.gpu

N, K, V = 1088, 256, 3000


def rows(n=V):
    return (torch.randn((n, K), generator=torch.Generator("cuda").manual_seed(4), device="cuda") * 0.02).bfloat16()


@pytest.fixture(scope="module")
def head():
    keep = np.zeros(V, np.uint8)
    keep[np.random.default_rng(0).permutation(V)[:N]] = 1
    return dh.nvfp4_head(rows(), keep)


@pytest.fixture(scope="module")
def h():
    return torch.randn((5, K), generator=torch.Generator("cuda").manual_seed(5), device="cuda").bfloat16()


@pytest.mark.parametrize("quantise", ["nvfp4_quantize_rows", "fp8_quantize_rows"])
def test_row_quantisers(quantise):
    """Their scratch is zeroed by a fill, which has to run before their kernels."""
    W = rows()
    idx = torch.arange(N, dtype=torch.int32, device="cuda")
    nb = dh.lib().draft_head_quantize_workspace_bytes() + dh.DH_WORKSPACE_ALIGN
    beside_pending_work(lambda s: getattr(dh, quantise)(W, idx, stream=s), [nb])


def test_pack_and_activations(h):
    q, sf, _ = dh.nvfp4_quantize_rows(rows(N), torch.arange(N, dtype=torch.int32, device="cuda"))
    beside_pending_work(lambda s: dh.nvfp4_pack_head(q, sf, stream=s))
    beside_pending_work(lambda s: dh.fp8_quantize_activations(h, stream=s))


def test_draft_step(head, h):
    beside_pending_work(lambda s: head.top_tokens(h, stream=s))
    beside_pending_work(lambda s: head.compute_logits(h, stream=s))
    beside_pending_work(lambda s: head.top_keys(h, stream=s))
    keys = head.top_keys(h)
    beside_pending_work(lambda s: dh.keys_to_ids(keys, stream=s))
    assert head.device_error() == 0


def test_linear(h):
    W = rows(N)
    lin = dh.NVFP4Linear(W)
    beside_pending_work(lambda s: lin(h, stream=s))

    def build(s):
        made = dh.NVFP4Linear(W, stream=s)
        return made.q, made.sf, made.g, made.packed
    beside_pending_work(build, [4 * N])


def test_sharded_exchange_runs_on_the_given_stream(head, h, monkeypatch):
    """The exchange (a stand-in here: one shard, whose keys and logits it rewrites on the
    current stream) is ordered between the shard's step and what follows."""
    from nvfp4_draft_head_gb300 import sharded
    seen = []

    def exchange(t, *args, **kw):
        seen.append(torch.cuda.current_stream())
        t.copy_(t.clone())
        return t

    monkeypatch.setattr(sharded, "exchange_keys", exchange)
    monkeypatch.setattr(sharded.dist, "all_reduce", exchange)
    shard = sharded.ShardedDraftHead(head)
    want_ids, want = head.top_tokens(h), head.compute_logits(h)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    ids, out = torch.empty_like(want_ids), torch.empty_like(want)
    made = shard.top_tokens(h, stream=side), shard.compute_logits(h, stream=side)
    shard.top_tokens(h, ids, stream=side)
    shard.compute_logits(h, out, stream=side)
    assert seen == [side] * 4
    side.synchronize()
    torch.cuda.synchronize()
    for got in (made, (ids, out)):
        assert torch.equal(got[0], want_ids) and torch.equal(got[1], want)
