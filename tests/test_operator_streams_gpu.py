"""The many-token operators on a stream of the caller's choice while the caller's
own stream is busy: what a call allocates must not be a block that work pending on
the caller's stream still writes."""
import pytest
import torch

import nvfp4_draft_head_gb300 as dh
from test_matmul_gpu import rand_x, weight
from test_rows_gpu import rand_rows, teacher

pytestmark = pytest.mark.gpu

BUSY = 100_000_000   # cycles: some 50 ms


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU test needs a CUDA device"
    from nvfp4_draft_head_gb300 import build
    build.build()


def tensors(out):
    if isinstance(out, dh.NVFP4Matmul):
        return [out.packed, out.error]
    return [t for t in (out if isinstance(out, tuple) else (out,)) if t is not None]


def beside_pending_work(call, scratch=()):
    """call(stream) on a side stream, with fills pending on the current one that
    write blocks freed just before the call: of every size that the call allocates,
    and of `scratch` bytes."""
    ref = call(None)
    want = [t.clone() for t in tensors(ref)]
    sizes = [t.untyped_storage().nbytes() for t in tensors(ref)] + list(scratch)
    del ref
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    junk = [torch.empty(max(n, 1), dtype=torch.uint8, device="cuda") for n in sizes for _ in range(8)]
    torch.cuda._sleep(BUSY)
    for t in junk:
        t.fill_(0x55)
    del junk, t
    out = call(side)
    assert not torch.cuda.current_stream().query(), "the caller's stream was to be busy still"
    side.synchronize()
    torch.cuda.synchronize()
    for got, ref in zip(tensors(out), want, strict=True):
        assert torch.equal(got.view(torch.uint8), ref.view(torch.uint8))


def test_product():
    q, sf, g, _ = weight(1088, 528, 1)
    mm = dh.NVFP4Matmul(q, sf, g)
    x = rand_x(150, 528, torch.bfloat16, 2)
    nb = dh.lib().nvfp4_matmul_workspace_bytes(150, 528)
    for dtype in (torch.bfloat16, torch.float32):
        beside_pending_work(lambda s: mm(x, out_dtype=dtype, stream=s), [nb])
    assert mm.device_error() == 0


def test_product_constructor():
    q, sf, g, _ = weight(1088, 528, 3)
    beside_pending_work(lambda s: dh.NVFP4Matmul(q, sf, g, stream=s))


@pytest.mark.parametrize("given", [False, True])
def test_product_from_bf16_rows(given):
    """The row ids that the call makes for itself, the quantiser's scratch and the
    weight are all made on the stream that reads them."""
    W = (torch.randn((1088, 528), generator=torch.Generator("cuda").manual_seed(4), device="cuda") * 0.02).bfloat16()
    idx = torch.arange(1087, -1, -1, dtype=torch.int32, device="cuda") if given else None
    beside_pending_work(lambda s: dh.NVFP4Matmul.from_weight(W, idx, stream=s), [1088 * 4, 1088 * 528 // 2, 1088 * 528 // 16, 4, 1024])


def test_row_map():
    idx = torch.randperm(9000, generator=torch.Generator().manual_seed(1))[:3777].int().cuda()
    beside_pending_work(lambda s: dh.draft_head_row_map(idx, 3777, 9000, stream=s))


def test_token_logprobs():
    z = rand_rows(300, 4001, torch.float32, 5)
    tokens = torch.randint(0, 4001, (300, 2), device="cuda", dtype=torch.int32)
    beside_pending_work(lambda s: dh.token_logprobs(z, tokens, top_k=20, stream=s))


@pytest.mark.parametrize("mode", ["both", "forward", "backward"])
def test_distillation(mode):
    z = rand_rows(300, 4001, torch.bfloat16, 6)
    ids, val = teacher(z, 16, 1)
    lse = dh.distill_topk_forward(z, ids, val)[1]
    call = {"both": lambda s: dh.distill_topk(z, ids, val, stream=s),
            "forward": lambda s: dh.distill_topk_forward(z, ids, val, stream=s),
            "backward": lambda s: dh.distill_topk_backward(z, ids, val, lse, stream=s)}[mode]
    beside_pending_work(call)


def test_results_outlive_the_callers_work():
    """A result dropped while the caller's stream still reads it is not handed to
    the side stream's next call."""
    q, sf, g, _ = weight(1088, 528, 1)
    mm = dh.NVFP4Matmul(q, sf, g)
    x = rand_x(150, 528, torch.bfloat16, 2)
    other = rand_x(150, 528, torch.bfloat16, 9)
    want = mm(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = mm(x, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(BUSY)
    kept = y.clone()
    del y
    later = [mm(other, stream=side) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(kept, want) and torch.equal(later[0], mm(other))


def test_device_error_waits_for_every_stream():
    """An error recorded by work still pending on another stream is read (here the
    word is set by a fill behind a busy side stream)."""
    mm = dh.NVFP4Matmul(*weight(64, 32, 1)[:3])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
        mm.error.fill_(dh.DH_DEVERR_TIMEOUT)
    assert mm.device_error() == dh.DH_DEVERR_TIMEOUT
    assert mm.device_error() == 0
