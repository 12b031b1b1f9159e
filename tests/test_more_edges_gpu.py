"""Calls at the edges of what the quantisers, the FP8 block-scaled product and the vocabulary cross
entropy document: answered, or refused before anything is launched."""
import pytest
import torch

import nvfp4_draft_head_gb300 as dh

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from nvfp4_draft_head_gb300 import build
    build.build()


def rand(shape, seed=1, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=torch.Generator(DEV).manual_seed(seed), device=DEV) * scale).to(dtype)


@pytest.mark.parametrize("quantise", [dh.fp8_quantize_blocks, dh.fp8_quantize_rows, dh.nvfp4_quantize_rows])
def test_ids_that_are_not_contiguous_are_refused(quantise):
    W = rand((256, 256))
    ids = torch.arange(128, dtype=torch.int32, device=DEV)
    for bad in (ids[::2], ids[:1].expand(64)):
        with pytest.raises(ValueError, match="contiguous"):
            quantise(W, bad)
        with pytest.raises(ValueError, match="contiguous"):
            quantise(W, bad, stream=torch.cuda.Stream())
    quantise(W, ids[::2].contiguous())
