"""The many-token operators launch on the current device: tensors on another one
are refused before any launch (the current device is a stand-in here)."""
from types import SimpleNamespace

import pytest
import torch

import nvfp4_draft_head_gb300 as dh


def test_stream_of_a_tensor_elsewhere_is_refused(monkeypatch):
    monkeypatch.setattr(dh, "_current_device", lambda: 0)
    monkeypatch.setattr(dh, "_raw_stream", lambda device: 77 + device)
    assert dh._stream_of(SimpleNamespace(get_device=lambda: 0)) == 77
    with pytest.raises(ValueError, match="cuda:1"):
        dh._stream_of(SimpleNamespace(get_device=lambda: 1))


@pytest.mark.gpu
def test_every_operator_refuses(monkeypatch):
    from nvfp4_draft_head_gb300 import build
    build.build()
    f32, i32 = dict(device="cuda"), dict(device="cuda", dtype=torch.int32)
    W = torch.randn((64, 32), **f32).bfloat16()
    q, sf, g = dh.nvfp4_quantize_rows(W, torch.arange(64, **i32))
    mm = dh.NVFP4Matmul(q, sf, g)
    z, x = torch.randn((4, 64), **f32), torch.randn((4, 32), **f32)
    ids, val, lse = torch.zeros((4, 2), **i32), torch.zeros((4, 2), **f32), torch.zeros(4, **f32)
    idx = torch.arange(64, **i32)
    side = torch.cuda.Stream()
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
        for call in (lambda: mm(x, stream=stream), lambda: dh.NVFP4Matmul(q, sf, g, stream=stream),
                     lambda: dh.NVFP4Matmul.from_weight(W, stream=stream),
                     lambda: dh.draft_head_row_map(idx, 64, 64, stream=stream),
                     lambda: dh.token_logprobs(z, stream=stream), lambda: dh.distill_topk(z, ids, val, stream=stream),
                     lambda: dh.distill_topk_forward(z, ids, val, stream=stream),
                     lambda: dh.distill_topk_backward(z, ids, val, lse, stream=stream)):
            with pytest.raises(ValueError, match="cuda:0"):
                call()
    assert launched == []
