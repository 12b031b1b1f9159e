"""Refusals of the operators on logits rows at the ends of their arguments' ranges
(answered before any CUDA call; the addresses are never dereferenced)."""
import ctypes as C
from types import SimpleNamespace

import pytest
import torch

import nvfp4_draft_head_gb300 as dh
from test_rows_abi import A, L, desc  # noqa: F401


@pytest.mark.parametrize("t", [1e-45, 2e-39, 3e-39, 4.2e-39])
def test_temperatures_whose_scale_overflows(L, t):  # noqa: F811
    """1 / t, or the exponents' scale log2(e) / t, is infinite in fp32."""
    d = desc(temperature=t)
    assert L.draft_head_token_logprobs(d, A, 1, A, A, A, 5, A, A, None) == dh.DH_ERR_ARG
    assert L.draft_head_distill(d, A, A, dh.DH_T_F32, 8, None, A, None, None, 0, None) == dh.DH_ERR_ARG
    assert L.draft_head_distill_backward(d, A, A, dh.DH_T_F32, 8, A, None, A, 104, None) == dh.DH_ERR_ARG


def test_the_smallest_temperature_gets_past_that_check(L):  # noqa: F811
    assert L.draft_head_token_logprobs(desc(temperature=4.3e-39), A, -1, A, A, A, 5, A, A, None) == dh.DH_ERR_SHAPE


def stand_in(M, n):
    """What the descriptor is made from, without the memory."""
    return SimpleNamespace(dtype=torch.float32, shape=(M, n), is_cuda=True, device=torch.device("cuda:0"), dim=lambda: 2,
                           stride=lambda: (n, 1), data_ptr=lambda: A)


@pytest.mark.parametrize("M, n, t, status", [
    (4, 100, "1", dh.DH_ERR_ARG), (4, 100, None, dh.DH_ERR_ARG), (4, 100, 10 ** 400, dh.DH_ERR_ARG),
    (2 ** 31, 100, 1.0, dh.DH_ERR_SHAPE), (1, 2 ** 31, 1.0, dh.DH_ERR_SHAPE)],
                         ids=["text", "none", "past float64", "rows", "columns"])
def test_arguments_past_the_descriptors_fields(L, M, n, t, status):  # noqa: F811
    with pytest.raises(dh.DraftHeadError) as e:
        dh._logits_desc(stand_in(M, n), t, None)
    assert e.value.status == status
    assert len(dh._logits_desc(stand_in(4, 100), 1.0, None)) == C.sizeof(dh.dh_logits_t)


@pytest.mark.parametrize("t", [1e39, -1e39, 1e300, 1e-50])
def test_temperatures_that_fp32_does_not_hold(L, t):  # noqa: F811
    """They become infinite or zero in the descriptor, which the library refuses."""
    d = dh._logits_desc(stand_in(4, 100), t, None)
    assert L.draft_head_token_logprobs(d, A, 1, A, A, A, 5, A, A, None) == dh.DH_ERR_ARG
