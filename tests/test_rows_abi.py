"""Host-side refusals of the operators on logits rows: every bad argument is
answered before any CUDA call, so these run without a GPU (the addresses are
never dereferenced)."""
import ctypes as C

import pytest

import nvfp4_draft_head_gb300 as dh

Z, A = 0x10000, 0x20000


@pytest.fixture(scope="module")
def L():
    from nvfp4_draft_head_gb300 import build
    build.build()
    return dh.lib()


def desc(**kw):
    d = dict(z=Z, type=dh.DH_T_BF16, M=4, C=100, ld=104, temperature=1.0, row_of=None, V=0, idx=None)
    d.update(kw)
    return C.byref(dh.dh_logits_t(*(d[f] for f, _ in dh.dh_logits_t._fields_)))


BAD = [
    (dict(z=None), dh.DH_ERR_ARG), (dict(type=0), dh.DH_ERR_ARG), (dict(type=4), dh.DH_ERR_ARG),
    (dict(temperature=0.0), dh.DH_ERR_ARG), (dict(temperature=-1.0), dh.DH_ERR_ARG),
    (dict(temperature=float("nan")), dh.DH_ERR_ARG), (dict(temperature=float("inf")), dh.DH_ERR_ARG),
    (dict(M=0), dh.DH_ERR_SHAPE), (dict(C=0), dh.DH_ERR_SHAPE), (dict(C=(1 << 30) + 1, ld=1 << 31), dh.DH_ERR_SHAPE),
    (dict(ld=99), dh.DH_ERR_SHAPE), (dict(row_of=A, V=0), dh.DH_ERR_SHAPE),
    (dict(z=Z + 1), dh.DH_ERR_ALIGN), (dict(z=Z + 2, type=dh.DH_T_F32), dh.DH_ERR_ALIGN),
    (dict(row_of=A + 2, V=9), dh.DH_ERR_ALIGN), (dict(idx=A + 1), dh.DH_ERR_ALIGN),
]


@pytest.mark.parametrize("kw,status", BAD)
def test_logits_descriptor(L, kw, status):
    d = desc(**kw)
    assert L.draft_head_token_logprobs(d, A, 1, A, A, A, 5, A, A, None) == status
    assert L.draft_head_distill(d, A, A, dh.DH_T_F32, 8, None, A, None, None, 0, None) == status
    assert L.draft_head_distill_backward(d, A, A, dh.DH_T_F32, 8, A, None, A, 104, None) == status


def test_null_descriptor(L):
    assert L.draft_head_token_logprobs(None, A, 1, A, A, A, 5, A, A, None) == dh.DH_ERR_ARG
    assert L.draft_head_distill(None, A, A, dh.DH_T_F32, 8, None, A, None, None, 0, None) == dh.DH_ERR_ARG


@pytest.mark.parametrize("args,status", [
    ((None, 1, A, A, A, 5, A, A), dh.DH_ERR_ARG), ((A, 1, None, A, A, 5, A, A), dh.DH_ERR_ARG),
    ((A, 1, A, A, A, 5, None, A), dh.DH_ERR_ARG), ((A, 1, A, A, A, 5, A, None), dh.DH_ERR_ARG),
    ((A, -1, A, A, A, 5, A, A), dh.DH_ERR_SHAPE), ((A, 1, A, A, A, 129, A, A), dh.DH_ERR_SHAPE),
    ((A, 1, A, A, A, -1, A, A), dh.DH_ERR_SHAPE), ((A + 2, 1, A, A, A, 5, A, A), dh.DH_ERR_ALIGN),
    ((A, 1, A, A + 1, A, 5, A, A), dh.DH_ERR_ALIGN), ((A, 1, A, A, A + 2, 5, A, A), dh.DH_ERR_ALIGN),
    ((A, 1, A, A, A, 5, A + 2, A), dh.DH_ERR_ALIGN),
])
def test_token_logprobs_arguments(L, args, status):
    assert L.draft_head_token_logprobs(desc(), *args, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(ids=None), dh.DH_ERR_ARG), (dict(val=None), dh.DH_ERR_ARG), (dict(vt=9), dh.DH_ERR_ARG),
    (dict(K=0), dh.DH_ERR_SHAPE), (dict(K=513), dh.DH_ERR_SHAPE), (dict(ids=A + 2), dh.DH_ERR_ALIGN),
    (dict(val=A + 2), dh.DH_ERR_ALIGN), (dict(w=A + 1), dh.DH_ERR_ALIGN), (dict(loss=None), dh.DH_ERR_ARG),
    (dict(loss=A + 2), dh.DH_ERR_ALIGN), (dict(lse=A, dz=A), dh.DH_ERR_ARG), (dict(dz=A, ld=99), dh.DH_ERR_SHAPE),
    (dict(dz=A + 1), dh.DH_ERR_ALIGN), (dict(dz=Z, ld=112), dh.DH_ERR_SHAPE),
])
def test_distill_arguments(L, kw, status):
    a = dict(ids=A, val=A, vt=dh.DH_T_F32, K=8, w=None, loss=A, lse=None, dz=None, ld=104)
    a.update(kw)
    assert L.draft_head_distill(desc(), a["ids"], a["val"], a["vt"], a["K"], a["w"], a["loss"], a["lse"], a["dz"], a["ld"],
                                None) == status
    if not set(kw) & {"loss", "lse"}:
        assert L.draft_head_distill_backward(desc(), a["ids"], a["val"], a["vt"], a["K"], A, a["w"], a["dz"] or A, a["ld"],
                                             None) == status
    assert L.draft_head_distill_backward(desc(), A, A, dh.DH_T_F32, 8, None, None, A, 104, None) == dh.DH_ERR_ARG
    assert L.draft_head_distill_backward(desc(), A, A, dh.DH_T_F32, 8, A, None, None, 104, None) == dh.DH_ERR_ARG


def test_row_map_arguments(L):
    assert L.draft_head_row_map(None, 5, A, 9, None) == dh.DH_ERR_ARG
    assert L.draft_head_row_map(A, 5, None, 9, None) == dh.DH_ERR_ARG
    assert L.draft_head_row_map(A, 0, A, 9, None) == dh.DH_ERR_SHAPE
    assert L.draft_head_row_map(A, 5, A, 0, None) == dh.DH_ERR_SHAPE
    assert L.draft_head_row_map(A + 2, 5, A, 9, None) == dh.DH_ERR_ALIGN
    assert L.draft_head_row_map(A, 5, A + 1, 9, None) == dh.DH_ERR_ALIGN
