"""Host-side refusals of the vocabulary cross entropy (answered before any CUDA call)."""
import ctypes as C

import pytest
import torch

import nvfp4_draft_head_gb300 as dh

A, B, WS, D = 0x10000, 0x20000, 0x100000, 0x101000


@pytest.fixture(scope="module")
def L():
    from nvfp4_draft_head_gb300 import build
    build.build()
    return dh.lib()


def test_sizes(L):
    nb = L.draft_head_cross_entropy_workspace_bytes
    assert nb(1, 1, 8, dh.DH_CE_LOSS) == 256 + 4 * 256                                 # two parts, three rows of floats
    assert nb(4096, 64026, 2560, dh.DH_CE_LOSS) == 256 + 4096 * 2 * 251 * 8 + 3 * 4096 * 4
    assert nb(4096, 64026, 2560, dh.DH_CE_DHEAD) == 256 + 4096 * 64256 * 2 + 4096 * 2560 * 2
    assert nb(131072, 248320, 2560, dh.DH_CE_DHEAD) == 256 + (1 << 29) + 131072 * 2560 * 2   # g of a piece: 512 MiB
    assert nb(1, 100, 8, 7) < nb(1, 100, 8, 7 ^ dh.DH_CE_LOSS) + (1 << 12)
    for t, n, k, o in ((0, 1, 8, 1), (1, 0, 8, 1), (1, 1, 12, 1), (1, 1, 0, 1), (1, 1, 8, 0), (1, 1, 8, 8), ((1 << 24) + 1, 1, 8, 1),
                       (1, (1 << 24) + 1, 8, 1), (1, 1, (1 << 20) + 8, 1), (1 << 24, 1 << 24, 8, 1)):
        assert nb(t, n, k, o) == 0


BAD = [
    (dict(hidden=None), dh.DH_ERR_ARG), (dict(head=None), dh.DH_ERR_ARG), (dict(tokens=None), dh.DH_ERR_ARG),
    (dict(type=dh.DH_T_F32), dh.DH_ERR_ARG), (dict(type=0), dh.DH_ERR_ARG),
    (dict(T=0), dh.DH_ERR_SHAPE), (dict(N=0), dh.DH_ERR_SHAPE), (dict(K=100), dh.DH_ERR_SHAPE), (dict(K=0), dh.DH_ERR_SHAPE),
    (dict(T=(1 << 24) + 1), dh.DH_ERR_SHAPE), (dict(ld_hidden=120), dh.DH_ERR_SHAPE), (dict(ld_head=-128), dh.DH_ERR_SHAPE),
    (dict(ld_head=1 << 39), dh.DH_ERR_SHAPE), (dict(row_of=A, V=0), dh.DH_ERR_SHAPE),
    (dict(hidden=A + 8), dh.DH_ERR_ALIGN), (dict(head=B + 2), dh.DH_ERR_ALIGN), (dict(ld_hidden=132), dh.DH_ERR_ALIGN),
    (dict(ld_head=129), dh.DH_ERR_ALIGN), (dict(tokens=A + 2), dh.DH_ERR_ALIGN), (dict(weight=A + 1), dh.DH_ERR_ALIGN),
    (dict(row_of=A + 2, V=9), dh.DH_ERR_ALIGN),
]


def desc(**kw):
    d = dict(hidden=A, head=B, type=dh.DH_T_BF16, T=4, K=128, N=100, ld_hidden=128, ld_head=128, tokens=A, weight=None, row_of=None, V=0)
    d.update(kw)
    return C.byref(dh.dh_cross_entropy_t(*(d[f] for f, _ in dh.dh_cross_entropy_t._fields_)))


@pytest.mark.parametrize("kw,status", BAD)
def test_descriptor(L, kw, status):
    d, n = desc(**kw), 1 << 30
    assert L.draft_head_cross_entropy(d, A, A, A, None, 0, None, 0, WS, n, None, None) == status
    assert L.draft_head_cross_entropy_backward(d, A, None, WS, 128, None, 0, WS, n, None, None) == status
    assert L.draft_head_cross_entropy_wait_probe(d, A, WS, n, 1, 16, A, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(loss=None), dh.DH_ERR_ARG), (dict(ws=None), dh.DH_ERR_ARG), (dict(dh=A), dh.DH_ERR_ARG), (dict(dw=B), dh.DH_ERR_ARG), (dict(dw=WS), dh.DH_ERR_ARG),
    (dict(ldh=120), dh.DH_ERR_SHAPE), (dict(ldw=0), dh.DH_ERR_SHAPE), (dict(dh=WS + 8), dh.DH_ERR_ALIGN), (dict(ldw=132), dh.DH_ERR_ALIGN),
    (dict(loss=A + 2), dh.DH_ERR_ALIGN), (dict(lse=A + 1), dh.DH_ERR_ALIGN), (dict(rest=A + 1), dh.DH_ERR_ALIGN), (dict(err=A + 1), dh.DH_ERR_ALIGN),
    (dict(ws=WS + 64), dh.DH_ERR_WORKSPACE), (dict(nb=4096), dh.DH_ERR_WORKSPACE),
])
def test_outputs(L, kw, status):
    a = dict(loss=A, lse=None, rest=None, dh=WS, ldh=128, dw=D, ldw=128, ws=WS, nb=1 << 30, err=None)
    a.update(kw)
    assert L.draft_head_cross_entropy(desc(), a["loss"], a["lse"], a["rest"], a["dh"], a["ldh"], a["dw"], a["ldw"], a["ws"], a["nb"], a["err"],
                                      None) == status


@pytest.mark.parametrize("args,status", [
    ((None, None, WS, 128, D, 128), dh.DH_ERR_ARG), ((A, None, None, 0, None, 0), dh.DH_ERR_ARG), ((A, None, D, 128, D, 128), dh.DH_ERR_ARG),
    ((A, A + 2, WS, 128, D, 128), dh.DH_ERR_ALIGN), ((A + 2, None, WS, 128, D, 128), dh.DH_ERR_ALIGN),
])
def test_backward(L, args, status):
    assert L.draft_head_cross_entropy_backward(desc(), *args, WS, 1 << 30, None, None) == status
    assert L.draft_head_cross_entropy_backward(None, A, None, WS, 128, None, 0, WS, 1 << 30, None, None) == dh.DH_ERR_ARG


@pytest.mark.parametrize("loss,role,rounds,err", [(None, 0, 1, A), (A, -1, 1, A), (A, 3, 1, A), (A, 0, 0, A), (A, 0, 4097, A), (A, 0, 1, None)])
def test_wait_probe(L, loss, role, rounds, err):
    assert L.draft_head_cross_entropy_wait_probe(desc(), loss, WS, 1 << 20, role, rounds, err, None) == dh.DH_ERR_ARG


def test_binding_refuses():
    h, W, t = torch.zeros((4, 16), dtype=torch.bfloat16), torch.zeros((9, 16), dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    for call in (dh.linear_cross_entropy, dh.linear_cross_entropy_forward, dh.LinearCrossEntropy.apply):
        with pytest.raises(ValueError):
            call(h, W, t)
    with pytest.raises(ValueError, match="at least one"):
        dh.linear_cross_entropy_backward(h, W, t, torch.zeros(4), dhidden=False, dhead=False)
