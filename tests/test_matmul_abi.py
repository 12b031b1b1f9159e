"""Host-side refusals of the many-token product (answered before any CUDA call)."""
import ctypes as C

import pytest

import nvfp4_draft_head_gb300 as dh

A, WS = 0x10000, 0x100000


@pytest.fixture(scope="module")
def L():
    from nvfp4_draft_head_gb300 import build
    build.build()
    return dh.lib()


def test_sizes(L):
    assert L.nvfp4_matmul_packed_bytes(64, 16) == 18432
    assert L.nvfp4_matmul_packed_bytes(64064, 2560) == 501 * 10 * 18432
    assert L.nvfp4_matmul_workspace_bytes(1, 16) == 18432 + 256
    assert L.nvfp4_matmul_workspace_bytes(129, 2560) == 2 * 10 * 18432 + 768
    for n, k in ((0, 16), (63, 16), (64, 8), (64, 0), (-64, 16), (64, 24), ((1 << 24) + 64, 16), (64, (1 << 20) + 16)):
        assert L.nvfp4_matmul_packed_bytes(n, k) == 0
    for m, k in ((0, 16), (-1, 16), (1, 17), ((1 << 24) + 1, 16)):
        assert L.nvfp4_matmul_workspace_bytes(m, k) == 0


@pytest.mark.parametrize("args,status", [
    ((None, A, 64, 16, A), dh.DH_ERR_ARG), ((A, None, 64, 16, A), dh.DH_ERR_ARG), ((A, A, 64, 16, None), dh.DH_ERR_ARG),
    ((A, A, 60, 16, A), dh.DH_ERR_SHAPE), ((A, A, 64, 8, A), dh.DH_ERR_SHAPE), ((A + 8, A, 64, 16, A), dh.DH_ERR_ALIGN),
    ((A, A, 64, 16, A + 8), dh.DH_ERR_ALIGN),
])
def test_pack_arguments(L, args, status):
    assert L.nvfp4_pack_matmul(*args, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(packed=None), dh.DH_ERR_ARG), (dict(scale=None), dh.DH_ERR_ARG), (dict(x=None), dh.DH_ERR_ARG),
    (dict(y=None), dh.DH_ERR_ARG), (dict(xt=0), dh.DH_ERR_ARG), (dict(yt=4), dh.DH_ERR_ARG), (dict(ws=None), dh.DH_ERR_ARG),
    (dict(N=100), dh.DH_ERR_SHAPE), (dict(K=40), dh.DH_ERR_SHAPE), (dict(M=0), dh.DH_ERR_SHAPE),
    (dict(M=(1 << 24) + 1), dh.DH_ERR_SHAPE), (dict(ldx=255), dh.DH_ERR_SHAPE), (dict(ldy=127), dh.DH_ERR_SHAPE),
    (dict(packed=A + 8), dh.DH_ERR_ALIGN), (dict(scale=A + 2), dh.DH_ERR_ALIGN), (dict(x=A + 1), dh.DH_ERR_ALIGN),
    (dict(y=A + 2, yt=dh.DH_T_F32), dh.DH_ERR_ALIGN), (dict(err=A + 2), dh.DH_ERR_ALIGN),
    (dict(ws=WS + 16), dh.DH_ERR_WORKSPACE), (dict(nb=18432), dh.DH_ERR_WORKSPACE),
])
def test_matmul_arguments(L, kw, status):
    a = dict(N=128, K=256, packed=A, scale=A, x=A, xt=dh.DH_T_BF16, ldx=256, M=4, y=A, yt=dh.DH_T_BF16, ldy=128, ws=WS,
             nb=1 << 20, err=None)
    a.update(kw)
    w = dh.dh_matmul_t(a["N"], a["K"], a["packed"], a["scale"])
    assert L.nvfp4_matmul(C.byref(w), a["x"], a["xt"], a["ldx"], a["M"], a["y"], a["yt"], a["ldy"], a["ws"], a["nb"], a["err"],
                          None) == status
    assert L.nvfp4_matmul(None, A, 1, 256, 4, A, 1, 128, WS, 1 << 20, None, None) == dh.DH_ERR_ARG
