"""Host-side refusals of the FP8 block-scaled product (answered before any CUDA call)."""
import ctypes as C

import pytest
import torch

import nvfp4_draft_head_gb300 as dh

A, B, WS = 0x10000, 0x20000, 0x100000


@pytest.fixture(scope="module")
def L():
    from nvfp4_draft_head_gb300 import build
    build.build()
    return dh.lib()


def test_sizes(L):
    nb = L.fp8_block_matmul_workspace_bytes
    assert nb(1, 2560, 4608) == nb(16, 5120, 64) == 256          # quantised in the product's own kernel
    assert nb(1024, 2560, 4608) == 1024 * 2560 + 1024 * 20 * 4
    assert nb(129, 1, 1) == 129 * 16 + 240 + 768             # codes in rows of 16, one scale a token
    assert nb(200, 64026, 2560) > 200 * 64032 + 200 * 501 * 4    # a long contraction: sums of its parts too
    assert nb(16, 1 << 20, 64) > 256                             # too long for that kernel's shared memory
    for m, w, o in ((0, 16, 16), (-1, 16, 16), (1, 0, 16), (1, 16, 0), ((1 << 24) + 1, 16, 16), (1 << 24, 1 << 20, 16), (1, (1 << 24) + 1, 1)):
        assert nb(m, w, o) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), dh.DH_ERR_ARG), (dict(scale=None), dh.DH_ERR_ARG), (dict(x=None), dh.DH_ERR_ARG), (dict(y=None), dh.DH_ERR_ARG),
    (dict(xt=0), dh.DH_ERR_ARG), (dict(y=A), dh.DH_ERR_ARG), (dict(yt=4), dh.DH_ERR_ARG), (dict(ws=None), dh.DH_ERR_ARG),
    (dict(N=0), dh.DH_ERR_SHAPE), (dict(K=24), dh.DH_ERR_SHAPE), (dict(K=0), dh.DH_ERR_SHAPE), (dict(M=0), dh.DH_ERR_SHAPE),
    (dict(M=-3), dh.DH_ERR_SHAPE), (dict(M=(1 << 24) + 1), dh.DH_ERR_SHAPE), (dict(N=(1 << 24) + 1), dh.DH_ERR_SHAPE),
    (dict(ldx=127), dh.DH_ERR_SHAPE), (dict(ldy=-256), dh.DH_ERR_SHAPE),
    (dict(q=A + 8), dh.DH_ERR_ALIGN), (dict(scale=A + 2), dh.DH_ERR_ALIGN), (dict(x=A + 1), dh.DH_ERR_ALIGN),
    (dict(y=A + 2, yt=dh.DH_T_F32), dh.DH_ERR_ALIGN), (dict(err=A + 2), dh.DH_ERR_ALIGN),
    (dict(ws=WS + 16), dh.DH_ERR_WORKSPACE), (dict(nb=255), dh.DH_ERR_WORKSPACE), (dict(M=100, nb=256), dh.DH_ERR_WORKSPACE),
])
def test_products(L, kw, status):
    a = dict(N=256, K=256, q=A, scale=A, x=A, xt=dh.DH_T_BF16, ldx=256, M=4, y=B, yt=dh.DH_T_BF16, ldy=256, ws=WS, nb=1 << 20, err=None)
    a.update(kw)
    w = dh.dh_fp8_blocks_t(a["N"], a["K"], a["q"], a["scale"])
    for f in (L.fp8_block_matmul, L.fp8_block_matmul_input_gradient):
        assert f(C.byref(w), a["x"], a["xt"], a["ldx"], a["M"], a["y"], a["yt"], a["ldy"], a["ws"], a["nb"], a["err"], None) == status
        assert f(None, A, 1, 256, 4, B, 1, 256, WS, 1 << 20, None, None) == dh.DH_ERR_ARG


@pytest.mark.parametrize("args,status", [
    ((None, 300, 256, A, 256, A, A, WS, 256), dh.DH_ERR_ARG), ((A, 300, 256, None, 256, A, A, WS, 256), dh.DH_ERR_ARG),
    ((A, 300, 256, A, 256, None, A, WS, 256), dh.DH_ERR_ARG), ((A, 300, 256, A, 256, A, None, WS, 256), dh.DH_ERR_ARG),
    ((A, 300, 256, A, 256, A, A, None, 256), dh.DH_ERR_ARG), ((A, 0, 256, A, 256, A, A, WS, 256), dh.DH_ERR_SHAPE),
    ((A, 300, 264, A, 256, A, A, WS, 256), dh.DH_ERR_SHAPE), ((A, 300, 256, A, 0, A, A, WS, 256), dh.DH_ERR_SHAPE),
    ((A + 8, 300, 256, A, 256, A, A, WS, 256), dh.DH_ERR_ALIGN), ((A, 300, 256, A + 2, 256, A, A, WS, 256), dh.DH_ERR_ALIGN),
    ((A, 300, 256, A, 256, A + 8, A, WS, 256), dh.DH_ERR_ALIGN), ((A, 300, 256, A, 256, A, A, WS + 8, 256), dh.DH_ERR_WORKSPACE),
    ((A, 300, 256, A, 256, A, A, WS, 128), dh.DH_ERR_WORKSPACE),
])
def test_quantise(L, args, status):
    assert L.fp8_quantize_blocks(*args, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(role=-1), dh.DH_ERR_ARG), (dict(role=3), dh.DH_ERR_ARG), (dict(rounds=0), dh.DH_ERR_ARG), (dict(rounds=4097), dh.DH_ERR_ARG),
    (dict(err=None), dh.DH_ERR_ARG), (dict(w=False), dh.DH_ERR_ARG), (dict(x=None), dh.DH_ERR_ARG), (dict(M=0), dh.DH_ERR_SHAPE),
    (dict(x=A + 1), dh.DH_ERR_ALIGN), (dict(nb=100), dh.DH_ERR_WORKSPACE),
])
def test_wait_probe(L, kw, status):
    a = dict(w=True, x=A, M=4, nb=1 << 20, role=1, rounds=16, err=A)
    a.update(kw)
    w = C.byref(dh.dh_fp8_blocks_t(128, 256, A, A)) if a["w"] else None
    assert L.fp8_block_matmul_wait_probe(w, a["x"], a["M"], B, WS, a["nb"], a["role"], a["rounds"], a["err"], None) == status


def test_binding_refuses_host_tensors():
    q, s = torch.zeros((128, 128), dtype=torch.uint8), torch.zeros((1, 1))
    for call in (lambda: dh.FP8BlockMatmul(q, s), lambda: dh.FP8BlockMatmul(q[:, ::2], s), lambda: dh.FP8BlockMatmul(q.float(), s),
                 lambda: dh.fp8_quantize_blocks(torch.zeros((4, 16), dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            call()
