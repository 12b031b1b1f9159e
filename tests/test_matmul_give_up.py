"""The product's bounded waits: a role of the kernel's warps that does nothing makes
the others give up, and the kernel ends in order."""
import ctypes as C

import pytest
import torch

import nvfp4_draft_head_gb300 as dh
from test_matmul_abi import A, WS, L  # noqa: F401

PRODUCER, SCALES, ISSUER, EPILOGUE = range(4)


@pytest.mark.parametrize("kw,status", [
    (dict(role=-1), dh.DH_ERR_ARG), (dict(role=4), dh.DH_ERR_ARG), (dict(rounds=0), dh.DH_ERR_ARG),
    (dict(rounds=4097), dh.DH_ERR_ARG), (dict(err=None), dh.DH_ERR_ARG), (dict(w=False), dh.DH_ERR_ARG),
    (dict(x=None), dh.DH_ERR_ARG), (dict(M=0), dh.DH_ERR_SHAPE), (dict(N=100), dh.DH_ERR_SHAPE),
    (dict(x=A + 1), dh.DH_ERR_ALIGN), (dict(err=A + 2), dh.DH_ERR_ALIGN), (dict(nb=18432), dh.DH_ERR_WORKSPACE),
])
def test_arguments(L, kw, status):  # noqa: F811
    a = dict(w=True, N=128, x=A, M=4, nb=1 << 20, role=SCALES, rounds=16, err=A)
    a.update(kw)
    w = C.byref(dh.dh_matmul_t(a["N"], 256, A, A)) if a["w"] else None
    assert L.nvfp4_matmul_wait_probe(w, a["x"], a["M"], A, WS, a["nb"], a["role"], a["rounds"], a["err"], None) == status


# (M, N, K): one stage, less than a ring and many of them, in 128-wide tiles, one tile per SM;
# several tiles per SM (152 of them) in 128-wide and in 256-wide ones
SIZES = {"one stage": (5, 64, 256), "two stages": (40, 320, 512), "a ring and more": (130, 192, 4096),
         "three tiles": (384, 13056, 512),
         "wide tiles": (1500, 20032, 512), "wide tiles, two stages and a rest": (600, 29440, 528)}


@pytest.mark.gpu
@pytest.mark.parametrize("size, role", [(s, r) for s in SIZES for r in (PRODUCER, SCALES, ISSUER, EPILOGUE)
                                        if r != EPILOGUE or "tiles" in s])   # (one tile per SM: nobody waits for the results)
def test_an_idle_role_is_given_up_on(size, role):
    from nvfp4_draft_head_gb300 import build
    build.build()
    M, N, K = SIZES[size]
    W = (torch.randn((N, K), generator=torch.Generator("cuda").manual_seed(1), device="cuda") * 0.02).bfloat16()
    mm = dh.NVFP4Matmul.from_weight(W)
    x = torch.randn((M, K), generator=torch.Generator("cuda").manual_seed(2), device="cuda").bfloat16()
    want = mm(x)
    assert mm.device_error() == 0
    mm.wait_probe(x, role, 16)
    assert mm.device_error() == dh.DH_DEVERR_TIMEOUT
    assert mm.device_error() == 0
    assert torch.equal(mm(x), want) and mm.device_error() == 0
