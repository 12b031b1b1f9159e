"""Refusals and workspace sizes of the FP8 block-scaled product and of the vocabulary cross entropy that
need no GPU."""
import ctypes as C

import pytest

import nvfp4_draft_head_gb300 as dh


@pytest.fixture(scope="module")
def L():
    from nvfp4_draft_head_gb300 import build
    build.build()
    return dh.lib()


def test_error_word(L):
    assert L.draft_head_cross_entropy_error_word(None) == dh.DH_ERR_ARG


@pytest.mark.parametrize("M,width,out", [(16, 2560, 20000), (16, 5120, 64026), (64, 5120, 64026), (5, 8192, 64026)])
def test_few_tokens_have_no_room_for_parts(L, M, width, out):
    """Codes and scales alone, where the product of few tokens reads them (the parts of the contraction
    are another form's)."""
    def up(n):
        return -(-n // 256) * 256
    assert L.fp8_block_matmul_workspace_bytes(M, width, out) == up(M * width) + up(M * width // 128 * 4)


def test_two_terms_of_the_gradient(L):
    nb = L.draft_head_cross_entropy_workspace_bytes
    assert nb(300, 1000, 64, dh.DH_CE_TWO_TERMS) == 0
    assert nb(300, 1000, 64, dh.DH_CE_LOSS | dh.DH_CE_TWO_TERMS) == nb(300, 1000, 64, dh.DH_CE_LOSS)
    assert nb(128, 1000, 64, 7 | dh.DH_CE_TWO_TERMS) == nb(128, 1000, 64, 7)
    # g and the copy of the hidden states once more
    assert nb(2048, 4096, 64, dh.DH_CE_DHEAD | dh.DH_CE_TWO_TERMS) >= nb(2048, 4096, 64, dh.DH_CE_DHEAD) + 2048 * 4096 * 2 + 2048 * 64 * 2
    # small products of up to 1,024 tokens have both terms anyway (T N K <= 2^28)
    for size, both in (((1024, 1024, 256), True), ((1024, 1025, 256), False), ((1025, 1024, 8), False), ((129, 1, 8), True), ((200, 64026, 16), True),
                       ((200, 64026, 24), False)):
        assert (nb(*size, 6) == nb(*size, 6 | dh.DH_CE_TWO_TERMS)) == both
    for t in (0, dh.DH_T_F32, 4, dh.DH_T_BF16 | 16):
        d = dh.dh_cross_entropy_t(0x10000, 0x20000, t | dh.DH_CE_TWO_TERMS, 4, 128, 100, 128, 128, 0x10000, None, None, 0)
        assert L.draft_head_cross_entropy(C.byref(d), 0x10000, None, None, None, 0, None, 0, 0x100000, 1 << 30, None, None) == dh.DH_ERR_ARG
