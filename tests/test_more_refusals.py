"""Refusals and workspace sizes of the FP8 block-scaled product and of the vocabulary cross entropy that
need no GPU."""
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
