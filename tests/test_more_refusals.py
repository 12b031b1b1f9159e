"""Refusals of the FP8 block-scaled product and of the vocabulary cross entropy that need no GPU."""
import pytest

import nvfp4_draft_head_gb300 as dh


@pytest.fixture(scope="module")
def L():
    from nvfp4_draft_head_gb300 import build
    build.build()
    return dh.lib()


def test_error_word(L):
    assert L.draft_head_cross_entropy_error_word(None) == dh.DH_ERR_ARG
