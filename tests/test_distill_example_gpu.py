"""The example that runs the many-token operators together learns."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu


def test_distilling_the_small_head():
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import distill_head
    losses, before, after = distill_head.main(steps=40, quiet=True)
    assert losses[-1] < 0.7 * losses[0], losses[::8]
    assert after > before + 0.1, (before, after)
