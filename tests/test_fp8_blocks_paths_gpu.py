"""The FP8 block-scaled product of many tokens in each way that its tiles are split: wide and narrow
tiles, all of them in parts of the contraction or those behind whole rounds over the SMs. Against 64
bits, with the tolerances of test_fp8_blocks_gpu; which way a size takes is read from its workspace."""
import pytest
import torch

import nvfp4_draft_head_gb300 as dh
from test_fp8_blocks_gpu import BF, F, HF, check, layer, quantise, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from nvfp4_draft_head_gb300 import build
    build.build()


def up(n, to=256):
    return -(-n // to) * to


# (tokens, results, features), the tiles' width, whole tiles, parts
WAYS = [((100, 20112, 2496), 128, 152, 5), ((129, 656, 6560), 256, 0, 13), ((100, 40192, 1040), 256, 152, 2), ((400, 19536, 1424), 256, 304, 3),
        ((129, 112, 1520), 128, 0, 3)]


@pytest.mark.parametrize("size,tn,whole,parts", WAYS)
@pytest.mark.parametrize("grad,tx,ty", [(False, BF, F), (True, HF, BF)])
def test_ways(size, tn, whole, parts, grad, tx, ty):
    M, out, width = size
    tiles = -(-M // 128) * -(-out // tn)
    nb = dh.lib().fp8_block_matmul_workspace_bytes(M, width, out) - up(M * up(width, 16)) - up(M * -(-width // 128) * 4)
    assert nb == up(4 * parts * (M * up(out, 8) if whole == 0 else (tiles - whole) * 128 * tn))
    mm, wv = layer(*((width, out) if grad else (out, width)))
    x = rows(M, width, tx)
    call = mm.input_gradient if grad else mm
    y = call(x, out_dtype=ty)
    check(y, quantise(x, 1)[2], wv if grad else wv.t(), width)
    odd = torch.full((M, out + 3), 7.0, dtype=ty, device="cuda")     # rows at odd addresses
    call(x, odd[:, 1:out + 1])
    assert torch.equal(odd[:, 1:out + 1], y) and (odd[:, out + 1:] == 7).all() and (odd[:, 0] == 7).all()
    assert mm.device_error() == 0
