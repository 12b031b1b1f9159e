"""The vocabulary cross entropy at sizes that take the paths of real training: the gradient in the hidden
states in whole tiles with a last round in parts, several pieces of the vocabulary with parts, few
tokens over a vocabulary of several column blocks. Against 64 bits, with the tolerances of
test_cross_entropy_gpu; which path a size takes is read from its workspace."""
import pytest
import torch

import nvfp4_draft_head_gb300 as dh
from test_cross_entropy_gpu import check, make, near, reference

pytestmark = pytest.mark.gpu
TILE, PAIRS = 256, 76      # a tile's rows and columns; pairs of the 152 SMs


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.get_device_properties(0).multi_processor_count == 2 * PAIRS
    from nvfp4_draft_head_gb300 import build
    build.build()


def up(n, to=256):
    return -(-n // to) * to


def hidden_parts(T, N, K, piece):
    """(tiles of dh that are whole, that are in parts, parts of each) from the workspace of dh alone."""
    rows = 2 * T if T <= 128 else T
    nb = dh.lib().draft_head_cross_entropy_workspace_bytes(T, N, K, dh.DH_CE_DHIDDEN)
    parts = nb - 256 - up(rows * min(piece, up(N)) * 2) - up(rows * K * 4)
    tiles = -(-rows // TILE) * -(-K // TILE)
    rest = tiles % PAIRS
    assert parts >= 0 and parts % (rest * TILE * TILE * 4) == 0
    return tiles - rest, rest, parts // (rest * TILE * TILE * 4) + 1


def piece_of(T):
    rows = 2 * T if T <= 128 else T
    return max((1 << 28) // rows // TILE * TILE, 2048)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,N,K", [(2500, 8000, 2056), (100, 4000, 20480), (700, 20000, 6664)])
def test_whole_tiles_and_a_last_round_in_parts(T, N, K, dtype):
    whole, rest, parts = hidden_parts(T, N, K, piece_of(T))
    assert N <= piece_of(T) and whole > 0 and rest > 0 and parts > 1
    check(make(T, N, K, dtype))


# the last piece: one part of a tile, and two of four
@pytest.mark.parametrize("dtype,last", [(torch.bfloat16, 777), (torch.float16, 777), (torch.bfloat16, 2499)])
def test_pieces_of_the_vocabulary_with_parts(dtype, last):
    T, K = 40_000, 64
    piece = piece_of(T)
    N = 2 * piece + last
    whole, rest, parts = hidden_parts(T, N, K, piece)
    assert whole == 2 * PAIRS and rest == 5 and parts == 4
    steps = -(-piece // 64 // 4)             # a part's, of 64 rows
    assert -(-last // 64 // steps) == (1 if last == 777 else 2)
    s = make(T, N, K, dtype)
    out, tol, _ = reference(s)
    loss, dx, dw = dh.linear_cross_entropy(**s)
    near(loss, out["loss"], tol["loss"], "loss")
    near(dx, out["dhidden"], tol["dhidden"], "dhidden")
    near(dw, out["dhead"], tol["dhead"], "dhead")
    _, lse, rest_ = dh.linear_cross_entropy_forward(**s)
    bx, bw = dh.linear_cross_entropy_backward(s["hidden"], s["head"], s["tokens"], lse, s["weights"], rest_, s["row_of"])
    assert torch.equal(bx, dx) and torch.equal(bw, dw)
    assert dh.linear_cross_entropy_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,N,K", [(16, 4097, 136), (128, 8192, 72), (12, 33001, 136), (1, 100_000, 64)])
def test_kept_logits_of_a_large_vocabulary(T, N, K, dtype):
    """Two blocks of 4,096 columns and more, and more than 128 parts of 128 columns to a token."""
    L = dh.lib()
    nb = [L.draft_head_cross_entropy_workspace_bytes(T, N, K, o) for o in (dh.DH_CE_LOSS, dh.DH_CE_DHIDDEN | dh.DH_CE_DHEAD, 7)]
    assert nb[2] - nb[1] - (nb[0] - 256) == up(T * up(N) * 4)      # the logits
    check(make(T, N, K, dtype))
    check(make(T, N, K, dtype, mapped=True, pad_h=8, pad_w=16, seed=1))
