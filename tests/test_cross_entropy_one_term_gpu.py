"""The vocabulary cross entropy of more than 1,024 tokens, whose g has one 16-bit term at any size (small
products of fewer have two): small and odd sizes, strides, rows that are left out and that are not
finite, given results. Against 64 bits, with the tolerances of test_cross_entropy_gpu."""
import pytest
import torch

import nvfp4_draft_head_gb300 as dh
from test_cross_entropy_gpu import DEV, check, make, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from nvfp4_draft_head_gb300 import build
    build.build()


def one_term(T, N, K):
    nb = dh.lib().draft_head_cross_entropy_workspace_bytes
    return nb(T, N, K, 6) < nb(T, N, K, 6 | dh.DH_CE_TWO_TERMS)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,N,K", [(1025, 1, 8), (1026, 2, 8), (1030, 257, 72), (1300, 700, 200), (2000, 41, 1032), (6000, 5, 520), (1100, 2561, 136)])
def test_sizes(T, N, K, dtype):
    assert one_term(T, N, K)
    check(make(T, N, K, dtype))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("pad_h,pad_w,mapped", [(8, 0, False), (0, 24, True), (72, 8, True)])
def test_strides_and_maps(pad_h, pad_w, mapped, dtype):
    check(make(1200, 700, 136, dtype, pad_h=pad_h, pad_w=pad_w, mapped=mapped))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("scale", [1e-30, 1.0, -300.0])
def test_row_weights(dtype, scale):
    s = make(1040, 300, 72, dtype)
    s["weights"] *= scale
    s["weights"][5::9] *= 1e-3
    if dtype == torch.float16 and abs(scale) < 1e-6:
        s["weights"] *= 1e26       # f16 results hold no less
    check(s)


def test_rows_that_are_left_out_and_not_finite():
    s = make(1100, 500, 136, torch.bfloat16)
    want = dh.linear_cross_entropy(**s)
    _, _, live = reference(s)
    junk = s["hidden"].clone()
    junk[~live] = float("nan")
    junk[(~live).nonzero()[::2, 0]] = float("inf")
    for a, b in zip(dh.linear_cross_entropy(**{**s, "hidden": junk}), want):
        assert torch.equal(a, b)
    assert not want[0][~live].any() and not want[1][~live].any()
    bad = s["hidden"].clone()
    rows = live.nonzero()[[3, 700], 0]
    bad[rows[0], 3], bad[rows[1], 0] = float("nan"), float("inf")
    loss, dx, dw = dh.linear_cross_entropy(**{**s, "hidden": bad})
    others = torch.ones(1100, dtype=torch.bool, device=DEV)
    others[rows] = False
    assert loss[rows].isnan().all() and dx[rows].isnan().all() and dw.isnan().any()
    assert torch.equal(loss[others], want[0][others]) and torch.equal(dx[others], want[1][others])


def test_given_results():
    s = make(1100, 40, 64, torch.float16, dead=False)
    want = dh.linear_cross_entropy(**s)
    dx = torch.full((1100, 96), 3.0, dtype=torch.float16, device=DEV)
    dw = torch.full((42, 72), 3.0, dtype=torch.float16, device=DEV)
    got = dh.linear_cross_entropy(**s, dhidden=dx[:, 16:80], dhead=dw[1:41, :64])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert (dx[:, :16] == 3).all() and (dx[:, 80:] == 3).all() and (dw[0] == 3).all() and (dw[41] == 3).all() and (dw[:, 64:] == 3).all()
    lse = dh.linear_cross_entropy_forward(**s)[1]
    a = (s["hidden"], s["head"], s["tokens"], lse, s["weights"])
    both = dh.linear_cross_entropy_backward(*a)
    assert torch.equal(dh.linear_cross_entropy_backward(*a, dhead=False)[0], both[0])
    assert torch.equal(dh.linear_cross_entropy_backward(*a, dhidden=False)[1], both[1])


def test_graph():
    s, t = make(1100, 700, 136, torch.bfloat16), make(1100, 700, 136, torch.bfloat16, seed=5)
    want = {id(a): dh.linear_cross_entropy(**a) for a in (s, t)}
    static = {k: None if v is None else v.clone() for k, v in s.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = dh.linear_cross_entropy(**static)
    for a in (s, t, s):
        for k, v in static.items():
            if v is not None:
                v.copy_(a[k])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, want[id(a)]))
    assert dh.linear_cross_entropy_device_error() == 0
