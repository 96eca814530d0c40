"""Routing on the GPU where f32 scores alone would choose another expert than the
definition, and over many rows."""

import math

import pytest
import torch

from oracle import model as M
from so_edge_convolution_b200 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from so_edge_convolution_b200 import build
    build.build()
    B.load()
    torch.cuda.init()


def _index(x, bias, **kw):
    """The chosen experts, after a check against the definition."""
    d = B.make_route_desc(x.shape[1], **kw)
    _, i, _ = B.route_forward(d, x.to(DEV), bias.to(DEV))
    _, ri, _ = M.route_forward(x, bias, **kw)
    assert torch.equal(i.cpu().long(), ri)
    return ri


@pytest.mark.parametrize("K,per_lane,lanes", [(128, 16, 8), (256, 16, 16), (512, 16, 32), (1024, 32, 32)])
def test_scores_that_a_sum_rounds_away(K, per_lane, lanes):
    # beside one expert's 1, exponentials just below half a step of it: each is lost
    # in an f32 sum that meets it alone, together they are 18 to 31 halves of a step
    x = torch.full((1, K), -math.inf)
    x[0, 1:per_lane] = -16.65
    x[0, [per_lane << i for i in range(int(math.log2(lanes)))]] = -16.65
    x[0, 0], x[0, K - 1] = 0.0, -60.0
    bias = torch.zeros(K)
    bias[K - 1] = 1.0 - 17 * U  # above the first one's score, which f32 takes for 1
    assert _index(x, bias, top_k=1).item() == K - 1
    assert _index(x, bias, top_k=2).tolist() == [[K - 1, 0]]
    assert _index(x, bias, top_k=9)[0, :2].tolist() == [K - 1, 0]
    bias[K - 1] = 1.0 - 40 * U  # below it
    assert _index(x, bias, top_k=1).item() == 0


@pytest.mark.parametrize("K,k", [(40, 1), (40, 10), (600, 2)])
def test_scores_far_below_an_expert_that_the_bias_takes_out(K, k):
    # -80 - 3.75e-6 rounds to -80, half a step or 63 * 2^-24 of the score: small beside
    # the largest score, large beside those that are left
    x, bias = torch.full((1, K), -200.0), torch.zeros(K)
    x[0, 0], bias[0] = 3.75e-6, -math.inf
    x[0, 1] = -80.0
    bias[2] = math.exp(-80.0 - 3.75e-6) * (1 + 5 * U)
    assert _index(x, bias, top_k=k)[0, 0] == 2


@pytest.mark.parametrize("K,k", [(40, 1), (40, 10), (600, 2)])
def test_sigmoids_that_vanish_beside_tiny_biases(K, k):
    # e^-89 is 2.2e-39, but e^89 overflows f32: the score is 0 there
    x, bias = torch.full((1, K), -200.0), torch.zeros(K)
    x[0, 3] = -89.0
    bias[1] = 1e-39
    assert _index(x, bias, top_k=k, score="sigmoid")[0, 0] == 3
    bias[1] = 3e-39
    assert _index(x, bias, top_k=k, score="sigmoid")[0, 0] == 1


# Many rows: every row's result is its own, so rows that repeat 97 others give the
# bits of a call on those, which is checked against the definition.  A grid has
# 9,472 warps at most, of one to eight rows each; every case takes several steps.
@pytest.mark.parametrize("n,K,kw", [
    (30001, 40, dict(top_k=12, renormalise=True)),                    # a warp a row, by logit
    (20003, 600, dict(top_k=3, score="sigmoid")),
    (30001, 70, dict(top_k=70)),                                      # nothing to select
    (90001, 40, dict(top_k=12, n_groups=8, top_groups=4, group_top=2)),
    (170003, 24, dict(top_k=4, renormalise=True)),                    # eight lanes a row
    (90001, 60, dict(top_k=7, score="sigmoid", renormalise=True, n_groups=5, top_groups=2,
                     group_top=2)),
    (50001, 200, dict(top_k=8)),                                      # sixteen lanes a row
    (170003, 30, dict(top_k=30, score="sigmoid", renormalise=True)),
    (30001, 64, dict(top_k=40, score="sigmoid", renormalise=True)),
])
@pytest.mark.parametrize("biased", [False, True])
def test_many_rows(n, K, kw, biased):
    g = torch.Generator().manual_seed(K)
    x = torch.randn((97, K), generator=g)
    x[torch.rand((97, K), generator=g) < 0.1] = -math.inf
    x[5] = -math.inf
    bias = (torch.randn(K, generator=g) * 0.2).to(DEV) if biased else None
    gw = torch.randn((97, kw["top_k"]), generator=g)
    d = B.make_route_desc(K, **kw)
    few = [x.to(DEV), gw.to(DEV)]
    at = torch.arange(n, device=DEV) % 97
    many = [t[at].contiguous() for t in few]
    res = []
    for xs, gs in (few, many):
        w, i, c = B.route_forward(d, xs, bias)
        res.append((w, i, B.route_backward(d, xs, i, gs), c))
    _, ri, _ = M.route_forward(x, None if bias is None else bias.cpu(), **kw)
    assert torch.equal(res[0][1].cpu().long(), ri)
    for a, b in zip(res[0][:3], res[1][:3]):
        assert torch.equal(a[at], b)
    want = torch.bincount(res[1][1][res[1][1] >= 0].long(), minlength=K)
    assert torch.equal(res[1][3].long(), want)


def test_biases_of_the_types_lowest_value():
    # every other score is near next to them, so each row is ranked in 64 bits
    g = torch.Generator().manual_seed(3)
    for K, k in ((64, 6), (300, 9)):
        x = torch.randn((200, K), generator=g)
        bias = torch.randn(K, generator=g) * 0.1
        bias[::3] = torch.finfo(torch.float32).min
        for kw in (dict(top_k=k), dict(top_k=k, score="sigmoid", n_groups=4, top_groups=2, group_top=2)):
            _index(x, bias, **kw)
