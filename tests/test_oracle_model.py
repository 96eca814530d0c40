"""Pins of the float64 definitions of the model operators: published vectors of
the generator, central differences of the gradients, hand-written selections."""

import math

import pytest
import torch

from oracle import model as M


def test_generator_known_answers():
    # the published known-answer vectors of Philox-4x32-10
    assert M.philox(0, 0) == [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]
    assert M.philox((1 << 128) - 1, (1 << 64) - 1) == [0x408f276d, 0x41c83b0e, 0xa20bc7c6,
                                                       0x6d5451fd]


def test_keep_rate():
    keep = M.dropout_keep((40, 5, 20), "element", 0.25, 7, 3)
    # 4,000 draws: a standard deviation of 0.0068; six of them
    assert abs(keep.double().mean().item() - 0.75) < 0.042
    one = M.dropout_keep((40, 5, 20), "channel", 0.25, 7, 3)
    assert (one == one[:, :1]).all()


def test_hand_written_selections():
    inf = math.inf
    s, chosen, w = M.route_row([0.0, 1.0, 1.0, -inf], None, 2, True)
    assert chosen == [1, 2] and w[0] == w[1]
    assert M.route_row([-inf] * 3, None, 2, True)[1:] == ([-1, -1], [0.0, 0.0])
    # a bias selects but does not weigh
    s, chosen, w = M.route_row([0.0, 0.0, 0.0], [0.0, 0.0, 5.0], 1, False)
    assert chosen == [2] and w == [0.5]
    # groups by the sum of two: (3, 0) loses to (2, 2) although it has the best expert
    args = dict(top_k=1, softmax=False, n_groups=2, top_groups=1)
    x = [3.0, -9.0, 2.0, 2.0]
    assert M.route_row(x, None, group_top=2, **args)[1] == [2]
    assert M.route_row(x, None, group_top=1, **args)[1] == [0]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_against_differences(score, renorm):
    g = torch.Generator().manual_seed(0)
    x = torch.randn((3, 6), generator=g, dtype=torch.float64)
    gw = torch.randn((3, 2), generator=g, dtype=torch.float64)
    kw = dict(top_k=2, score=score, renormalise=renorm, scale=1.5)
    _, index, _ = M.route_forward(x, None, **kw)
    got = M.route_backward(x, index, gw, score, renorm, 1.5)
    h = 1e-6
    for t in range(3):
        for e in range(6):
            d = []
            for sign in (1, -1):
                y = x.clone()
                y[t, e] += sign * h
                w, i2, _ = M.route_forward(y, None, **kw)
                assert (i2 == index).all()
                d.append((w * gw).sum().item())
            # second-order differences: h^2 and 2^-53 / h, both about 1e-10
            assert abs((d[0] - d[1]) / (2 * h) - got[t, e].item()) < 1e-8


def test_mix_gradients_are_the_adjoints():
    g = torch.Generator().manual_seed(1)
    experts = torch.randn((5, 7), generator=g, dtype=torch.float64)
    w = torch.randn((4, 3), generator=g, dtype=torch.float64)
    index = torch.tensor([[0, 1, 1], [4, -1, 2], [-1, -1, -1], [3, 3, 3]])
    G = torch.randn((4, 7), generator=g, dtype=torch.float64)
    out, _ = M.mix_forward(experts, w, index)
    (ge, _), (gw, _) = M.mix_backward(experts, w, G, index)
    value = (G * out).sum()
    # linear in either argument
    assert abs((ge * experts).sum() - value) < 1e-12
    assert abs((gw * w).sum() - value) < 1e-12
    assert gw[2].abs().max() == 0 and gw[1, 1] == 0


def test_embed_gradient_is_the_adjoint():
    g = torch.Generator().manual_seed(2)
    ids = torch.tensor([0, 3, 3, -1, 9, 2])
    table = torch.randn((4, 5), generator=g, dtype=torch.float64)
    G = torch.randn((6, 5), generator=g, dtype=torch.float64)
    out = M.embed_forward(ids, table, 3, 0.5, pad_id=-1)
    grad, _, count = M.embed_backward(ids, G, 4, 0.5, pad_id=-1)
    assert abs((G * out[:, 0]).sum() - (grad * table).sum()) < 1e-12
    assert out[:, 1:].abs().max() == 0 and count.tolist() == [1, 0, 1, 2]
