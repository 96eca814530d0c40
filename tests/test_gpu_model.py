"""The model operators on the GPU against their float64 definitions.

Tolerances count roundings.  u = 2^-24 is half a step of f32, 2^-8 of bf16; a
sum of m terms in f32, in any order, is within (m + 1) u of its terms'
magnitudes, and a bf16 output adds 2^-8 of the value.
"""

import math

import numpy as np
import pytest
import torch

from oracle import model as M
from so_edge_convolution_b200 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
HALF = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8}
DT = {"f32": (torch.float32, B.SO2_F32), "bf16": (torch.bfloat16, B.SO2_BF16)}
TINY = 2.0 ** -126  # f32's smallest normal number; below it steps are absolute


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from so_edge_convolution_b200 import build
    build.build()
    B.load()
    torch.cuda.init()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _close(got, ref, bound, what):
    got = got.detach().cpu()
    half = HALF[got.dtype]
    err = (got.double() - ref).abs()
    lim = torch.as_tensor(bound, dtype=torch.float64) + half * ref.abs() + TINY
    bad = err > lim
    assert not bad.any(), (what, int(bad.sum()), float((err / lim).max()))


# ---- embedding ------------------------------------------------------------------
EMBED = [  # n, rows, channels, components, pad
    (1, 1, 1, 1, False), (33, 7, 5, 4, False), (64, 100, 16, 9, False), (257, 100, 16, 9, True),
    (1000, 3, 128, 1, False), (2000, 1, 7, 1, False), (3001, 70000, 20, 1, True),
    (4097, 255, 33, 1, False), (4096, 256, 64, 2, True), (9000, 2, 130, 1, True),
    (20000, 90, 4, 1, False), (5000, 66000, 3, 1, False),
]


def _embed_case(n, rows, c, s, pad, table, out, seed=0):
    g = _gen(seed)
    ids = torch.randint(0, rows, (n,), generator=g)
    ids[: n // 3] = ids[0]  # one long run
    if pad:
        ids[torch.rand(n, generator=g) < 0.3] = -1
    t = torch.randn((rows, c), generator=g).to(DT[table][0])
    G = torch.randn((n, s, c), generator=g).to(DT[out][0])
    d = B.make_embed_desc(rows, c, s, scale=0.7, table_dtype=DT[table][1], out_dtype=DT[out][1],
                          pad_id=-1 if pad else None)
    return d, ids, t, G


def _check_embed_grad(got, ids, G, rows, pad, scale=0.7):
    scale = float(np.float32(scale))
    ref, mag, count = M.embed_backward(ids, G[:, 0], rows, scale, pad)
    _close(got, ref, (count[:, None] + 2) * U * mag, "grad_table")


@pytest.mark.parametrize("table,out", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"),
                                       ("bf16", "f32")])
@pytest.mark.parametrize("n,rows,c,s,pad", EMBED)
def test_embed(n, rows, c, s, pad, table, out):
    d, ids, t, G = _embed_case(n, rows, c, s, pad, table, out)
    scale = float(np.float32(0.7))
    got = B.embed_forward(d, ids.to(DEV), t.to(DEV))
    assert B.check(DEV) == 0
    ref = M.embed_forward(ids, t, s, scale, -1 if pad else None)
    _close(got, ref, U * ref.abs(), "out")
    gt = B.embed_backward(d, ids.to(DEV), G.to(DEV))
    assert B.check(DEV) == 0
    _check_embed_grad(gt, ids, G, rows, -1 if pad else None)
    assert torch.equal(gt, B.embed_backward(d, ids.to(DEV), G.to(DEV)))


def test_embed_empty_and_all_padded():
    d = B.make_embed_desc(5, 8, 4, pad_id=-1)
    t = torch.ones((5, 8), device=DEV)
    none = torch.zeros(0, dtype=torch.int64, device=DEV)
    assert B.embed_forward(d, none, t).shape == (0, 4, 8)
    assert B.embed_backward(d, none, torch.zeros((0, 4, 8), device=DEV)).abs().max() == 0
    pad = torch.full((70,), -1, dtype=torch.int64, device=DEV)
    assert B.embed_forward(d, pad, t).abs().max() == 0
    nan = torch.full((70, 4, 8), float("nan"), device=DEV)
    assert B.embed_backward(d, pad, nan).abs().max() == 0
    assert B.check(DEV) == 0


@pytest.mark.parametrize("n", [5, 300, 10000])
def test_embed_bad_ids_give_zero_rows_and_a_status(n):
    g = _gen(3)
    ids = torch.randint(0, 9, (n,), generator=g)
    ids[1], ids[n - 1] = 9, -(1 << 62)
    t, G = torch.randn((9, 12), generator=g), torch.randn((n, 1, 12), generator=g)
    d = B.make_embed_desc(9, 12)
    out = B.embed_forward(d, ids.to(DEV), t.to(DEV))
    assert B.check(DEV) == 5 and B.check(DEV) == 0
    _close(out, M.embed_forward(ids, t, 1, 1.0), 0.0, "out")
    gt = B.embed_backward(d, ids.to(DEV), G.to(DEV))
    assert B.check(DEV) == 5
    _check_embed_grad(gt, ids, G, 9, None, 1.0)


def test_embed_strides_and_alignment():
    g = _gen(4)
    n, c = 301, 24
    ids = torch.randint(0, 11, (n,), generator=g)
    for off, width in ((0, 64), (1, 61), (4, 2 * c + 2)):
        wide = torch.full((n, width), 7.0, device=DEV)
        out = wide[:, off:off + 2 * c].unflatten(1, (2, c)) if width >= off + 2 * c else None
        base = torch.randn(11 * c + 1, generator=g).to(DEV)
        t = base[1:].view(11, c) if off == 1 else base[:-1].view(11, c)
        d = B.make_embed_desc(11, c, 2, scale=2.0)
        if out is None:
            continue
        got = B.embed_forward(d, ids.to(DEV), t, out=out)
        assert got.data_ptr() == out.data_ptr()
        assert torch.equal(got.cpu()[:, 0], t.cpu()[ids] * 2) and got[:, 1].abs().max() == 0
        keep = torch.ones(width, dtype=torch.bool)
        keep[off:off + 2 * c] = False
        assert (wide.cpu()[:, keep] == 7.0).all()  # what lies between the rows stays
        # the gradient from a slice of wider rows
        G = torch.randn((n, width), generator=g).to(DEV)
        gt = B.embed_backward(d, ids.to(DEV), G[:, off:off + 2 * c].unflatten(1, (2, c)))
        _check_embed_grad(gt, ids, G.cpu()[:, None, off:off + c], 11, None, 2.0)
    # one gradient row for all tokens (an expanded tensor)
    row = torch.randn((1, c), generator=g)
    gt = B.embed_backward(d, ids.to(DEV), row.to(DEV).expand(n, c))
    _check_embed_grad(gt, ids, row.expand(n, c)[:, None], 11, None, 2.0)
    # rows beyond the tokens stay as they were
    out = torch.full((n + 5, 2, c), 3.0, device=DEV)
    B.embed_forward(d, ids.to(DEV), t, out=out[:n])
    assert (out[n:] == 3.0).all()


# ---- routing ---------------------------------------------------------------------
def _route_case(n, K, seed, masked, dtype="f32", spread=1.0):
    g = _gen(seed)
    x = torch.randn((n, K), generator=g) * spread
    if masked:
        x[torch.rand((n, K), generator=g) < 0.3] = -math.inf
        x[n // 2] = -math.inf
    return x.to(DT[dtype][0]), torch.randn(K, generator=g) * 0.3


def _score_bound(x):
    """Relative error of an f32 softmax weight: the argument's rounding, expf
    (2 ulp), the sum of K terms and the divisions; of the renormalised one too."""
    fin = torch.where(torch.isinf(x), 0.0, x.double())
    span = (fin.amax(1) - fin.amin(1)).clamp(max=104.0)
    return ((span + x.shape[1] + 24) * 2 * U)[:, None]


def _check_route(x, bias, kw, dtype="f32", grads=True):
    d = B.make_route_desc(x.shape[1], dtype=DT[dtype][1], **kw)
    bx = None if bias is None else bias.to(DEV)
    w, i, c = B.route_forward(d, x.to(DEV), bx)
    okw = dict(kw)
    rw, ri, rc = M.route_forward(x, bias, **okw)
    assert torch.equal(i.cpu().long(), ri), "index"
    assert torch.equal(c.cpu().long(), rc), "counts"
    rel = _score_bound(x)
    _close(w, rw, rel * rw.abs(), "weights")
    assert (w.cpu()[ri < 0] == 0).all()
    if not grads:
        return
    gw = torch.randn(w.shape, generator=_gen(9))
    gw[ri < 0] = math.nan  # unused slots' gradients are not read
    got = B.route_backward(d, x.to(DEV), i, gw.to(DEV))
    soft = dict(score=kw.get("score", "softmax"), renormalise=kw.get("renormalise", False),
                scale=kw.get("scale", 1.0))
    ref = M.route_backward(x, ri, torch.nan_to_num(gw), **soft)
    # each product of the chain is a score, a weight or a gradient within `rel`;
    # sums over the slots and experts keep magnitudes below max |gw| each
    rows = rw.new_zeros(x.shape)
    s = torch.tensor([M._scores(r, soft["score"] == "softmax") for r in x.double().tolist()])
    if soft["renormalise"]:  # scores over the sum of the chosen ones
        for t in range(len(s)):
            e = [int(v) for v in ri[t] if v >= 0]
            total = s[t, e].sum()
            s[t] = s[t] / total if e and total > 0 else s[t]
            rows[t, e] = 1.0
    else:
        rows[:] = 1.0
    amp = torch.nan_to_num(gw).double().abs().amax(1, keepdim=True) * abs(soft["scale"])
    # and the reference's own roundings: for an expert that was not chosen its K top_k
    # products, each at most 2 amp and off by 2^-53 of that, cancel only to that much
    own = x.shape[1] * kw["top_k"] * 2.0 ** -51 * amp
    _close(got, ref, 4 * rel * s * rows * amp * (1 + min(kw["top_k"], 8)) + own, "grad_logits")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("n,K,k", [(1, 1, 1), (3, 2, 1), (9, 32, 32), (37, 33, 5), (16, 64, 6),
                                   (21, 100, 33), (8, 130, 130), (5, 257, 8), (4, 1024, 12),
                                   (3, 600, 600), (2, 1024, 1024)])
def test_route(n, K, k, score, renorm, masked, dtype):
    x, _ = _route_case(n, K, K + k, masked and n > 1, dtype)
    _check_route(x, None, dict(top_k=k, score=score, renormalise=renorm, scale=1.5), dtype)


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("K,k,groups,tg,gt", [(16, 2, 1, 1, 1), (64, 6, 8, 4, 2), (64, 8, 8, 4, 1),
                                              (60, 3, 5, 1, 2), (12, 12, 1, 1, 1), (48, 5, 48, 9, 1),
                                              (256, 8, 8, 4, 2), (1000, 16, 10, 3, 2),
                                              (24, 6, 4, 4, 2)])
@pytest.mark.parametrize("biased", [False, True])
def test_route_groups_and_bias(K, k, groups, tg, gt, biased, score, masked):
    x, bias = _route_case(40, K, K + groups, masked)
    kw = dict(top_k=k, score=score, n_groups=groups, top_groups=tg, group_top=gt,
              renormalise=True, scale=2.5)
    _check_route(x, bias if biased else None, kw)


def test_route_ties_go_to_the_lowest_index():
    x = torch.zeros((5, 70))
    x[1] = -torch.finfo(torch.float32).max  # the type's lowest value is an ordinary logit
    x[2, 40:] = 1.0
    x[3, ::2] = -0.0
    x[4, [3, 69]] = 2.0
    for bias in (None, torch.zeros(70)):
        _check_route(x, bias, dict(top_k=4))
        _check_route(x, bias, dict(top_k=4, n_groups=7, top_groups=2, group_top=2,
                                   renormalise=True))
    # neighbours that f32 scores cannot tell apart keep their order in 64 bits
    x = torch.full((2, 40), 3.0)
    x[0, 20] = float(np.nextafter(np.float32(3), np.float32(4)))
    x[1, 5] = float(np.nextafter(np.float32(3), np.float32(2)))
    _check_route(x, torch.zeros(40), dict(top_k=6, score="sigmoid"))
    _check_route(x, torch.full((40,), 0.125), dict(top_k=39, score="softmax"))


def test_route_far_logits():
    x = torch.tensor([[0.0, -200.0, -300.0, -1e30], [3e38, -3e38, 0.0, 1.0], [90.0, 95.0, 88.0, 0.0]])
    _check_route(x, None, dict(top_k=2, renormalise=True), grads=False)
    _check_route(x, None, dict(top_k=3, score="sigmoid"), grads=False)
    # by bias, only experts whose softmax vanishes in f32: renormalised, their ratio stays
    bias = torch.tensor([-5.0, 5.0, 5.0, 0.0])
    d = B.make_route_desc(4, 2, renormalise=True)
    w, i, _ = B.route_forward(d, torch.tensor([[0.0, -200.0, -200.5, 0.0]], device=DEV), bias.to(DEV))
    assert i.cpu().tolist() == [[1, 2]]
    assert abs(w[0, 0].item() - 1 / (1 + math.exp(-0.5))) < 4 * U
    # sigmoids that are all 0 in f32
    d = B.make_route_desc(4, 2, score="sigmoid", renormalise=True)
    w, i, _ = B.route_forward(d, torch.full((1, 4), -500.0, device=DEV))
    assert w.abs().max() == 0 and i.cpu().tolist() == [[0, 1]]
    g = B.route_backward(d, torch.full((1, 4), -500.0, device=DEV), i, torch.ones((1, 2), device=DEV))
    assert g.abs().max() == 0


def test_route_nan_and_infinite_bias():
    nan, inf = math.nan, math.inf
    x = torch.tensor([[0.0, nan, 1.0, -inf, 2.0], [nan, nan, nan, -inf, nan]])
    d = B.make_route_desc(5, 4, score="sigmoid")
    w, i, c = B.route_forward(d, x.to(DEV))
    assert i.cpu().tolist() == [[4, 2, 0, 1], [0, 1, 2, 4]]
    assert torch.isfinite(w[0, :3]).all() and torch.isnan(w[0, 3]) and torch.isnan(w[1]).all()
    bias = torch.tensor([-inf, 0.0, inf, 0.0, 0.0])
    w, i, c = B.route_forward(B.make_route_desc(5, 3), torch.zeros((1, 5), device=DEV), bias.to(DEV))
    assert i.cpu().tolist() == [[2, 1, 3]] and c.cpu().tolist() == [0, 1, 1, 1, 0]
    assert (w == w[0, 0]).all() and abs(w[0, 0].item() - 0.2) < 4 * U
    d = B.make_route_desc(5, 5)
    w, i, _ = B.route_forward(d, torch.zeros((1, 5), device=DEV), bias.to(DEV))
    assert i.cpu().tolist() == [[-1, 1, 2, 3, 4]] and w[0, 0] == 0


def test_route_backward_takes_any_index():
    # an expert named twice adds up; indices outside the experts are unused slots
    x = torch.randn((3, 9), generator=_gen(5))
    index = torch.tensor([[2, 2, 5], [-1, 8, 9], [1 << 30, -7, -1]], dtype=torch.int32)
    gw = torch.randn((3, 3), generator=_gen(6))
    for score in ("softmax", "sigmoid"):
        d = B.make_route_desc(9, 3, score=score)
        got = B.route_backward(d, x.to(DEV), index.to(DEV), gw.to(DEV))
        ref = M.route_backward(x, index, gw, score)
        # magnitudes of at most 3 max |gw| and a few tens of roundings
        _close(got, ref, 200 * U * gw.abs().max().item(), score)
        assert got[2].abs().max() == 0


def test_route_many_rows_and_none():
    d = B.make_route_desc(8, 2)
    w, i, c = B.route_forward(d, torch.zeros((0, 8), device=DEV))
    assert w.shape == (0, 2) and c.abs().max() == 0
    assert B.route_backward(d, torch.zeros((0, 8), device=DEV), i, w).shape == (0, 8)
    x = torch.randn((50001, 8), generator=_gen(1))
    w, i, c = B.route_forward(d, x.to(DEV))
    assert torch.equal(i.cpu().long(), torch.sort(x, dim=1, descending=True, stable=True)[1][:, :2])
    assert int(c.sum()) == 100002
    assert torch.equal(c.cpu().long(), torch.bincount(i.cpu().flatten().long(), minlength=8))


# ---- mixing ------------------------------------------------------------------------
MIX = [  # systems, experts, slots (None: every expert in order), weights
    (6, 40, 12, 260), (9, 30, 16, 132), (97, 50, 3, 132), (40, 20, 2, 1028), (3, 6, 6, 132),
    (15, 17, None, 2052), (16, 16, None, 2052), (6, 8, None, 1028), (4, 4, None, 77), (20, 30, 30, 516),
    (1, 1, None, 1), (1, 32, None, 4864), (3, 5, None, 33), (2, 7, 3, 130), (33, 64, 4, 1000),
    (64, 32, None, 2052), (17, 9, 9, 515), (5, 130, None, 257), (70, 3, 2, 96), (130, 40, 5, 260),
    (4, 8, 2, 70001), (9, 128, None, 1028),
]


def _mix_case(T, K, k, n, experts, out, seed=0):
    g = _gen(seed)
    e = torch.randn((K, n), generator=g).to(DT[experts][0])
    kk = K if k is None else k
    w = torch.randn((T, kk), generator=g)
    index = None
    if k is not None:
        index = torch.randint(-1, K, (T, k), generator=g).to(torch.int32)
        index[0] = index[0, 0]  # the same expert in every slot
        if T > 2:
            index[2] = -1       # a system without any expert
    d = B.make_mix_desc(K, n, kk, expert_dtype=DT[experts][1], out_dtype=DT[out][1])
    G = torch.randn((T, n), generator=g)
    return d, e, w, index, G


def _dev(t):
    return None if t is None else t.to(DEV)


@pytest.mark.parametrize("experts,out", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"),
                                         ("bf16", "f32")])
@pytest.mark.parametrize("T,K,k,n", MIX)
def test_mix(T, K, k, n, experts, out):
    d, e, w, index, G = _mix_case(T, K, k, n, experts, out)
    if index is not None:
        w[index < 0] = math.nan  # unused slots' weights are not read
        named = torch.bincount((index + 1).flatten().long(), minlength=K + 1)[1:]
        e[named == 0] = math.nan  # nor are experts that no slot names
    got = B.mix_experts_forward(d, _dev(e), _dev(w), _dev(index))
    assert B.check(DEV) == 0
    w0 = torch.nan_to_num(w)
    ref, mag = M.mix_forward(e, w0, index)
    _close(got, ref, (w.shape[1] + 2) * U * mag, "out")
    g = B.mix_experts_backward(d, _dev(e), _dev(w), _dev(G), index=_dev(index))
    assert B.check(DEV) == 0
    (ge, me), (gw, mw) = M.mix_backward(e, w0, G, index)
    _close(g["grad_experts"], ge, (T * w.shape[1] + 2) * U * me, "grad_experts")
    _close(g["grad_weights"], gw, (n + 2) * U * mw, "grad_weights")
    again = B.mix_experts_backward(d, _dev(e), _dev(w), _dev(G), index=_dev(index))
    for name in g:
        assert torch.equal(g[name], again[name]), name
    for name in g:  # one at a time, the same
        one = B.mix_experts_backward(d, _dev(e), _dev(w), _dev(G), index=_dev(index), need=[name])
        assert set(one) == {name} and torch.equal(one[name], g[name])


@pytest.mark.parametrize("experts,out", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("T,K,n", [(16, 32, 128), (33, 31, 4), (64, 64, 1500), (130, 40, 516),
                                   (65, 17, 300), (20, 256, 260), (24, 300, 132), (40, 33, 40004),
                                   (100, 129, 1028), (64, 32, 60004), (33, 24, 20000), (64, 12, 516),
                                   (48, 32, 128 * 148 * 3 + 4)])
def test_mix_large_dense(T, K, n, experts, out):
    # shapes whose products are matrix products; 40,004 columns make a block take several tiles
    d, e, w, _, G = _mix_case(T, K, None, n, experts, out, seed=T)
    got = B.mix_experts_forward(d, _dev(e), _dev(w))
    ref, mag = M.mix_forward(e, w)
    _close(got, ref, (K + 2) * U * mag, "out")
    g = B.mix_experts_backward(d, _dev(e), _dev(w), _dev(G))
    assert B.check(DEV) == 0
    (ge, me), (gw, mw) = M.mix_backward(e, w, G)
    _close(g["grad_experts"], ge, (T + 2) * U * me, "grad_experts")
    _close(g["grad_weights"], gw, (n + 2) * U * mw, "grad_weights")
    again = B.mix_experts_backward(d, _dev(e), _dev(w), _dev(G))
    for name in g:
        assert torch.equal(g[name], again[name]), name


@pytest.mark.parametrize("experts", ["f32", "bf16"])
def test_mix_infinities_and_nan_stay_in_their_columns(experts):
    d, e, w, _, G = _mix_case(48, 40, None, 400, experts, "f32", seed=7)
    big = 3.0e38  # its product with a weight below 1 is finite
    e[3, 130], e[7, 5], e[9, 300] = math.inf, math.nan, big
    w[:, 9] *= 0.1 / w[:, 9].abs().max()
    G[1, 399], G[2, 17] = -math.inf, math.nan
    got = B.mix_experts_forward(d, _dev(e), _dev(w)).cpu().double()
    ref = w.double() @ e.double()
    bad = torch.zeros(400, dtype=torch.bool)
    bad[[130, 5, 300]] = True
    assert torch.isfinite(got[:, ~bad]).all()
    _, mag = M.mix_forward(e[:, ~bad], w)
    assert ((got - ref)[:, ~bad].abs() <= 42 * U * mag).all()
    assert torch.equal(got[:, 130], torch.where(w[:, 3] > 0, math.inf, -math.inf).double())
    assert torch.isnan(got[:, 5]).all()
    assert ((got - ref)[:, 300].abs() <= 42 * U * (w.double().abs() @ e.double().abs())[:, 300]).all()
    g = B.mix_experts_backward(d, _dev(torch.zeros_like(e)), _dev(w), _dev(G), need=["grad_experts"])
    ge = g["grad_experts"].cpu()
    assert torch.isnan(ge[:, 17]).all() and torch.isinf(ge[:, 399]).all()
    ge[:, [17, 399]] = 0
    assert torch.isfinite(ge).all()


@pytest.mark.parametrize("experts", ["f32", "bf16"])
def test_mix_gradients_with_infinities_and_nan(experts):
    d, e, w, _, G = _mix_case(40, 30, None, 1000, experts, "f32", seed=8)
    G[1, 900], G[2, 17], e[4, 500], e[5, 200] = -math.inf, math.nan, math.inf, math.nan
    g = B.mix_experts_backward(d, _dev(e), _dev(w), _dev(G))
    one = B.mix_experts_backward(d, _dev(e), _dev(w), _dev(G), need=["grad_weights"])
    assert B.check(DEV) == 0
    (ge, me), (gw, mw) = M.mix_backward(e, w, G)
    for name, got, ref, mag in (("grad_experts", g["grad_experts"], ge, 42 * U * me),
                                ("grad_weights", g["grad_weights"], gw, 1002 * U * mw),
                                ("grad_weights alone", one["grad_weights"], gw, 1002 * U * mw)):
        got = got.cpu().double()
        assert torch.equal(torch.isnan(got), torch.isnan(ref)), name
        assert torch.equal(torch.isinf(got), torch.isinf(ref)), name
        inf, fin = torch.isinf(ref), torch.isfinite(ref)
        assert torch.equal(got[inf], ref[inf]), name
        assert ((got - ref)[fin].abs() <= mag[fin] + TINY).all(), name


def test_mix_bad_index_is_skipped_with_a_status():
    d, e, w, index, G = _mix_case(6, 5, 3, 40, "f32", "f32")
    index[1, 0], index[4, 2] = 5, -2
    ref, mag = M.mix_forward(e, w, index)
    got = B.mix_experts_forward(d, _dev(e), _dev(w), _dev(index))
    assert B.check(DEV) == 5
    _close(got, ref, 5 * U * mag, "out")
    g = B.mix_experts_backward(d, _dev(e), _dev(w), _dev(G), index=_dev(index))
    assert B.check(DEV) == 5
    (ge, me), (gw, mw) = M.mix_backward(e, w, G, index)
    _close(g["grad_experts"], ge, 20 * U * me, "grad_experts")
    _close(g["grad_weights"], gw, 42 * U * mw, "grad_weights")


def test_mix_no_systems_and_unaligned():
    d = B.make_mix_desc(3, 10)
    e = torch.ones((3, 10), device=DEV)
    none = torch.zeros((0, 3), device=DEV)
    assert B.mix_experts_forward(d, e, none).shape == (0, 10)
    g = B.mix_experts_backward(d, e, none, torch.zeros((0, 10), device=DEV))
    assert g["grad_experts"].abs().max() == 0 and g["grad_weights"].shape == (0, 3)
    for dt in ("f32", "bf16"):  # pointers one element off a vector's boundary
        d, e, w, index, G = _mix_case(3, 6, None, 64, dt, dt, seed=2)
        shift = lambda t: torch.cat([t.flatten()[:1], t.flatten()]).to(DEV)[1:].view(t.shape)  # noqa
        out = torch.zeros(3 * 64 + 1, dtype=DT[dt][0], device=DEV)[1:].view(3, 64)
        got = B.mix_experts_forward(d, shift(e), shift(w), out=out)
        ref, mag = M.mix_forward(e, w)
        _close(got, ref, 8 * U * mag, "out")
        g = B.mix_experts_backward(d, shift(e), shift(w), shift(G))
        (ge, me), (gw, mw) = M.mix_backward(e, w, G)
        _close(g["grad_experts"], ge, 5 * U * me, "grad_experts")
        _close(g["grad_weights"], gw, 66 * U * mw, "grad_weights")


# ---- dropout -------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("unit", ["element", "channel", "row"])
@pytest.mark.parametrize("n,s,c", [(1, 1, 1), (7, 4, 5), (13, 9, 16), (5, 25, 20), (3, 1, 130),
                                   (40, 4, 8), (2, 3, 257), (9, 2, 6)])
def test_dropout(n, s, c, unit, dtype):
    g = _gen(n + c)
    dt = DT[dtype][0]
    x, res = torch.randn((n, s, c), generator=g).to(dt), torch.randn((n, s, c), generator=g).to(dt)
    rows = torch.randint(-(1 << 60), 1 << 60, (n,), generator=g)
    for p, seed, offset, r, a in ((0.3, 12345, 0, None, rows), (0.5, -1, (1 << 63) - 1, res, None),
                                  (0.0, 1, 2, res, None), (1.0, 1, 2, None, None),
                                  (1.0, 1, 2, res, None)):
        a = a if unit == "row" else None
        d = B.make_dropout_desc(c, s, unit, p, DT[dtype][1])
        rng = torch.tensor([seed, offset], device=DEV)
        keep = M.dropout_keep((n, s, c), unit, p, seed, offset, None if a is None else a.tolist())
        bad = x.clone()
        bad[~keep] = math.nan  # what is dropped is not used
        got = B.dropout(d, bad.to(DEV), rng, residual=_dev(r), rows=_dev(a))
        ref = M.dropout(x, keep, p, r)
        mag = M.dropout(x, keep, p).abs() + (0 if r is None else r.double().abs())
        _close(got, ref, 3 * U * mag, "out")
        if r is None:
            assert (got.cpu()[~keep] == 0).all()


def test_dropout_in_place_and_empty():
    d = B.make_dropout_desc(12, 3, "channel", 0.4)
    rng = torch.tensor([5, 6], device=DEV)
    x, res = (torch.randn((50, 3, 12), generator=_gen(i)).to(DEV) for i in (0, 1))
    want = B.dropout(d, x, rng, residual=res)
    a, b = x.clone(), res.clone()
    assert torch.equal(B.dropout(d, a, rng, residual=res, out=a), want)
    assert torch.equal(B.dropout(d, x, rng, residual=b, out=b), want)
    assert B.dropout(d, x[:0], rng).shape == (0, 3, 12)
    # offset pointers, and rows beyond the tensor left as they were
    base = torch.full((50 * 36 + 40,), 9.0, device=DEV)
    view = base[1:1 + 50 * 36].view(50, 3, 12)
    view.copy_(x)
    assert torch.equal(B.dropout(d, view, rng, residual=res, out=view), want)
    assert base[0] == 9.0 and (base[1 + 50 * 36:] == 9.0).all()


def test_dropout_backward_is_the_same_call():
    # <G, drop(x)> = <drop(G), x>, exactly the same mask
    d = B.make_dropout_desc(16, 4, "element", 0.3)
    rng = torch.tensor([77, 3], device=DEV)
    x, G = (torch.randn((31, 4, 16), generator=_gen(i)).to(DEV) for i in (2, 3))
    gx = B.dropout(d, G, rng)
    y = B.dropout(d, x, rng)
    assert torch.equal(gx != 0, y != 0)
    assert abs(((G * y).double().sum() - (gx * x).double().sum()).item()) < 1e-4


# ---- together --------------------------------------------------------------------------
def _chain_inputs(seed=0):
    import oracle as O
    from so_edge_convolution_b200 import synth
    p = synth.make_problem("esen", seed=seed, n_atoms=60, max_nb=8, lmax=2, mmax=1, c=16)
    g = _gen(seed)
    Z = torch.randint(0, 12, (60,), generator=g)
    nw = p.w.size
    return dict(p=p, O=O, Z=Z, nw=nw, table=torch.randn((12, 16), generator=g),
                experts=torch.randn((6, nw), generator=g) / 8, wr=torch.randn((16, 6), generator=g),
                bias=torch.randn(6, generator=g) * 0.1, G=torch.randn((60, 9, 16), generator=g))


def test_the_operators_around_the_convolution():
    """Embedding -> router on the mean embedding -> mixed weights -> convolution ->
    channel dropout onto the residual, and the gradients of the table, the experts
    and the router, against the same chain in 64 bits."""
    c = _chain_inputs()
    p, O = c["p"], c["O"]
    t = lambda a: torch.as_tensor(np.asarray(a)).float().to(DEV)  # noqa: E731
    ei = torch.as_tensor(p.edge_index).to(DEV)
    ev, wrad, brad = t(p.edge_vec), t(p.w_rad), t(p.b_rad)
    ids, table, experts = c["Z"].to(DEV), c["table"].to(DEV), c["experts"].to(DEV)
    rng = torch.tensor([11, 4], device=DEV)
    ed = B.make_embed_desc(12, 16, 9)
    rd = B.make_route_desc(6, 3, renormalise=True)
    md = B.make_mix_desc(6, c["nw"], 3)
    dd = B.make_dropout_desc(16, 9, "channel", 0.25)
    cd = B.make_desc(2, 1, 16, 16, p.n_rbf, p.rbf_cutoff)
    G = c["G"].to(DEV)

    x = B.embed_forward(ed, ids, table)
    assert B.check(DEV) == 0
    mean = x[:, 0].mean(0, keepdim=True)
    logits = mean @ c["wr"].to(DEV)
    w, index, _ = B.route_forward(rd, logits, c["bias"].to(DEV))
    wmix = B.mix_experts_forward(md, experts, w, index)
    y = B.forward(cd, x, ei, ev, wmix[0], wrad, brad)
    assert B.check(DEV) == 0
    out = B.dropout(dd, y, rng, residual=x)
    gy = B.dropout(dd, G, rng)
    gc = B.backward(cd, x, ei, ev, wmix[0], wrad, brad, gy)
    gm = B.mix_experts_backward(md, experts, w, gc["grad_w"][None], index=index)
    gl = B.route_backward(rd, logits, index, gm["grad_weights"])
    gx = G + gc["grad_x"]
    gx[:, 0] += (gl @ c["wr"].to(DEV).T) / 60
    gt = B.embed_backward(ed, ids, gx)
    assert B.check(DEV) == 0

    # the same in 64 bits
    od = O.Desc(2, 1, 16, 16, p.n_rbf, p.rbf_cutoff)
    f = lambda a: torch.as_tensor(np.asarray(a)).float().double()  # noqa: E731
    rx = M.embed_forward(c["Z"], c["table"], 9, 1.0)
    rl = rx[:, 0].mean(0, keepdim=True) @ c["wr"].double()
    rw, ri, _ = M.route_forward(rl, c["bias"], top_k=3, renormalise=True)
    assert torch.equal(ri, index.cpu().long())
    rmix, _ = M.mix_forward(c["experts"], rw, ri)
    args = (rx, torch.as_tensor(p.edge_index[0]), torch.as_tensor(p.edge_index[1]), f(p.edge_vec),
            rmix[0], f(p.w_rad), f(p.b_rad), od)
    ry = O.forward(*args)
    keep = M.dropout_keep((60, 9, 16), "channel", 0.25, 11, 4)
    rout = M.dropout(ry, keep, 0.25, rx)
    rgc = O.backward(*args, M.dropout(c["G"], keep, 0.25))
    (rge, _), (rgw, _) = M.mix_backward(c["experts"], rw, rgc["grad_w"][None], ri)
    rgl = M.route_backward(rl, ri, rgw, renormalise=True)
    rgx = c["G"].double() + rgc["grad_x"]
    rgx[:, 0] += (rgl @ c["wr"].double().T) / 60
    rgt, _, _ = M.embed_backward(c["Z"], rgx[:, 0], 12, 1.0)
    for name, got, ref in (("out", out, rout), ("grad_experts", gm["grad_experts"], rge),
                           ("grad_logits", gl, rgl), ("grad_table", gt, rgt)):
        # the convolution's own tolerance on its f32 path, over the chain's few steps
        err = (got.double().cpu() - ref).abs().max() / ref.abs().max()
        assert err < 4e-4, (name, float(err))


def test_offsets_beyond_32_bits():
    # one tensor of over 2^31 elements at a time; the far end is looked at
    n, c = 34000, 65536
    d = B.make_dropout_desc(c, 1, "element", 0.5, B.SO2_BF16)
    x = torch.ones((n, 1, c), dtype=torch.bfloat16, device=DEV)
    rng = torch.tensor([3, 4], device=DEV)
    B.dropout(d, x, rng, out=x)
    keep = [M.philox((m // 4) | (4 << 64), 3)[m % 4] >= 1 << 31
            for m in range((n - 1) * c, (n - 1) * c + 64)]
    assert x[n - 1, 0, :64].float().cpu().tolist() == [2.0 if k else 0.0 for k in keep]
    # embedding rows and their gradient 2^26 elements apart
    wide = x.view(-1)[: 33 << 26].view(33, 1 << 26)
    ids = (torch.arange(33) % 5).to(DEV)
    t = torch.randn((5, 48), generator=_gen(1)).to(DEV)
    ed = B.make_embed_desc(5, 48, out_dtype=B.SO2_BF16)
    B.embed_forward(ed, ids, t, out=wide[:, 64:112].unflatten(1, (1, 48)))
    assert torch.equal(wide[:, 64:112].cpu(), t.bfloat16()[ids].cpu())
    gt = B.embed_backward(ed, ids, wide[:, 64:112])
    _check_embed_grad(gt, ids.cpu(), wide[:, None, 64:112].cpu(), 5, None, 1.0)
    # 33 experts of 2^26 weights, by index and in order
    w = torch.randn((1, 33), generator=_gen(2)).to(DEV)
    e = wide[:, -8:].float().cpu()
    for k, index in ((33, None), (2, torch.tensor([[32, 31]], dtype=torch.int32, device=DEV))):
        md = B.make_mix_desc(33, 1 << 26, k, B.SO2_BF16, B.SO2_F32)
        got = B.mix_experts_forward(md, wide, w[:, :k].contiguous(), index=index)
        ref, mag = M.mix_forward(e, w[:, :k].cpu(), index)
        _close(got[:, -8:], ref, (k + 2) * U * mag, "out")
    G = torch.ones((1, 1 << 26), device=DEV)
    g = B.mix_experts_backward(md, wide, w[:, :2].contiguous(), G, index=index)
    assert (g["grad_experts"][32] == w[0, 0]).all() and (g["grad_experts"][:31] == 0).all()


def _all_ops(s):
    """Every operator once on the state's tensors."""
    r = [B.embed_forward(s["ed"], s["ids"], s["table"]),
         B.embed_backward(s["ed"], s["ids"], s["G"])]
    w, i, c = B.route_forward(s["rd"], s["logits"], s["bias"])
    r += [w, i, c, B.route_backward(s["rd"], s["logits"], i, s["gw"])]
    r += [B.mix_experts_forward(s["md"], s["experts"], w, i)]
    r += list(B.mix_experts_backward(s["md"], s["experts"], w, s["GW"], index=i).values())
    r += [B.mix_experts_forward(s["mdd"], s["experts"], s["dense"])]
    r += list(B.mix_experts_backward(s["mdd"], s["experts"], s["dense"], s["GW"]).values())
    r += [B.dropout(s["dd"], s["G"], s["rng"], residual=s["res"])]
    return r


def _all_state(seed, n=700, T=20, K=24, k=4, nw=1000):
    g = _gen(seed)
    f = lambda *a: torch.randn(a, generator=g).to(DEV)  # noqa: E731
    return dict(ed=B.make_embed_desc(50, 24, 4), ids=torch.randint(0, 50, (n,), generator=g).to(DEV),
                table=f(50, 24), G=f(n, 4, 24), res=f(n, 4, 24),
                rd=B.make_route_desc(K, k, "sigmoid", n_groups=4, top_groups=2, group_top=2,
                                     renormalise=True),
                logits=f(T, K), bias=f(K), gw=f(T, k), md=B.make_mix_desc(K, nw, k),
                mdd=B.make_mix_desc(K, nw), dense=f(T, K), experts=f(K, nw), GW=f(T, nw),
                dd=B.make_dropout_desc(24, 4, "element", 0.3),
                rng=torch.tensor([seed, 1], device=DEV))


def test_captured_graphs_replay_on_new_inputs():
    states = [_all_state(1), _all_state(2)]
    eager = [[t.clone() for t in _all_ops(s)] for s in states]
    live = {k: (v.clone() if torch.is_tensor(v) else v) for k, v in states[0].items()}
    graphs = []
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):  # two graphs, captured before either is replayed
        for _ in range(2):
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr, stream=side):
                outs = _all_ops(live)
            graphs.append((gr, outs))
    torch.cuda.synchronize()
    for which in (1, 0, 1):
        for k, v in states[which].items():
            if torch.is_tensor(v):
                live[k].copy_(v)
        torch.cuda.synchronize()
        for gr, outs in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for gr, outs in graphs:
            for a, b in zip(outs, eager[which]):
                assert torch.equal(a, b)


def test_streams_side_by_side():
    states = [_all_state(i, n=500 + 900 * i) for i in range(3)]
    want = [[t.clone() for t in _all_ops(s)] for s in states]
    streams = [torch.cuda.Stream() for _ in states]
    torch.cuda.synchronize()
    got = [None] * 3
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = _all_ops(states[i])
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for a, b in zip(g, w):
            assert torch.equal(a, b)


def test_a_callers_workspace():
    s = _all_state(4)
    ws = B.Workspace(DEV)
    bad = s["ids"].clone()
    bad[5] = 50
    B.embed_backward(s["ed"], bad, s["G"], ws=ws)
    B.embed_backward(s["ed"], s["ids"], s["G"])
    assert B.check(DEV) == 0 and B.check(DEV, ws=ws) == 5 and B.check(DEV, ws=ws) == 0


def test_launches_are_counted():
    s = _all_state(5)
    before = B.launch_count()
    B.embed_forward(s["ed"], s["ids"], s["table"])
    B.dropout(s["dd"], s["G"], s["rng"])
    assert B.launch_count() >= before + 2
