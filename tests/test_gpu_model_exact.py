"""Sums of the model operators over many tiles, at values whose results are known
to the bit: integers whose sums f32 holds, and rows picked out by a single 1.
"""

import math

import pytest
import torch

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


def _gen(seed):
    return torch.Generator().manual_seed(seed)


# ---- embedding gradient: more tokens than 64 tiles of the sort -----------------------
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,rows,c", [(65537, 100, 32), (70001, 3, 20), (300007, 60000, 8),
                                      (131073, 70001, 5), (1000003, 100, 12), (262144, 1, 4)])
def test_embedding_gradient_of_many_tokens(n, rows, c, dtype):
    g = _gen(n)
    ids = torch.randint(0, rows, (n,), generator=g)
    ids[torch.rand(n, generator=g) < 0.4] = rows // 2  # one long run
    ids[torch.rand(n, generator=g) < 0.05] = -1
    G = torch.randint(-8, 9, (n, c), generator=g)  # sums below 2^24: any order is exact
    d = B.make_embed_desc(rows, c, scale=0.5, out_dtype=B.SO2_F32 if dtype == torch.float32 else B.SO2_BF16,
                          pad_id=-1)
    got = B.embed_backward(d, ids.to(DEV), G.to(dtype).to(DEV)[:, None])
    keep = ids >= 0
    ref = torch.zeros((rows, c), dtype=torch.int64).index_add_(0, ids[keep], G[keep])
    assert ref.abs().max() < 1 << 24
    assert torch.equal(got.cpu(), ref.float() * 0.5)
    assert B.check(DEV) == 0


# ---- mixing ---------------------------------------------------------------------------
# Blocks of the tensor-core products take the tiles of 128 columns 296 (forward, one
# or two a processor) or 148 (both gradients) apart.
WIDE = 128 * 296 * 3 + 4
# A value is picked out through its three parts, which are added from the smallest on:
# exact, but for a last bit where the first part is a power of two above the value.
PICKED = 2 * U


def _near(got, ref, what):
    got, ref = got.cpu().double(), ref.double()
    bad = ~((got - ref).abs() <= PICKED * ref.abs())
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[0].tolist())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,K,n", [(32, 32, WIDE), (64, 64, WIDE), (48, 33, WIDE), (70, 32, WIDE - 128),
                                   (40, 256, 128 * 148 * 3 + 4)])
def test_mixing_of_picked_experts(T, K, n, dtype):
    g = _gen(T + K)
    code = B.SO2_F32 if dtype == torch.float32 else B.SO2_BF16
    d = B.make_mix_desc(K, n, expert_dtype=code)
    e = torch.randn((K, n), generator=g).to(dtype)
    pick = torch.randint(0, K, (T,), generator=g)
    w = torch.nn.functional.one_hot(pick, K).float()
    _near(B.mix_experts_forward(d, e.to(DEV), w.to(DEV)), e[pick], "experts")
    # the weights through experts that are 1 in columns of their own
    e = torch.nn.functional.one_hot(torch.arange(n) % K, K).t().to(dtype).contiguous()
    w = torch.randn((T, K), generator=g)
    got = B.mix_experts_forward(d, e.to(DEV), w.to(DEV))
    _near(got, w[:, torch.arange(n) % K], "weights")
    # integers: products and sums of fewer than 24 bits
    e = torch.randint(-128, 129, (K, n), generator=g)
    w = torch.randint(-128, 129, (T, K), generator=g)
    got = B.mix_experts_forward(d, e.to(dtype).to(DEV), w.float().to(DEV))
    assert torch.equal(got.cpu().double(), w.double() @ e.double())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,K,n", [(64, 32, 128 * 148 * 4 + 4), (40, 20, 128 * 148 * 3 + 60),
                                   (64, 33, 30004), (70, 40, 20000), (12, 30, 128 * 148 * 3), (3, 7, 70000)])
def test_gradients_of_picked_rows(T, K, n, dtype):
    g = _gen(T * K)
    d = B.make_mix_desc(K, n, expert_dtype=B.SO2_F32 if dtype == torch.float32 else B.SO2_BF16)
    e, G = torch.randn((K, n), generator=g).to(dtype), torch.randn((T, n), generator=g)
    # experts' gradient: one system's row each; its weights' gradient: one column each
    pick = torch.randint(0, T, (K,), generator=g)
    w = torch.zeros((T, K))
    w[pick, torch.arange(K)] = 1.0
    for trial in range(3):
        at = torch.randint(0, n, (K,), generator=g)
        at[0], at[1 % K], at[2 % K] = 0, n - 1, n // 2
        one = torch.zeros((K, n), dtype=dtype)
        one[torch.arange(K), at] = 1.0
        r = B.mix_experts_backward(d, one.to(DEV), w.to(DEV), G.to(DEV))
        _near(r["grad_experts"], G[pick], "grad_experts")
        _near(r["grad_weights"], G[:, at], "grad_weights from grad_out")
        at = torch.randint(0, n, (T,), generator=g)
        one = torch.zeros((T, n))
        one[torch.arange(T), at] = 1.0
        r = B.mix_experts_backward(d, e.to(DEV), w.to(DEV), one.to(DEV))
        _near(r["grad_weights"], e[:, at].t().float(), "grad_weights from experts")
    # integers whose sums over all columns stay below 2^24
    e, G = torch.randint(-4, 5, (K, n), generator=g), torch.randint(-4, 5, (T, n), generator=g)
    w = torch.randint(-128, 129, (T, K), generator=g)
    r = B.mix_experts_backward(d, e.to(dtype).to(DEV), w.float().to(DEV), G.float().to(DEV))
    assert torch.equal(r["grad_experts"].cpu().double(), w.double().t() @ G.double())
    assert torch.equal(r["grad_weights"].cpu().double(), G.double() @ e.double().t())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tile", [[0], [1], [2], [3], [0, 2], [1, 2, 3], [0, 1, 2, 3]])
def test_infinities_in_a_blocks_tiles(tile, dtype):
    # integers again, with infinities in some of the tiles of one block
    g = _gen(len(tile))
    for K, apart in ((32, 296), (64, 296), (256, 148)):
        n = 128 * apart * 3 + 132
        e = torch.randint(-64, 65, (K, n), generator=g).double()
        w = torch.randint(-64, 65, (32, K), generator=g).double()
        w[w == 0] = 1.0
        cols = [128 * apart * t + 7 for t in tile]
        e[3, cols] = math.inf
        d = B.make_mix_desc(K, n, expert_dtype=B.SO2_F32 if dtype == torch.float32 else B.SO2_BF16)
        got = B.mix_experts_forward(d, e.to(dtype).to(DEV), w.float().to(DEV)).cpu().double()
        assert torch.equal(got, w @ e)
    # the joint gradients: a tile with one is computed apart, from both operands
    T, K, n = 64, 32, 128 * 148 * 3 + 132
    for into in ("experts", "grad_out"):
        e = torch.randint(-4, 5, (K, n), generator=g).double()
        G = torch.randint(-4, 5, (T, n), generator=g).double()
        w = torch.randint(-64, 65, (T, K), generator=g).double()
        e[e == 0], G[G == 0], w[w == 0] = 1.0, 1.0, 1.0  # (0 times infinity is NaN)
        cols = [128 * 148 * t + 7 for t in tile]
        (e if into == "experts" else G)[5, cols] = math.inf
        want = {"grad_experts": w.t() @ G, "grad_weights": G @ e.t()}
        want["grad_weights"][want["grad_weights"].isnan()] = 0.0  # inf - inf, both here and there
        d = B.make_mix_desc(K, n, expert_dtype=B.SO2_F32 if dtype == torch.float32 else B.SO2_BF16)
        r = B.mix_experts_backward(d, e.to(dtype).to(DEV), w.float().to(DEV), G.float().to(DEV))
        for name, ref in want.items():
            assert torch.equal(torch.nan_to_num(r[name].cpu().double(), 0.0, math.inf, -math.inf), ref), name
    assert B.check(DEV) == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_infinite_weights(dtype):
    # the forward and the experts' gradient are computed apart; the weights' gradient does not see them
    g = _gen(3)
    for T, K in ((64, 32), (48, 40), (5, 6)):
        n = 128 * 148 * 2 + 12
        e = torch.randint(-4, 5, (K, n), generator=g).double()
        G = torch.randint(-4, 5, (T, n), generator=g).double()
        w = torch.randint(-64, 65, (T, K), generator=g).double()
        e[e == 0], G[G == 0] = 1.0, 1.0
        w[3, 2] = math.inf
        d = B.make_mix_desc(K, n, expert_dtype=B.SO2_F32 if dtype == torch.float32 else B.SO2_BF16)
        args = [t.to(DEV) for t in (e.to(dtype), w.float())]
        assert torch.equal(B.mix_experts_forward(d, *args).cpu().double(), w @ e)
        r = B.mix_experts_backward(d, *args, G.float().to(DEV))
        assert torch.equal(r["grad_experts"].cpu().double(), w.t() @ G)
        assert torch.equal(r["grad_weights"].cpu().double(), G @ e.t())


@pytest.mark.parametrize("T,K,n", [(64, 32, 60004), (33, 24, 20000), (70, 40, 40004), (16, 16, 128 * 148 * 3)])
def test_error_of_the_weights_gradient(T, K, n):
    # Of random operands.  A rounding of the running sum is at most a step, 2^-23 of it,
    # and of its size are the eight high products of a tile, a few tiles a block and ten
    # additions of the join; sums are 1.5 magnitudes over sqrt(n).  Together, as a root
    # mean square of at most (8 + 10) 2^-23 1.5 / 2 = 1.6e-6.  One operand's lowest part
    # left out shows as 3.9e-6, its middle one as 2.6e-3 (the same operands on the CPU).
    g = _gen(n)
    e, G, w = (torch.randn(s, generator=g) for s in ((K, n), (T, n), (T, K)))
    d = B.make_mix_desc(K, n)
    got = B.mix_experts_backward(d, e.to(DEV), w.to(DEV), G.to(DEV))["grad_weights"].cpu().double()
    ref = G.double() @ e.double().t()
    mag = G.double().abs() @ e.double().t().abs()
    err = ((got - ref) / mag * math.sqrt(n)).square().mean().sqrt().item()
    assert err < 18 * 2.0 ** -23 * 0.75, err
