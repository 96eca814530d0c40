"""Calls of the model operators from several host threads, and their status."""

import threading

import pytest
import torch

from so_edge_convolution_b200 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from so_edge_convolution_b200 import build
    build.build()
    B.load()
    torch.cuda.init()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _in_threads(works):
    """Each of `works` in a host thread of its own, at the same time."""
    start, errors = threading.Barrier(len(works)), []

    def body(work):
        try:
            start.wait(30)
            work()
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=body, args=(w,)) for w in works]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


@pytest.mark.parametrize("n,tokens", [(1024, 5000), (70000, 40000)])
def test_host_threads_on_one_stream(n, tokens):
    # several kernels a call: lists, gradients and joins by index, sort and sums by id
    cases = []
    for seed in range(3):
        g = _gen(seed)
        cases.append(dict(
            md=B.make_mix_desc(16, n, 2), e=torch.randn((16, n), generator=g).to(DEV),
            w=torch.randn((8, 2), generator=g).to(DEV), G=torch.randn((8, n), generator=g).to(DEV),
            i=torch.randint(0, 16, (8, 2), generator=g).to(torch.int32).to(DEV),
            ed=B.make_embed_desc(300, 24), ids=torch.randint(0, 300, (tokens,), generator=g).to(DEV),
            ge=torch.randn((tokens, 24), generator=g).to(DEV)))

    def both(c):
        r = list(B.mix_experts_backward(c["md"], c["e"], c["w"], c["G"], index=c["i"]).values())
        return r + [B.embed_backward(c["ed"], c["ids"], c["ge"])]
    want = [both(c) for c in cases]
    torch.cuda.synchronize()
    wrong = []

    def work(k):
        def run():
            got = [both(cases[k]) for _ in range(60)]
            torch.cuda.current_stream().synchronize()
            wrong.extend(k for r in got for a, b in zip(r, want[k]) if not torch.equal(a, b))
        return run
    _in_threads([work(k) for k in range(3)])
    assert not wrong


def test_status_of_a_call_on_another_stream():
    side = torch.cuda.Stream()
    d = B.make_embed_desc(9, 12)
    ids = torch.tensor([1, 9, 2], device=DEV)  # 9 is no row
    t, a = torch.ones((9, 12), device=DEV), torch.ones((4096, 4096), device=DEV)
    own = B.Workspace(DEV)
    for ws in (None, own):
        B.embed_forward(d, ids[:1], t, ws=ws)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(50):  # some milliseconds before the call's kernel
                a @ a
            B.embed_forward(d, ids, t, ws=ws)
        assert B.check(DEV, ws=ws) == 5
    # a refused call leaves the last one's status alone, a recorded one too
    B.embed_forward(d, ids, t)
    with pytest.raises(B.So2Error):
        B.embed_forward(d, ids[1:], t, out=torch.zeros((1, 1, 12), device=DEV).expand(2, 1, 12))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.embed_forward(d, ids, t)
        B.embed_forward(d, ids, t, ws=own)
    assert B.check(DEV) == 5 and B.check(DEV) == 0
    with torch.cuda.stream(side):
        graph.replay()
    assert B.check(DEV, ws=own) == 5


def test_host_threads_with_kernels_of_different_sizes():
    # calls that run the same kernels with more and with less shared memory
    g = _gen(5)
    x = torch.randn((16, 1024), generator=g).to(DEV)
    bias = torch.randn(1024, generator=g).to(DEV)
    m = torch.randn((256, 64), generator=g).to(DEV)
    works = []
    for K, S in ((1024, 256), (1000, 128)):
        d, md = B.make_route_desc(K, 12), B.make_mix_desc(S, 64)
        xs, bs = x[:, :K].contiguous(), bias[:K].contiguous()
        e, w = m[:S].contiguous(), torch.randn((32, S), generator=g).to(DEV)

        def run(d=d, md=md, xs=xs, bs=bs, e=e, w=w):
            for _ in range(1500):
                B.route_forward(d, xs, bs)
                B.mix_experts_forward(md, e, w)
            torch.cuda.current_stream().synchronize()
        works.append(run)
    _in_threads(works)
