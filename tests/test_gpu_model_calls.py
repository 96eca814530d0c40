"""Calls of the model operators from several host threads."""

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
