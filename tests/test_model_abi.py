"""The model operators' C ABI without a GPU: workspace sizes and refusals, all
before any launch (the pointers are never dereferenced)."""

import ctypes

import pytest

from so_edge_convolution_b200 import binding as B
from so_edge_convolution_b200 import build

P = ctypes.c_void_p(0x10000)
WS = ctypes.c_void_p(0x100000)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.load()


def test_workspace_sizes(lib):
    d = B.make_embed_desc(100, 128, 25)
    size = lambda n, w: lib.so2conv_embed_workspace_size(ctypes.byref(d), n, w)  # noqa: E731
    assert 0 < size(2000, 0) <= size(2000, 1) < size(1000000, 1)
    assert size(0, 1) > 0 and size(-1, 0) == 0 and size(10, 2) == 0
    bad = B.make_embed_desc(0, 128)
    assert lib.so2conv_embed_workspace_size(ctypes.byref(bad), 10, 0) == 0
    m = B.make_mix_desc(32, 1000)
    size = lambda n, w: lib.so2conv_mix_workspace_size(ctypes.byref(m), n, w)  # noqa: E731
    assert 0 < size(4, 0) <= size(4, 1)
    assert size(70000, 0) == 0 and size(4, 2) == 0
    bad = B.make_mix_desc(5000, 1000)
    assert lib.so2conv_mix_workspace_size(ctypes.byref(bad), 4, 0) == 0


def _embed(lib, d, n=4, ids=P, table=P, out=P, ld=None, ws=WS, nbytes=BIG, back=False):
    ld = d.n_comp * d.channels if ld is None else ld
    if back:
        return lib.so2conv_embed_backward(ctypes.byref(d), n, ids, out, ld, table, ws, nbytes, None)
    return lib.so2conv_embed_forward(ctypes.byref(d), n, ids, table, out, ld, ws, nbytes, None)


@pytest.mark.parametrize("back", [False, True])
def test_embed_refusals(lib, back):
    good = B.make_embed_desc(10, 16, 4)
    call = lambda d=good, **k: _embed(lib, d, back=back, **k)  # noqa: E731
    for bad in (B.make_embed_desc(0, 16), B.make_embed_desc(2**31 - 1, 16),
                B.make_embed_desc(10, 0), B.make_embed_desc(10, 65537),
                B.make_embed_desc(10, 16, 0), B.make_embed_desc(10, 16, 1025),
                B.make_embed_desc(10, 16, table_dtype=2), B.make_embed_desc(10, 16, out_dtype=-1)):
        assert call(bad) == 2
    assert call(n=-1) == 1 and call(n=(1 << 30) + 1) == 1
    assert call(ids=None) == 1 and call(table=None) == 1 and call(out=None) == 1
    assert call(ids=ctypes.c_void_p(0x10004)) == 1        # not 8-byte aligned
    assert call(out=ctypes.c_void_p(0x10001)) == 1
    assert call(table=ctypes.c_void_p(0x10002)) == 1
    assert call(ld=15) == 1                                # rows overlap
    if not back:
        assert call(ld=63) == 1
    assert call(ws=None) == 3 and call(ws=ctypes.c_void_p(0x100010)) == 3
    assert call(nbytes=8) == 3
    assert (lib.so2conv_embed_backward if back else lib.so2conv_embed_forward)(
        None, 1, P, P, *((16, P) if back else (P, 16)), WS, BIG, None) == 1


def _route(lib, d, n=4, logits=P, weights=P, index=P, bias=None, back=False, grad=P):
    if back:
        return lib.so2conv_route_backward(ctypes.byref(d), n, logits, index, weights, grad, None)
    return lib.so2conv_route_forward(ctypes.byref(d), n, logits, bias, weights, index, None, None)


@pytest.mark.parametrize("back", [False, True])
def test_route_refusals(lib, back):
    D = B.make_route_desc
    call = lambda d=D(8, 2), **k: _route(lib, d, back=back, **k)  # noqa: E731
    for bad in (D(0, 1), D(1025, 1), D(8, 0), D(8, 9), D(8, 2, n_groups=3), D(8, 2, n_groups=0),
                D(8, 2, n_groups=4, top_groups=5), D(8, 2, n_groups=4, top_groups=0),
                D(8, 2, group_top=3), D(8, 1, n_groups=8, group_top=2),
                D(8, 3, n_groups=4, top_groups=1), D(8, 2, dtype=2)):
        assert call(bad) == 2
    odd = D(8, 2)
    odd.score = 2
    assert call(odd) == 2
    odd = D(8, 2)
    odd.renormalise = 2
    assert call(odd) == 2
    for scale in (0.0, float("inf"), float("nan")):
        assert call(D(8, 2, scale=scale)) == 1
    assert call(n=-1) == 1 and call(n=(1 << 30) + 1) == 1
    assert call(logits=None) == 1 and call(weights=None) == 1 and call(index=None) == 1
    assert call(logits=ctypes.c_void_p(0x10002)) == 1
    if back:
        assert call(grad=None) == 1
    else:
        assert call(bias=ctypes.c_void_p(0x10002)) == 1
        assert lib.so2conv_route_forward(None, 1, P, None, P, P, None, None) == 1


def _mix(lib, d, n=4, experts=P, weights=P, index=P, out=P, ws=WS, nbytes=BIG, back=False):
    if back:
        return lib.so2conv_mix_experts_backward(ctypes.byref(d), n, experts, weights, index, out,
                                                P, P, ws, nbytes, None)
    return lib.so2conv_mix_experts_forward(ctypes.byref(d), n, experts, weights, index, out, ws,
                                           nbytes, None)


@pytest.mark.parametrize("back", [False, True])
def test_mix_refusals(lib, back):
    D = B.make_mix_desc
    call = lambda d=D(8, 100, 2), **k: _mix(lib, d, back=back, **k)  # noqa: E731
    for bad in (D(0, 100, 0), D(4097, 100, 2), D(8, 100, 0), D(8, 100, 9), D(8, 0, 2),
                D(8, (1 << 32) + 1, 2), D(8, 100, 2, expert_dtype=3), D(8, 100, 2, out_dtype=2)):
        assert call(bad) == 2
    assert call(n=-1) == 1 and call(n=65536) == 1
    assert call(D(4096, 100, 4096), n=2000) == 1           # too many slots
    assert call(index=None) == 1                           # only with every expert
    assert call(experts=None) == 1 and call(weights=None) == 1 and call(out=None) == 1
    assert call(experts=ctypes.c_void_p(0x10002)) == 1
    assert call(weights=ctypes.c_void_p(0x10002)) == 1
    assert call(index=ctypes.c_void_p(0x10002)) == 1
    assert call(ws=None) == 3 and call(ws=ctypes.c_void_p(0x100010)) == 3 and call(nbytes=0) == 3


def test_dropout_refusals(lib):
    D = B.make_dropout_desc

    def call(d=D(16, 4), n=4, x=P, res=None, rows=None, rng=P, out=P):
        return lib.so2conv_dropout(ctypes.byref(d), n, x, res, rows, rng, out, None)
    for bad in (D(0), D(65537), D(16, 0), D(16, 1025), D(16, dtype=2)):
        assert call(bad) == 2
    odd = D(16)
    odd.unit = 3
    assert call(odd) == 2
    for p in (-0.1, 1.1, float("nan")):
        assert call(D(16, p=p)) == 1
    assert call(n=-1) == 1 and call(n=(1 << 30) + 1) == 1
    assert call(x=None) == 1 and call(out=None) == 1 and call(rng=None) == 1
    assert call(rows=P) == 1                               # rows only name rows
    assert call(x=ctypes.c_void_p(0x10002)) == 1
    assert call(res=ctypes.c_void_p(0x10002)) == 1
    assert call(rng=ctypes.c_void_p(0x10004)) == 1
    assert call(D(16, unit="row"), rows=ctypes.c_void_p(0x10004)) == 1
    assert lib.so2conv_dropout(None, 1, P, None, None, P, P, None) == 1


def test_binding_checks_its_tensors():
    import torch
    z = torch.zeros
    d = B.make_embed_desc(10, 16, 4)
    with pytest.raises(ValueError):
        B.embed_forward(d, z(3, dtype=torch.int32), z(10, 16))   # ids are int64
    with pytest.raises(ValueError):
        B.embed_forward(d, z(3, dtype=torch.int64), z(10, 16))   # not on a CUDA device
    with pytest.raises(ValueError):
        B.route_forward(B.make_route_desc(8, 2), z(4, 7))
    with pytest.raises(ValueError):
        B.dropout(B.make_dropout_desc(16, 4), z(3, 4, 15), z(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        B.mix_experts_forward(B.make_mix_desc(4, 10, 2), z(4, 9), z(3, 2))


def test_calls_run_on_their_tensors_device(monkeypatch):
    import torch
    entered = []

    class Guard:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            entered.append(self.device)

        def __exit__(self, *exc):
            entered.append(None)

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", Guard)
    monkeypatch.setattr(B, "_stream", lambda device: ("stream", device.index))
    calls = []
    for index in (0, 1):
        B._run(torch.device("cuda", index), "x", lambda *a: calls.append((a, list(entered))) or 0, 7)
    assert calls[0] == ((7, ("stream", 0)), [])
    assert calls[1] == ((7, ("stream", 1)), [torch.device("cuda", 1)]) and entered[-1] is None
    with pytest.raises(B.So2Error):
        B._run(torch.device("cuda", 0), "x", lambda *a: 5)
