"""The binding's workspaces of the model operators, without a GPU: the library,
the stream and the device checks are stand-ins, the tensors lie in host memory."""

import threading

import pytest
import torch

from so_edge_convolution_b200 import binding as B


class Lib:
    """Any function of the library; sizes are `need`."""

    def __init__(self, need):
        self.need = need

    def __getattr__(self, name):
        return (lambda *a: self.need) if name.endswith("workspace_size") else name


class Tracked(B.Workspace):
    gone = []

    def __del__(self):
        Tracked.gone.append(id(self))


@pytest.fixture
def host(monkeypatch):
    """Operator calls on host tensors; `calls` get each library call's arguments."""
    calls = []
    monkeypatch.setattr(B, "_on_device", lambda *a: None)
    monkeypatch.setattr(B, "_stream", lambda device: B.ctypes.c_void_p(7))
    monkeypatch.setattr(B, "_MODEL_WS", {})
    monkeypatch.setattr(B, "Workspace", Tracked)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(B, "_run", lambda dev, where, call, *args: calls.append(args) or call)

    def use(need, run=None):
        monkeypatch.setattr(B, "load", lambda: Lib(need))
        if run is not None:
            monkeypatch.setattr(B, "_run", run)
        return calls
    return use


def _mix_backward():
    d = B.make_mix_desc(3, 8, 2)
    index = torch.zeros((4, 2), dtype=torch.int32)
    return B.mix_experts_backward(d, torch.zeros(3, 8), torch.zeros(4, 2), torch.zeros(4, 8),
                                  index=index)


@pytest.mark.parametrize("need", [1024, 1 << 20])
def test_two_host_threads_on_one_stream_share_no_workspace(host, need):
    """While one thread is inside the library (the interpreter's lock is given up
    there), another one's call takes other memory and leaves the first one's alone."""
    spans, gone = {}, []

    def run(dev, where, call, *args):
        spans[threading.current_thread().name] = args[-2].value, args[-2].value + args[-1]
        if threading.current_thread().name == "second":
            return
        del Tracked.gone[:]
        other = threading.Thread(target=_mix_backward, name="second")
        other.start()
        other.join()
        gone.extend(Tracked.gone)

    host(need, run)
    _mix_backward()
    (a0, a1), (b0, b1) = spans["MainThread"], spans["second"]
    assert a1 - a0 >= need and b1 - b0 >= need
    assert a1 <= b0 or b1 <= a0, "one memory for both"
    # the first call's is not given back before its return (a thread that ends gives back its own)
    assert not gone or need <= 4096


def test_a_thread_keeps_its_small_workspace(host):
    calls = host(1024)
    _mix_backward()
    _mix_backward()
    assert calls[0][-2].value == calls[1][-2].value


def test_capture_is_looked_up_on_the_tensors_device(monkeypatch):
    # device 1's stream is being captured while device 0 is the current one
    current = [0]

    class Guard:
        def __init__(self, device):
            self.to = device.index

        def __enter__(self):
            self.was, current[0] = current[0], self.to

        def __exit__(self, *exc):
            current[0] = self.was

    class Memory(B.Workspace):
        def get(self, nbytes):
            return B.ctypes.c_void_p(256), nbytes

    monkeypatch.setattr(B, "Workspace", Memory)
    monkeypatch.setattr(B, "_MODEL_WS", {})
    monkeypatch.setattr(B, "_stream", lambda device: B.ctypes.c_void_p(7))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", Guard)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: current[0] == 1)
    ws = lambda i: B._model_ws(64, "x", torch.device("cuda", i), None)  # noqa: E731
    assert ws(1) is not ws(1)  # recorded calls never share one
    assert ws(0) is ws(0) and current == [0]


def test_check_waits_for_the_calls_stream(host, monkeypatch):
    waited, streams = [], [7]
    host(1024)
    lib = Lib(1024)
    lib.so2conv_check = lambda ws, stream: 0
    monkeypatch.setattr(B, "load", lambda: lib)
    monkeypatch.setattr(B, "_device", torch.device)
    monkeypatch.setattr(B, "_stream", lambda device: B.ctypes.c_void_p(streams[0]))
    monkeypatch.setattr(torch.cuda, "synchronize", waited.append)
    _mix_backward()
    assert B.check("cpu") == 0 and not waited  # the same stream: the library waits for it
    streams[0] = 0
    assert B.check("cpu") == 0 and waited == ["cpu"]
    own = B.Workspace("cpu")
    d = B.make_mix_desc(3, 8)
    B.mix_experts_forward(d, torch.zeros(3, 8), torch.zeros(4, 3), ws=own)
    assert B.check("cpu", ws=own) == 0 and len(waited) == 1
    streams[0] = 9
    assert B.check("cpu", ws=own) == 0 and len(waited) == 2


def test_check_looks_at_calls_that_ran(host, monkeypatch):
    def refuse(dev, where, call, *args):
        raise B.So2Error(1, where)

    host(1 << 20)
    _mix_backward()
    last = B._MODEL_WS[torch.device("cpu")]
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    _mix_backward()  # recorded: nothing has written its status
    assert B._MODEL_WS[torch.device("cpu")] is last
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    host(1 << 20, refuse)
    with pytest.raises(B.So2Error):
        _mix_backward()
    assert B._MODEL_WS[torch.device("cpu")] is last


def test_a_workspace_of_another_device_is_refused(host):
    calls = host(64)
    for device in ("meta", "cuda:1"):
        with pytest.raises(ValueError):
            B.mix_experts_forward(B.make_mix_desc(3, 8), torch.zeros(3, 8), torch.zeros(4, 3),
                                  ws=B.Workspace(device))
    assert not calls


def test_a_device_without_its_index_is_the_current_one(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(B, "_WS", {})
    assert B.workspace("cuda") is B.workspace("cuda:0")  # so check("cuda") sees the calls on it
