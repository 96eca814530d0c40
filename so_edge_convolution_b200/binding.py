"""Thin ctypes binding of libso2conv (include/so2conv.h, so2model.h) for torch tensors.

Argument marshalling only: every step of the convolution runs in the
library's CUDA kernels.  Torch supplies device memory (inputs, outputs and
the workspace) and the current stream.  If the shared library is missing or
does not load, every call raises -- there is no fallback path.
"""

import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libso2conv.so")

SO2_F32, SO2_BF16 = 0, 1
WS_FORWARD, WS_BACKWARD, WS_DOUBLE_BACKWARD = 0, 1, 2
STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported", 3: "workspace",
          4: "cuda", 5: "index", 6: "timeout", 7: "degenerate edge"}


class Desc(ctypes.Structure):
    _fields_ = [("lmax", ctypes.c_int32), ("mmax", ctypes.c_int32),
                ("c_in", ctypes.c_int32), ("c_out", ctypes.c_int32),
                ("n_rbf", ctypes.c_int32), ("rbf_cutoff", ctypes.c_float),
                ("dtype", ctypes.c_int32)]


class Params(ctypes.Structure):
    _fields_ = [("w", ctypes.c_void_p), ("w_rad", ctypes.c_void_p),
                ("b_rad", ctypes.c_void_p)]


class EmbedDesc(ctypes.Structure):
    _fields_ = [("n_rows", ctypes.c_int64), ("channels", ctypes.c_int32),
                ("n_comp", ctypes.c_int32), ("scale", ctypes.c_float),
                ("table_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("pad_id", ctypes.c_int64)]


class RouteDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("n_experts", "top_k", "n_groups", "top_groups", "group_top", "score",
                 "renormalise")] + [("scale", ctypes.c_float), ("dtype", ctypes.c_int32)]


class MixDesc(ctypes.Structure):
    _fields_ = [("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("n_weights", ctypes.c_int64), ("expert_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32)]


class DropoutDesc(ctypes.Structure):
    _fields_ = [("channels", ctypes.c_int32), ("n_comp", ctypes.c_int32),
                ("unit", ctypes.c_int32), ("p", ctypes.c_float), ("dtype", ctypes.c_int32)]


class So2Error(RuntimeError):
    def __init__(self, code, where):
        super().__init__(f"{where}: {STATUS.get(code, code)} (status {code})")
        self.code = code


_lib = None


def load():
    """Load libso2conv.so (raises if it is missing: there is no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing; build it with "
            "`python -m so_edge_convolution_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i64, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
    pd = ctypes.POINTER(Desc)
    lib.so2conv_workspace_size.argtypes = [pd, i64, i64, ctypes.c_int]
    lib.so2conv_workspace_size.restype = sz
    lib.so2conv_num_weights.argtypes = [pd]
    lib.so2conv_num_weights.restype = i64
    lib.so2conv_forward.argtypes = [pd, i64, i64, vp, vp, vp, Params, vp, vp, sz, vp]
    lib.so2conv_forward.restype = ctypes.c_int
    lib.so2conv_backward.argtypes = [pd, i64, i64, vp, vp, vp, Params, vp, vp, vp, vp,
                                     vp, vp, vp, sz, vp]
    lib.so2conv_backward.restype = ctypes.c_int
    lib.so2conv_double_backward.argtypes = [pd, i64, i64, vp, vp, vp, Params, vp, vp, vp,
                                            vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.so2conv_double_backward.restype = ctypes.c_int
    lib.so2conv_check.argtypes = [vp, vp]
    lib.so2conv_check.restype = ctypes.c_int
    lib.so2conv_status_string.argtypes = [ctypes.c_int]
    lib.so2conv_status_string.restype = ctypes.c_char_p
    lib.so2conv_edge_frames.argtypes = [ctypes.c_int32, i64, vp, vp, vp, vp]
    lib.so2conv_edge_frames.restype = ctypes.c_int
    lib.so2conv_forward_noalloc.argtypes = [pd, i64, i64, vp, vp, vp, Params, vp, vp]
    lib.so2conv_forward_noalloc.restype = ctypes.c_int
    lib.so2conv_block_workspace_size.argtypes = [pd, i64, i64, ctypes.c_int]
    lib.so2conv_block_workspace_size.restype = sz
    lib.so2conv_block_forward.argtypes = [pd, i64, i64, vp, vp, vp, Params, Params, vp, vp, sz, vp]
    lib.so2conv_block_forward.restype = ctypes.c_int
    lib.so2conv_block_backward.argtypes = [pd, i64, i64, vp, vp, vp, Params, Params, vp,
                                           vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.so2conv_block_backward.restype = ctypes.c_int
    lib.so2conv_noalloc_check.argtypes = [vp]
    lib.so2conv_noalloc_check.restype = ctypes.c_int
    lib.so2conv_launch_count.argtypes = []
    lib.so2conv_launch_count.restype = ctypes.c_longlong
    lib.so2conv_wait_selftest.argtypes = [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64,
                                          ctypes.c_void_p]
    lib.so2conv_wait_selftest.restype = ctypes.c_int
    lib.so2conv_set_max_chunk_edges.argtypes = [ctypes.c_int64]
    lib.so2conv_set_max_chunk_edges.restype = ctypes.c_int
    lib.so2conv_max_chunk_edges.argtypes = []
    lib.so2conv_max_chunk_edges.restype = ctypes.c_int64
    lib.so2conv_profile_enable.argtypes = [ctypes.c_int]
    lib.so2conv_profile_enable.restype = None
    lib.so2conv_profile_read.argtypes = [ctypes.c_int, ctypes.POINTER(ctypes.c_int),
                                         ctypes.POINTER(ctypes.c_double)]
    lib.so2conv_profile_read.restype = ctypes.c_int
    pe, pr, pm, pp = (ctypes.POINTER(c) for c in (EmbedDesc, RouteDesc, MixDesc, DropoutDesc))
    lib.so2conv_embed_workspace_size.argtypes = [pe, i64, ctypes.c_int]
    lib.so2conv_embed_workspace_size.restype = sz
    lib.so2conv_embed_forward.argtypes = [pe, i64, vp, vp, vp, i64, vp, sz, vp]
    lib.so2conv_embed_forward.restype = ctypes.c_int
    lib.so2conv_embed_backward.argtypes = [pe, i64, vp, vp, i64, vp, vp, sz, vp]
    lib.so2conv_embed_backward.restype = ctypes.c_int
    lib.so2conv_route_forward.argtypes = [pr, i64, vp, vp, vp, vp, vp, vp]
    lib.so2conv_route_forward.restype = ctypes.c_int
    lib.so2conv_route_backward.argtypes = [pr, i64, vp, vp, vp, vp, vp]
    lib.so2conv_route_backward.restype = ctypes.c_int
    lib.so2conv_mix_workspace_size.argtypes = [pm, i64, ctypes.c_int]
    lib.so2conv_mix_workspace_size.restype = sz
    lib.so2conv_mix_experts_forward.argtypes = [pm, i64, vp, vp, vp, vp, vp, sz, vp]
    lib.so2conv_mix_experts_forward.restype = ctypes.c_int
    lib.so2conv_mix_experts_backward.argtypes = [pm, i64, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.so2conv_mix_experts_backward.restype = ctypes.c_int
    lib.so2conv_dropout.argtypes = [pp, i64, vp, vp, vp, vp, vp, vp]
    lib.so2conv_dropout.restype = ctypes.c_int
    _lib = lib
    return lib


def make_desc(lmax, mmax, c_in, c_out, n_rbf, rbf_cutoff, dtype=SO2_F32):
    return Desc(lmax, mmax, c_in, c_out, n_rbf, float(rbf_cutoff), dtype)


def _ptr(t):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("so2conv tensors must be contiguous (row-major)")
    return ctypes.c_void_p(t.data_ptr())


def _c(t):
    return None if t is None else t.contiguous()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # without a Stream object


def _stream(device):
    if _raw_stream is not None and isinstance(device, torch.device) and device.index is not None:
        return ctypes.c_void_p(_raw_stream(device.index))
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _check_call(code, where):
    if code != 0:
        raise So2Error(code, where)


_RECORDED = -1  # in place of a stream: a call recorded into a graph, which any stream may replay


class Workspace:
    """A reusable device workspace (grown on demand, 256-byte aligned)."""

    def __init__(self, device):
        self.device = torch.device(device)
        self.buf = None
        self.stream = None  # of the last model operator in it, or _RECORDED

    def get(self, nbytes):
        if self.buf is None or self.buf.numel() < nbytes + 256:
            self.buf = torch.empty(nbytes + 256, dtype=torch.uint8,
                                   device=self.device)
        base = self.buf.data_ptr()
        off = (-base) % 256
        return ctypes.c_void_p(base + off), nbytes


_WS = {}
_MODEL_WS = {}  # device -> workspace of the last model operator there, if it came after the others


def workspace(device):
    key = _device(device)
    if key not in _WS:
        _WS[key] = Workspace(key)
    return _WS[key]


def num_weights(desc):
    return int(load().so2conv_num_weights(ctypes.byref(desc)))


def workspace_size(desc, n_nodes, n_edges, which):
    return int(load().so2conv_workspace_size(ctypes.byref(desc), n_nodes, n_edges, which))


def _wsarg(desc, n_nodes, n_edges, which, device, ws):
    need = workspace_size(desc, n_nodes, n_edges, which)
    if need == 0:
        raise So2Error(2, "workspace_size")
    return _default_ws(device, ws).get(need)


def _default_ws(device, ws):
    if ws:
        return ws
    _MODEL_WS.pop(_device(device), None)
    return workspace(device)


def _device(device):
    """The device with its index, so that "cuda" and "cuda:0" are one key."""
    d = torch.device(device)
    if d.type == "cuda" and d.index is None:
        return torch.device("cuda", torch.cuda.current_device())
    return d


def forward(desc, x, edge_index, edge_vec, w, w_rad, b_rad, out=None, ws=None):
    lib = load()
    x, edge_index, edge_vec, w, w_rad, b_rad = map(_c, (x, edge_index, edge_vec, w, w_rad, b_rad))
    N, E = x.shape[0], edge_index.shape[1]
    if out is None:
        out = torch.empty((N, (desc.lmax + 1) ** 2, desc.c_out), dtype=torch.float32,
                          device=x.device)
    p, nb = _wsarg(desc, N, E, WS_FORWARD, x.device, ws)
    code = lib.so2conv_forward(ctypes.byref(desc), N, E, _ptr(x), _ptr(edge_index),
                               _ptr(edge_vec), Params(_ptr(w).value, _ptr(w_rad).value, _ptr(b_rad).value),
                               _ptr(out), p, nb, _stream(x.device))
    _check_call(code, "so2conv_forward")
    return out


def _outputs(names, need, shapes, out, f32):
    """The output tensors: caller-given ones (checked) or new ones."""
    res = {}
    for n in names:
        if n not in need:
            res[n] = None
        elif out is not None and out.get(n) is not None:
            t = out[n]
            if (tuple(t.shape) != tuple(shapes[n]) or t.dtype != torch.float32
                    or t.device != f32["device"] or not t.is_contiguous()):
                raise ValueError(f"out[{n!r}] must be a contiguous float32 tensor of shape "
                                 f"{tuple(shapes[n])} on {f32['device']}")
            res[n] = t
        else:
            res[n] = torch.empty(shapes[n], **f32)
    return res


def backward(desc, x, edge_index, edge_vec, w, w_rad, b_rad, grad_out, need=None,
             ws=None, out=None):
    """Returns a dict of gradients; `need` limits which ones are computed and
    `out` (a dict) may give preallocated tensors for some of them."""
    lib = load()
    x, edge_index, edge_vec, w, w_rad, b_rad, grad_out = map(
        _c, (x, edge_index, edge_vec, w, w_rad, b_rad, grad_out))
    N, E = x.shape[0], edge_index.shape[1]
    names = ["grad_x", "grad_w", "grad_w_rad", "grad_b_rad", "grad_edge_vec"]
    need = set(names if need is None else need)
    dev = x.device
    f32 = dict(dtype=torch.float32, device=dev)
    S = (desc.lmax + 1) ** 2
    shapes = {"grad_x": (N, S, desc.c_in), "grad_w": (num_weights(desc),),
              "grad_w_rad": (desc.n_rbf, desc.c_out), "grad_b_rad": (desc.c_out,),
              "grad_edge_vec": (E, 3)}
    outs = _outputs(names, need, shapes, out, f32)
    p, nb = _wsarg(desc, N, E, WS_BACKWARD, dev, ws)
    code = lib.so2conv_backward(ctypes.byref(desc), N, E, _ptr(x), _ptr(edge_index),
                                _ptr(edge_vec), Params(w.data_ptr(), w_rad.data_ptr(),
                                                       b_rad.data_ptr()),
                                _ptr(grad_out), *[_ptr(outs[n]) for n in names], p, nb,
                                _stream(dev))
    _check_call(code, "so2conv_backward")
    return {n: t for n, t in outs.items() if t is not None}


def double_backward(desc, x, edge_index, edge_vec, w, w_rad, b_rad, grad_out, gg_x=None,
                    gg_edge_vec=None, need=None, ws=None, out=None):
    lib = load()
    x, edge_index, edge_vec, w, w_rad, b_rad, grad_out, gg_x, gg_edge_vec = map(
        _c, (x, edge_index, edge_vec, w, w_rad, b_rad, grad_out, gg_x, gg_edge_vec))
    N, E = x.shape[0], edge_index.shape[1]
    names = ["d_x", "d_w", "d_w_rad", "d_b_rad", "d_grad_out", "d_edge_vec"]
    need = set(names if need is None else need)
    dev = x.device
    f32 = dict(dtype=torch.float32, device=dev)
    S = (desc.lmax + 1) ** 2
    shapes = {"d_x": (N, S, desc.c_in), "d_w": (num_weights(desc),),
              "d_w_rad": (desc.n_rbf, desc.c_out), "d_b_rad": (desc.c_out,),
              "d_grad_out": (N, S, desc.c_out), "d_edge_vec": (E, 3)}
    outs = _outputs(names, need, shapes, out, f32)
    p, nb = _wsarg(desc, N, E, WS_DOUBLE_BACKWARD, dev, ws)
    code = lib.so2conv_double_backward(
        ctypes.byref(desc), N, E, _ptr(x), _ptr(edge_index), _ptr(edge_vec),
        Params(w.data_ptr(), w_rad.data_ptr(), b_rad.data_ptr()), _ptr(grad_out),
        _ptr(gg_x), _ptr(gg_edge_vec), *[_ptr(outs[n]) for n in names], p, nb,
        _stream(dev))
    _check_call(code, "so2conv_double_backward")
    return {n: t for n, t in outs.items() if t is not None}


def check(device, ws=None):
    """Synchronise and return the device status of the last call (0 = ok): the
    last one made with `ws`, or without a workspace of its own on `device`, on
    whatever stream.  Calls that were refused, and calls recorded into a graph
    without a workspace of their own, are not looked at.  (The workspace of
    the last call stays allocated for this until the next call.)"""
    w = ws or _MODEL_WS.get(_device(device)) or workspace(device)
    if w.buf is None:
        return 0
    if w.stream is not None and w.stream != (_stream(device).value or 0):
        torch.cuda.synchronize(device)
    base = w.buf.data_ptr()
    return int(load().so2conv_check(ctypes.c_void_p(base + (-base) % 256),
                                    _stream(device)))


def edge_frames(lmax, edge_vec):
    """Frames R [E, 3, 3] and full Wigner-D blocks [E, Dsz] as the library
    computes them."""
    E = edge_vec.shape[0]
    dsz = sum((2 * l + 1) ** 2 for l in range(lmax + 1))
    R = torch.empty((E, 9), dtype=torch.float32, device=edge_vec.device)
    D = torch.empty((E, dsz), dtype=torch.float32, device=edge_vec.device)
    code = load().so2conv_edge_frames(lmax, E, _ptr(edge_vec), _ptr(R), _ptr(D),
                                      _stream(edge_vec.device))
    _check_call(code, "so2conv_edge_frames")
    return R.view(E, 3, 3), D


def wait_selftest(device, limit_us=1000):
    """so2conv_wait_selftest, then so2conv_check: returns the recorded status
    (SO2_ERR_TIMEOUT = 6 when the bounded wait gave up as it should)."""
    lib = load()
    w = workspace(device)
    p, nb = w.get(256)
    _check_call(lib.so2conv_wait_selftest(p, nb, int(limit_us), _stream(device)),
                "so2conv_wait_selftest")
    return int(lib.so2conv_check(p, _stream(device)))


def set_max_chunk_edges(n):
    """so2conv_set_max_chunk_edges: edges per chunk of per-edge intermediates
    (0 restores the default); returns the value now in force."""
    lib = load()
    _check_call(lib.so2conv_set_max_chunk_edges(int(n)), "so2conv_set_max_chunk_edges")
    return int(lib.so2conv_max_chunk_edges())


def launch_count():
    """Kernels launched by the library so far in this process."""
    return int(load().so2conv_launch_count())


def profile_enable(on=True, all_kinds=False):
    """Record CUDA events around the tensor-core launches (and, with
    all_kinds, around every group of CUDA-core launches too)."""
    load().so2conv_profile_enable((2 if all_kinds else 1) if on else 0)


PROFILE_KINDS = {0: "mixing (x W^T)", 1: "mixing transposed (g W)", 2: "weight gradient",
                 3: "rotation on gather", 4: "edge preparation", 5: "edge gradient terms",
                 6: "radial sums", 7: "weight packing and node scatter"}
TENSOR_KINDS = (0, 1, 2)


def profile_read():
    """{kind: (ranges, total_ms)} of the recorded launches (kinds 0-2: one
    range per tcgen05 launch; 3-7: groups of CUDA-core launches)."""
    lib = load()
    res = {}
    for k in PROFILE_KINDS:
        n, ms = ctypes.c_int(0), ctypes.c_double(0.0)
        _check_call(lib.so2conv_profile_read(k, ctypes.byref(n), ctypes.byref(ms)),
                    "so2conv_profile_read")
        res[k] = (n.value, ms.value)
    return res


def forward_noalloc(desc, x, edge_index, edge_vec, w, w_rad, b_rad, out=None):
    """so2conv_forward_noalloc: the forward on the library's own scratch array
    (no workspace argument, nothing allocated by the library)."""
    lib = load()
    x, edge_index, edge_vec, w, w_rad, b_rad = map(_c, (x, edge_index, edge_vec, w, w_rad, b_rad))
    N, E = x.shape[0], edge_index.shape[1]
    if out is None:
        out = torch.empty((N, (desc.lmax + 1) ** 2, desc.c_out), dtype=torch.float32,
                          device=x.device)
    code = lib.so2conv_forward_noalloc(ctypes.byref(desc), N, E, _ptr(x), _ptr(edge_index),
                                       _ptr(edge_vec), Params(_ptr(w).value, _ptr(w_rad).value,
                                                              _ptr(b_rad).value),
                                       _ptr(out), _stream(x.device))
    _check_call(code, "so2conv_forward_noalloc")
    return out


def noalloc_check(device):
    """Synchronise and return the device status of the last no-alloc forward
    in the current context (0 = ok)."""
    return int(load().so2conv_noalloc_check(_stream(device)))


# ---------------------------------------------------------------------------
# Message block: two convolutions with the edge-frame activation between them
# ---------------------------------------------------------------------------
BLOCK_GRADS = ["grad_x", "grad_w1", "grad_w_rad1", "grad_b_rad1", "grad_w2", "grad_w_rad2",
               "grad_b_rad2", "grad_edge_vec"]


def block_workspace_size(desc, n_nodes, n_edges, which):
    return int(load().so2conv_block_workspace_size(ctypes.byref(desc), n_nodes, n_edges, which))


def _block_ws(desc, n_nodes, n_edges, which, device, ws):
    need = block_workspace_size(desc, n_nodes, n_edges, which)
    if need == 0:
        raise So2Error(2, "block_workspace_size")
    return _default_ws(device, ws).get(need)


def _params(w, w_rad, b_rad):
    return Params(_ptr(w).value, _ptr(w_rad).value, _ptr(b_rad).value)


def block_forward(desc, x, edge_index, edge_vec, w1, w_rad1, b_rad1, w2, w_rad2, b_rad2,
                  out=None, ws=None):
    """so2conv_block_forward: out [N, S, C] of the two-convolution block."""
    lib = load()
    x, edge_index, edge_vec, w1, w_rad1, b_rad1, w2, w_rad2, b_rad2 = map(
        _c, (x, edge_index, edge_vec, w1, w_rad1, b_rad1, w2, w_rad2, b_rad2))
    N, E = x.shape[0], edge_index.shape[1]
    if out is None:
        out = torch.empty((N, (desc.lmax + 1) ** 2, desc.c_out), dtype=torch.float32,
                          device=x.device)
    p, nb = _block_ws(desc, N, E, 0, x.device, ws)
    code = lib.so2conv_block_forward(ctypes.byref(desc), N, E, _ptr(x), _ptr(edge_index),
                                     _ptr(edge_vec), _params(w1, w_rad1, b_rad1),
                                     _params(w2, w_rad2, b_rad2), _ptr(out), p, nb,
                                     _stream(x.device))
    _check_call(code, "so2conv_block_forward")
    return out


def block_backward(desc, x, edge_index, edge_vec, w1, w_rad1, b_rad1, w2, w_rad2, b_rad2,
                   grad_out, need=None, ws=None, out=None):
    """so2conv_block_backward: a dict keyed by BLOCK_GRADS (those in `need`)."""
    lib = load()
    x, edge_index, edge_vec, w1, w_rad1, b_rad1, w2, w_rad2, b_rad2, grad_out = map(
        _c, (x, edge_index, edge_vec, w1, w_rad1, b_rad1, w2, w_rad2, b_rad2, grad_out))
    N, E = x.shape[0], edge_index.shape[1]
    need = set(BLOCK_GRADS if need is None else need)
    dev = x.device
    f32 = dict(dtype=torch.float32, device=dev)
    S = (desc.lmax + 1) ** 2
    nw = num_weights(desc)
    shapes = {"grad_x": (N, S, desc.c_in), "grad_w1": (nw,), "grad_w2": (nw,),
              "grad_w_rad1": (desc.n_rbf, desc.c_out), "grad_w_rad2": (desc.n_rbf, desc.c_out),
              "grad_b_rad1": (desc.c_out,), "grad_b_rad2": (desc.c_out,),
              "grad_edge_vec": (E, 3)}
    outs = _outputs(BLOCK_GRADS, need, shapes, out, f32)
    p, nb = _block_ws(desc, N, E, 1, dev, ws)
    code = lib.so2conv_block_backward(ctypes.byref(desc), N, E, _ptr(x), _ptr(edge_index),
                                      _ptr(edge_vec), _params(w1, w_rad1, b_rad1),
                                      _params(w2, w_rad2, b_rad2), _ptr(grad_out),
                                      *[_ptr(outs[n]) for n in BLOCK_GRADS], p, nb, _stream(dev))
    _check_call(code, "so2conv_block_backward")
    return {n: t for n, t in outs.items() if t is not None}


# ---------------------------------------------------------------------------
# Model operators beside the convolution (include/so2model.h)
# ---------------------------------------------------------------------------
NO_PAD = -(1 << 63)
SCORES = {"softmax": 0, "sigmoid": 1}
DROP_UNITS = {"element": 0, "channel": 1, "row": 2}
_TORCH_DTYPE = {SO2_F32: torch.float32, SO2_BF16: torch.bfloat16}


def _torch_dtype(code):
    if code not in _TORCH_DTYPE:
        raise So2Error(2, "dtype")
    return _TORCH_DTYPE[code]


class _Local(threading.local):
    def __init__(self):  # in each host thread
        self.small = {}  # (device index, stream) -> workspace


_LOCAL = _Local()
_SMALL_WS_BYTES = 4096


def _capturing(device):
    """Whether a graph is being captured on the current stream of `device`."""
    if torch.cuda.current_device() == device.index:
        return torch.cuda.is_current_stream_capturing()
    with torch.cuda.device(device):
        return torch.cuda.is_current_stream_capturing()


def _model_ws(need, where, device, ws):
    """The workspace of one model operator call, which holds it until the
    library has enqueued its kernels: the caller's; or, small, one that this
    host thread keeps for the current stream; or a new one from torch's
    allocator, which belongs to the stream, or to the graph being captured.
    (The interpreter's lock is given up inside the library, so calls of two
    threads may enqueue their kernels in turn, on one stream too.)"""
    if need == 0:
        raise So2Error(2, where)
    stream = _RECORDED if _capturing(device) else _stream(device).value or 0
    if ws:
        if _device(ws.device) != device:
            raise ValueError(f"ws must be on {device}, not {ws.device}")
        w = ws
    elif need <= _SMALL_WS_BYTES and stream != _RECORDED:
        key, small = (device.index, stream), _LOCAL.small
        w = small.get(key)
        if w is None:
            w = small[key] = Workspace(device)
            w.get(_SMALL_WS_BYTES)
    else:
        w = Workspace(device)
    w.stream = stream
    return w


def _run(dev, where, call, *args):
    """One library call on the current stream of the tensors' device, which is
    made current for it if another one is."""
    if torch.cuda.current_device() == dev.index:
        code = call(*args, _stream(dev))
    else:
        with torch.cuda.device(dev):
            code = call(*args, _stream(dev))
    _check_call(code, where)


def _run_ws(dev, where, need, ws, call, *args):
    """_run with a workspace of `need` bytes (0: none fits) as the last
    arguments, whose status check() then reads."""
    w = _model_ws(need, where, dev, ws)
    _run(dev, where, call, *args, *w.get(need))
    if not ws and w.stream != _RECORDED:
        _MODEL_WS[dev] = w


def _need(t, name, shape, dtype, device=None):
    """`t`, contiguous, after a check of its shape, dtype and device."""
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)}, not {t.dtype} of "
                         f"shape {tuple(t.shape)}")
    _on_device(t, name, device)
    return t if t.is_contiguous() else t.contiguous()


def _adr(t):
    """A checked tensor's address, for a pointer argument."""
    return None if t is None else t.data_ptr()


def _on_device(t, name, device):
    if not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{name} must be on {device or 'a CUDA device'}, not {t.device}")


def _given_out(out, name, shape, dtype, like):
    """A caller's output (checked: written in place) or a new one beside `like`."""
    if out is None:
        return like.new_empty(shape, dtype=dtype)
    if (out.shape != shape or out.dtype != dtype or out.device != like.device
            or not out.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} "
                         f"on {like.device}")
    return out


def make_embed_desc(n_rows, channels, n_comp=1, scale=1.0, table_dtype=SO2_F32,
                    out_dtype=SO2_F32, pad_id=None):
    return EmbedDesc(n_rows, channels, n_comp, float(scale), table_dtype, out_dtype,
                     NO_PAD if pad_id is None else pad_id)


def _rows_of(t, n, inner, name):
    """Row stride of [n, ...] whose rows are contiguous (`inner` elements)."""
    want = 1
    for size, stride in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if size > 1 and stride != want:
            raise ValueError(f"the rows of {name} must be contiguous")
        want *= size
    return inner if n <= 1 else t.stride(0)


def embed_forward(desc, ids, table, out=None, ws=None):
    """so2conv_embed_forward: out [n, n_comp, channels], element rows in
    component 0.  A given `out` may have any row stride."""
    lib = load()
    n = ids.shape[0]
    ids = _need(ids, "ids", (n,), torch.int64)
    dev = ids.device
    table = _need(table, "table", (desc.n_rows, desc.channels), _torch_dtype(desc.table_dtype),
                  dev)
    shape, dt = (n, desc.n_comp, desc.channels), _torch_dtype(desc.out_dtype)
    if out is None:
        out = ids.new_empty(shape, dtype=dt)
    elif out.shape != shape or out.dtype != dt or out.device != dev:
        raise ValueError(f"out must be {dt} of shape {shape} on {dev}")
    ld = _rows_of(out, n, desc.n_comp * desc.channels, "out")
    need = lib.so2conv_embed_workspace_size(ctypes.byref(desc), n, WS_FORWARD)
    _run_ws(dev, "so2conv_embed_forward", need, ws, lib.so2conv_embed_forward, ctypes.byref(desc), n,
            _adr(ids), _adr(table), out.data_ptr(), ld)
    return out


def embed_backward(desc, ids, grad_out, out=None, ws=None):
    """so2conv_embed_backward: grad_table [n_rows, channels] f32.  grad_out is
    [n, n_comp, channels] (or [n, channels]: its component 0), any row stride."""
    lib = load()
    n = ids.shape[0]
    ids = _need(ids, "ids", (n,), torch.int64)
    dev = ids.device
    dt = _torch_dtype(desc.out_dtype)
    shapes = ((n, desc.n_comp, desc.channels), (n, desc.channels))
    if tuple(grad_out.shape) not in shapes or grad_out.dtype != dt:
        raise ValueError(f"grad_out must be {dt} of shape {shapes[0]} or {shapes[1]}")
    _on_device(grad_out, "grad_out", dev)
    if grad_out.dim() == 3:
        grad_out = grad_out[:, 0, :]
    if desc.channels > 1 and grad_out.stride(1) != 1:
        grad_out = grad_out.contiguous()
    if n > 1 and grad_out.stride(0) < desc.channels:  # rows that overlap (an expanded tensor)
        grad_out = grad_out.contiguous()
    ld = desc.channels if n <= 1 else grad_out.stride(0)
    out = _given_out(out, "out", (desc.n_rows, desc.channels), torch.float32, ids)
    need = lib.so2conv_embed_workspace_size(ctypes.byref(desc), n, WS_BACKWARD)
    _run_ws(dev, "so2conv_embed_backward", need, ws, lib.so2conv_embed_backward, ctypes.byref(desc),
            n, _adr(ids), grad_out.data_ptr(), ld, _adr(out))
    return out


def make_route_desc(n_experts, top_k, score="softmax", n_groups=1, top_groups=1, group_top=1,
                    renormalise=False, scale=1.0, dtype=SO2_F32):
    return RouteDesc(n_experts, top_k, n_groups, top_groups, group_top, SCORES[score],
                     int(bool(renormalise)), float(scale), dtype)


def route_forward(desc, logits, bias=None):
    """so2conv_route_forward: (weights f32, index int32) [n, top_k] and counts
    int32 [n_experts]."""
    lib = load()
    n, dt = logits.shape[0], _torch_dtype(desc.dtype)
    logits = _need(logits, "logits", (n, desc.n_experts), dt)
    dev = logits.device
    if bias is not None:
        bias = _need(bias, "bias", (desc.n_experts,), torch.float32, dev)
    weights = logits.new_empty((n, desc.top_k), dtype=torch.float32)
    index = torch.empty_like(weights, dtype=torch.int32)
    counts = index.new_empty(desc.n_experts)
    _run(dev, "so2conv_route_forward", lib.so2conv_route_forward, ctypes.byref(desc), n,
         _adr(logits), _adr(bias), _adr(weights), _adr(index), _adr(counts))
    return weights, index, counts


def route_backward(desc, logits, index, grad_weights, out=None):
    """so2conv_route_backward: grad_logits [n, n_experts] f32."""
    lib = load()
    n, dt = logits.shape[0], _torch_dtype(desc.dtype)
    logits = _need(logits, "logits", (n, desc.n_experts), dt)
    dev = logits.device
    index = _need(index, "index", (n, desc.top_k), torch.int32, dev)
    grad_weights = _need(grad_weights, "grad_weights", (n, desc.top_k), torch.float32, dev)
    out = _given_out(out, "out", (n, desc.n_experts), torch.float32, logits)
    _run(dev, "so2conv_route_backward", lib.so2conv_route_backward, ctypes.byref(desc), n,
         _adr(logits), _adr(index), _adr(grad_weights), _adr(out))
    return out


def make_mix_desc(n_experts, n_weights, top_k=None, expert_dtype=SO2_F32, out_dtype=SO2_F32):
    return MixDesc(n_experts, n_experts if top_k is None else top_k, n_weights, expert_dtype,
                   out_dtype)


def _mix_inputs(desc, experts, weights, index):
    n = weights.shape[0]
    experts = _need(experts, "experts", (desc.n_experts, desc.n_weights),
                    _torch_dtype(desc.expert_dtype))
    dev = experts.device
    weights = _need(weights, "weights", (n, desc.top_k), torch.float32, dev)
    if index is not None:
        index = _need(index, "index", (n, desc.top_k), torch.int32, dev)
    return n, dev, experts, weights, index


def mix_experts_forward(desc, experts, weights, index=None, out=None, ws=None):
    """so2conv_mix_experts_forward: out [n_systems, n_weights] of out_dtype."""
    lib = load()
    n, dev, experts, weights, index = _mix_inputs(desc, experts, weights, index)
    out = _given_out(out, "out", (n, desc.n_weights), _torch_dtype(desc.out_dtype), experts)
    need = lib.so2conv_mix_workspace_size(ctypes.byref(desc), n, WS_FORWARD)
    _run_ws(dev, "so2conv_mix_experts_forward", need, ws, lib.so2conv_mix_experts_forward,
            ctypes.byref(desc), n, _adr(experts), _adr(weights), _adr(index), _adr(out))
    return out


def mix_experts_backward(desc, experts, weights, grad_out, index=None, need=None, ws=None,
                         out=None):
    """so2conv_mix_experts_backward: a dict with grad_experts and grad_weights
    (those in `need`)."""
    lib = load()
    n, dev, experts, weights, index = _mix_inputs(desc, experts, weights, index)
    grad_out = _need(grad_out, "grad_out", (n, desc.n_weights), torch.float32, dev)
    names = ["grad_experts", "grad_weights"]
    need = set(names if need is None else need)
    shapes = {"grad_experts": (desc.n_experts, desc.n_weights), "grad_weights": (n, desc.top_k)}
    outs = _outputs(names, need, shapes, out, dict(dtype=torch.float32, device=dev))
    size = lib.so2conv_mix_workspace_size(ctypes.byref(desc), n, WS_BACKWARD)
    _run_ws(dev, "so2conv_mix_experts_backward", size, ws, lib.so2conv_mix_experts_backward,
            ctypes.byref(desc), n, _adr(experts), _adr(weights), _adr(index), _adr(grad_out),
            *[_adr(outs[k]) for k in names])
    return {k: t for k, t in outs.items() if t is not None}


def make_dropout_desc(channels, n_comp=1, unit="channel", p=0.1, dtype=SO2_F32):
    return DropoutDesc(channels, n_comp, DROP_UNITS[unit], float(p), dtype)


def dropout(desc, x, rng, residual=None, rows=None, out=None):
    """so2conv_dropout: the dropped x [n, n_comp, channels], plus the residual.
    rng: int64 [2] on the device (key, offset).  The backward is the same call
    on the gradient, without the residual; `out` may be x or the residual."""
    lib = load()
    n, dt = x.shape[0], _torch_dtype(desc.dtype)
    shape = (n, desc.n_comp, desc.channels)
    x = _need(x, "x", shape, dt)
    dev = x.device
    rng = _need(rng, "rng", (2,), torch.int64, dev)
    if residual is not None:
        residual = _need(residual, "residual", shape, dt, dev)
    if rows is not None:
        rows = _need(rows, "rows", (n,), torch.int64, dev)
    out = _given_out(out, "out", shape, dt, x)
    _run(dev, "so2conv_dropout", lib.so2conv_dropout, ctypes.byref(desc), n, _adr(x),
         _adr(residual), _adr(rows), _adr(rng), _adr(out))
    return out
