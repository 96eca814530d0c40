"""Model operators around the SO(2) edge convolution: their cases, their plain forms and their calls.

Four operators that a potential built on the convolution runs beside it:

* ``embed``    element embedding: rows of a table by atomic number into the l = 0 rows of the node
               features (the others zero), and the table's gradient;
* ``route``    routing of systems or nodes to experts: softmax or sigmoid scores, a bias that only
               selects, groups, top-k, renormalised weights, and the gradient of the logits;
* ``mix``      the routed experts' packed convolution weights summed into one set of weights per
               system, with the gradients of the experts and of the routing weights;
* ``dropout``  dropout over elements, over channels (one draw for all components of an irrep
               channel) or over rows, from a counter-based generator, with a residual.

``run`` computes them from elementary torch operations, or with the library where ``own`` is set.
"""

import math

import torch

own = False

DEV = "cuda"
PAD = -1
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # embedding: the smallest graph, forward and backward; latency counts
        dict(name="embed_small", op="embed", mode="step", n=64, vocab=100, c=16, s=9, table="f32",
             out="f32", pad=0.0),
        # initial node features of the 20,000-atom graph: element rows in bf16, other rows zero
        dict(name="embed_nodes", op="embed", mode="fwd", n=20000, vocab=100, c=128, s=25,
             table="f32", out="bf16", pad=0.0),
        # gradient of the source-element embedding of a million edges: few, very long segments
        dict(name="embed_edges_grad", op="embed", mode="bwd", n=1000000, vocab=100, c=128, s=1,
             table="f32", out="f32", pad=0.0),
        # a large vocabulary with padded ids, most segments of length 0 or 1, odd sizes
        dict(name="embed_vocab", op="embed", mode="step", n=30011, vocab=50021, c=201, s=1,
             table="bf16", out="bf16", pad=0.1),
        # routing of one system to all of 32 experts, as each molecular-dynamics start does
        dict(name="route_one", op="route", mode="fwd", t=1, k=32, top=32, score="softmax", groups=1,
             top_groups=1, group_top=1, renorm=False, bias=False, masked=0.0, dtype="f32"),
        # node-level routing of a 20,000-atom graph with a balancing bias and groups, training
        dict(name="route_groups", op="route", mode="step", t=20000, k=64, top=6, score="sigmoid",
             groups=8, top_groups=4, group_top=2, renorm=True, bias=True, masked=0.05,
             dtype="bf16"),
        # a batch of 64 graphs of about 2,000 atoms, softmax top-8 of 128, training
        dict(name="route_large", op="route", mode="step", t=131071, k=128, top=8, score="softmax",
             groups=1, top_groups=1, group_top=1, renorm=True, bias=False, masked=0.0,
             dtype="f32"),
        # one system's weights from 32 experts for lmax 6, mmax 2, C 128: serving, bf16
        dict(name="mix_one", op="mix", mode="fwd", t=1, k=32, top=32, n=2801664, experts="f32",
             out="bf16"),
        # 64 systems over 32 experts for lmax 4, mmax 2, C 128: a training step, dense
        dict(name="mix_dense", op="mix", mode="step", t=64, k=32, top=32, n=1228800, experts="f32",
             out="f32"),
        # top-4 of 64 experts for 33 systems at C 64: a training step, sparse, bf16
        dict(name="mix_topk", op="mix", mode="step", t=33, k=64, top=4, n=307200, experts="bf16",
             out="bf16"),
        # channel dropout of the 2,000-atom graph's messages onto their residual
        dict(name="dropout_channels", op="dropout", n=2000, s=25, c=128, unit="channel", p=0.1,
             residual=True, dtype="f32"),
        # element dropout of the 20,000-atom graph's features
        dict(name="dropout_elements", op="dropout", n=20000, s=25, c=128, unit="element", p=0.2,
             residual=False, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed", "route", "mix", "dropout"])
    if op == "embed":
        s = rng.choice([1, 1, 4, 9, 16, 25, 49])
        c = _log_int(rng, 1, 512)
        n = _log_int(rng, 1, max(1, min(1000000, 64000000 // (s * c))))
        return dict(op=op, mode=rng.choice(["fwd", "bwd", "step"]), n=n,
                    vocab=_log_int(rng, 1, 60000), c=c, s=s, table=rng.choice(["f32", "bf16"]),
                    out=rng.choice(["f32", "bf16"]), pad=rng.choice([0.0, 0.3]))
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        per = _log_int(rng, 1 if groups == 1 else 2, 256 // groups)
        k = groups * per
        t = _log_int(rng, 1, max(1, min(131072, 16000000 // k)))
        top_groups = rng.randint(1, groups)
        top = rng.choice([_log_int(rng, 1, min(16, top_groups * per)), k if groups == 1 else 1])
        return dict(op=op, mode=rng.choice(["fwd", "step"]), t=t, k=k, top=top,
                    score=rng.choice(["softmax", "sigmoid"]), groups=groups, top_groups=top_groups,
                    group_top=rng.randint(1, min(2, per)), renorm=rng.random() < 0.5,
                    bias=rng.random() < 0.5, masked=rng.choice([0.0, 0.1]),
                    dtype=rng.choice(["f32", "bf16"]))
    if op == "mix":
        k = _log_int(rng, 1, 128)
        t = _log_int(rng, 1, 64)
        n = _log_int(rng, 1, min(2801664, 100000000 // (t + k)))
        return dict(op=op, mode=rng.choice(["fwd", "step"]), t=t, k=k,
                    top=rng.choice([k, _log_int(rng, 1, min(k, 8))]), n=n,
                    experts=rng.choice(["f32", "bf16"]), out=rng.choice(["f32", "bf16"]))
    s = rng.choice([1, 4, 9, 16, 25, 49])
    c = _log_int(rng, 1, 512)
    return dict(op=op, n=_log_int(rng, 1, max(1, min(1000000, 64000000 // (s * c)))), s=s, c=c,
                unit=rng.choice(["element", "channel", "row"]), p=round(rng.uniform(0.0, 0.9), 3),
                residual=rng.random() < 0.5, dtype=rng.choice(["f32", "bf16"]))


def _size(name):
    return 2 if name == "bf16" else 4


def work(case):
    if case["op"] == "embed":
        n, c, s, v = case["n"], case["c"], case["s"], case["vocab"]
        rows = min(n, v)  # table rows that the ids can touch
        b = 8 * n
        if case["mode"] in ("fwd", "step"):
            b += rows * c * _size(case["table"]) + n * s * c * _size(case["out"])
        if case["mode"] in ("bwd", "step"):
            b += n * c * _size(case["out"]) + v * c * 4
        return {"bytes": b, "flops": n * c * (2 if case["mode"] == "step" else 1)}
    if case["op"] == "route":
        t, k, top = case["t"], case["k"], case["top"]
        b = t * k * _size(case["dtype"]) + t * top * 8 + k * 4 * (2 if case["bias"] else 1)
        if case["mode"] == "step":
            b += t * top * 4 + t * k * 4
        return {"bytes": b, "flops": t * k * (8 if case["mode"] == "step" else 4)}
    if case["op"] == "mix":
        t, k, top, n = case["t"], case["k"], case["top"], case["n"]
        used = min(k, t * top)  # experts that the routing can touch
        b = used * n * _size(case["experts"]) + t * n * _size(case["out"]) + t * top * 8
        f = 2 * t * top * n
        if case["mode"] == "step":
            b += t * n * 4 + k * n * 4 + t * top * 4
            f *= 3
        return {"bytes": b, "flops": f}
    m = case["n"] * case["s"] * case["c"] * _size(case["dtype"])
    return {"bytes": m * (3 if case["residual"] else 2), "flops": m // _size(case["dtype"])}


def _normal(g, shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    st = {"case": case}
    if case["op"] == "embed":
        n, v, c, s = case["n"], case["vocab"], case["c"], case["s"]
        # element (or token) frequencies fall off as the rank to the power -1.2
        u = torch.rand(n, generator=g, device=DEV, dtype=torch.float64)
        rank = (1.0 - u * (1.0 - (v + 1.0) ** -0.2)) ** -5.0
        order = torch.argsort(torch.rand(v, generator=g, device=DEV), stable=True)
        ids = order[(rank.long() - 1).clamp(0, v - 1)]
        if case["pad"] > 0:
            drop = torch.rand(n, generator=g, device=DEV) < case["pad"]
            ids = torch.where(drop, torch.full_like(ids, PAD), ids)
        st["ids"] = ids
        st["table"] = _normal(g, (v, c), DTYPES[case["table"]])
        st["grad"] = _normal(g, (n, s, c), DTYPES[case["out"]]) if case["mode"] != "fwd" else None
        st["scale"] = 0.5
    elif case["op"] == "route":
        t, k = case["t"], case["k"]
        logits = _normal(g, (t, k))
        if case["masked"] > 0:
            off = torch.rand((t, k), generator=g, device=DEV) < case["masked"]
            logits = logits.masked_fill(off, float("-inf"))
        st["logits"] = logits.to(DTYPES[case["dtype"]])
        st["bias"] = _normal(g, (k,)) * 0.1 if case["bias"] else None
        st["grad"] = _normal(g, (t, case["top"])) if case["mode"] == "step" else None
        st["scale"] = 1.5
    elif case["op"] == "mix":
        t, k, top, n = case["t"], case["k"], case["top"], case["n"]
        st["experts"] = (_normal(g, (k, n)) / 32.0).to(DTYPES[case["experts"]])
        logits = _normal(g, (t, k))
        if top == k:
            st["index"], picked = None, logits
        else:
            picked, index = torch.topk(logits, top, dim=1)
            st["index"] = index.to(torch.int32)
        st["weights"] = torch.softmax(picked, dim=1)
        st["grad"] = _normal(g, (t, n)) if case["mode"] == "step" else None
    else:
        shape = (case["n"], case["s"], case["c"])
        st["x"] = _normal(g, shape, DTYPES[case["dtype"]])
        st["residual"] = _normal(g, shape, DTYPES[case["dtype"]]) if case["residual"] else None
        st["rng"] = torch.randint(0, 1 << 62, (2,), generator=g, device=DEV)
        # row dropout drops whole systems: the system of each row, in order
        st["rows"] = None
        if case["unit"] == "row":
            st["rows"] = torch.arange(case["n"], device=DEV) // 7
    return st


def run(state):
    if own:
        return _OWN[state["case"]["op"]](state)
    return _PLAIN[state["case"]["op"]](state)


# --- the plain forms ------------------------------------------------------------------------------

def _plain_embed(st):
    case, ids, table = st["case"], st["ids"], st["table"]
    n, c, s = case["n"], case["c"], case["s"]
    keep = (ids != PAD).unsqueeze(1)
    at = ids.clamp(min=0)
    res = {}
    if case["mode"] in ("fwd", "step"):
        out = torch.zeros((n, s, c), dtype=DTYPES[case["out"]], device=DEV)
        out[:, 0, :] = torch.where(keep, table[at].float() * st["scale"], 0.0).to(out.dtype)
        res["out"] = out
    if case["mode"] in ("bwd", "step"):
        # segments of up to a million rows: summed in 64 bits
        rows = torch.where(keep, st["grad"][:, 0, :].double(), 0.0)
        total = torch.zeros((case["vocab"], c), dtype=torch.float64, device=DEV)
        res["grad_table"] = (total.index_add_(0, at, rows) * st["scale"]).float()
    return res


def _ranked(case, logits, bias):
    """Scores s, and the selection scores with what may not be chosen at -inf; 64 bits, since two
    experts next to each other in the order must not change places by a rounding."""
    x = logits.double()
    if case["score"] == "softmax":
        e = torch.exp(x - x.amax(dim=1, keepdim=True))
        s = e / e.sum(dim=1, keepdim=True)
    else:
        s = 1.0 / (1.0 + torch.exp(-x))
    none = float("-inf")
    dead = x == none
    s = torch.where(dead, 0.0, torch.nan_to_num(s))  # a row that is masked throughout has no scores
    c = s if bias is None else s + bias.double()
    c = torch.where(dead, none, c)
    if case["groups"] > 1:
        t, groups = case["t"], case["groups"]
        best = torch.sort(c.view(t, groups, -1), dim=2, descending=True).values
        best = best[:, :, :case["group_top"]]
        gs = torch.where(best == none, 0.0, best).sum(dim=2)
        gs = torch.where(best[:, :, 0] == none, none, gs)
        order = torch.sort(gs, dim=1, descending=True, stable=True).indices
        kept = torch.zeros_like(gs, dtype=torch.bool)
        kept.scatter_(1, order[:, :case["top_groups"]], True)
        kept = kept.repeat_interleave(case["k"] // groups, dim=1)
        c = torch.where(kept, c, none)
    return s, c


def _plain_route(st):
    case, logits = st["case"], st["logits"]
    k, top = case["k"], case["top"]
    s, c = _ranked(case, logits, st["bias"])
    if top == k:  # nothing to select: slot j is expert j
        index = torch.arange(k, device=DEV).expand(case["t"], k)
    else:
        index = torch.sort(c, dim=1, descending=True, stable=True).indices[:, :top]
    live = torch.gather(c, 1, index) > float("-inf")
    w = torch.where(live, torch.gather(s, 1, index), 0.0)
    total = torch.ones_like(w[:, :1])
    if case["renorm"]:
        total = w.sum(dim=1, keepdim=True)
        total = torch.where(total > 0, total, math.inf)
    w = w / total
    counts = torch.zeros(k, dtype=torch.int32, device=DEV)
    counts.index_add_(0, index.reshape(-1), live.reshape(-1).to(torch.int32))
    res = {"weights": (w * st["scale"]).float(), "index": torch.where(live, index, -1).to(torch.int32),
           "counts": counts}
    if case["mode"] == "step":
        g = torch.where(live, st["grad"].double(), 0.0)
        if case["renorm"]:
            g = g - (g * w).sum(dim=1, keepdim=True)
        g = torch.where(live, g / total * st["scale"], 0.0)
        gs = torch.zeros_like(s).scatter_add_(1, index, g)
        if case["score"] == "softmax":
            gl = s * (gs - (s * gs).sum(dim=1, keepdim=True))
        else:
            gl = s * (1.0 - s) * gs
        res["grad_logits"] = gl.float()
    return res


def _dense_weights(st):
    case, w = st["case"], st["weights"]
    if st["index"] is None:
        return w
    a = torch.zeros((case["t"], case["k"]), device=DEV)
    return a.scatter_add_(1, st["index"].long(), w)


def _plain_mix(st):
    case, experts = st["case"], st["experts"].float()
    a = _dense_weights(st)
    res = {"out": (a @ experts).to(DTYPES[case["out"]])}
    if case["mode"] == "step":
        res["grad_experts"] = a.t() @ st["grad"]
        # sums over all weights of a layer: in 64 bits
        ga = st["grad"].double() @ experts.double().t()
        res["grad_weights"] = (ga if st["index"] is None
                               else torch.gather(ga, 1, st["index"].long())).float()
    return res


_LOW = 0xFFFFFFFF


def _philox(counter, rng):
    """Philox-4x32-10 (Salmon, Moraes, Dror and Shaw 2011): four words of 32 bits for each 64-bit
    counter; the key is rng[0], the counter's upper half rng[1]."""
    x0, x1 = counter & _LOW, (counter >> 32) & _LOW
    x2, x3 = (rng[1] & _LOW).expand_as(x0), ((rng[1] >> 32) & _LOW).expand_as(x0)
    k0, k1 = rng[0] & _LOW, (rng[0] >> 32) & _LOW
    for _ in range(10):
        p0, p1 = x0 * 0xD2511F53, x2 * 0xCD9E8D57  # the low 64 bits of the products are exact
        x0, x1, x2, x3 = (((p1 >> 32) & _LOW) ^ x1 ^ k0, p1 & _LOW,
                          ((p0 >> 32) & _LOW) ^ x3 ^ k1, p0 & _LOW)
        k0, k1 = (k0 + 0x9E3779B9) & _LOW, (k1 + 0xBB67AE85) & _LOW
    return torch.stack([x0, x1, x2, x3], dim=-1)


def _plain_dropout(st):
    case, x, p = st["case"], st["x"], st["case"]["p"]
    n, s, c = x.shape
    if case["unit"] == "row":
        u = st["rows"]
        words = torch.gather(_philox(u >> 2, st["rng"]), 1, (u & 3).unsqueeze(1))
        words = words.view(n, 1, 1)
    else:
        count = n * s * c if case["unit"] == "element" else n * c
        blocks = torch.arange((count + 3) // 4, device=DEV)
        words = _philox(blocks, st["rng"]).view(-1)[:count]
        words = words.view(n, s, c) if case["unit"] == "element" else words.view(n, 1, c)
    keep = words >= _threshold(p)
    y = torch.where(keep, x.float() * _keep_scale(p), 0.0)
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return {"out": y.to(x.dtype)}


def _threshold(p):
    # p is a 32-bit number in the call
    return int(round(torch.tensor(p, dtype=torch.float32).double().item() * 2.0 ** 32))


def _keep_scale(p):
    p = torch.tensor(p, dtype=torch.float32).double().item()
    return torch.tensor(1.0 / (1.0 - p), dtype=torch.float32).item()


_PLAIN = {"embed": _plain_embed, "route": _plain_route, "mix": _plain_mix,
          "dropout": _plain_dropout}


# --- the library's calls --------------------------------------------------------------------------

def _code(name):
    from so_edge_convolution_b200 import binding as B
    return B.SO2_BF16 if name == "bf16" else B.SO2_F32


def _own_embed(st):
    from so_edge_convolution_b200 import binding as B
    case = st["case"]
    desc = B.make_embed_desc(case["vocab"], case["c"], case["s"], scale=st["scale"],
                             table_dtype=_code(case["table"]), out_dtype=_code(case["out"]),
                             pad_id=PAD)
    res = {}
    if case["mode"] in ("fwd", "step"):
        res["out"] = B.embed_forward(desc, st["ids"], st["table"])
    if case["mode"] in ("bwd", "step"):
        res["grad_table"] = B.embed_backward(desc, st["ids"], st["grad"])
    return res


def _own_route(st):
    from so_edge_convolution_b200 import binding as B
    case = st["case"]
    desc = B.make_route_desc(case["k"], case["top"], score=case["score"], n_groups=case["groups"],
                             top_groups=case["top_groups"], group_top=case["group_top"],
                             renormalise=case["renorm"], scale=st["scale"],
                             dtype=_code(case["dtype"]))
    weights, index, counts = B.route_forward(desc, st["logits"], bias=st["bias"])
    res = {"weights": weights, "index": index, "counts": counts}
    if case["mode"] == "step":
        res["grad_logits"] = B.route_backward(desc, st["logits"], index, st["grad"])
    return res


def _own_mix(st):
    from so_edge_convolution_b200 import binding as B
    case = st["case"]
    desc = B.make_mix_desc(case["k"], case["n"], case["top"], expert_dtype=_code(case["experts"]),
                           out_dtype=_code(case["out"]))
    res = {"out": B.mix_experts_forward(desc, st["experts"], st["weights"], index=st["index"])}
    if case["mode"] == "step":
        res.update(B.mix_experts_backward(desc, st["experts"], st["weights"], st["grad"],
                                          index=st["index"]))
    return res


def _own_dropout(st):
    from so_edge_convolution_b200 import binding as B
    case = st["case"]
    desc = B.make_dropout_desc(case["c"], case["s"], unit=case["unit"], p=case["p"],
                               dtype=_code(case["dtype"]))
    return {"out": B.dropout(desc, st["x"], st["rng"], residual=st["residual"], rows=st["rows"])}


_OWN = {"embed": _own_embed, "route": _own_route, "mix": _own_mix, "dropout": _own_dropout}


# --- from the definitions, in 64 bits -------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    return {"embed": _exact_embed, "route": _exact_route, "mix": _exact_mix,
            "dropout": _exact_dropout}[case["op"]](case, st)


def _exact_embed(case, st):
    n, c, s, v = case["n"], case["c"], case["s"], case["vocab"]
    res = {}
    valid = torch.nonzero(st["ids"] != PAD).flatten()
    if case["mode"] in ("fwd", "step"):
        out = torch.zeros((n, s, c), dtype=torch.float64, device=DEV)
        rows = torch.index_select(st["table"].double(), 0, st["ids"][valid])
        out[valid, 0] = rows * st["scale"]
        res["out"] = out
    if case["mode"] in ("bwd", "step"):
        # by sorted ids: differences of running sums at the segments' ends, a few channels at a time
        ids, order = torch.sort(st["ids"][valid], stable=True)
        ends = torch.searchsorted(ids, torch.arange(v, device=DEV), right=True)
        total = torch.empty((v, c), dtype=torch.float64, device=DEV)
        for a in range(0, c, 32):
            run_ = torch.cumsum(st["grad"][valid[order], 0, a:a + 32].double(), dim=0)
            run_ = torch.cat([torch.zeros_like(total[:1, a:a + 32]), run_])
            total[:, a:a + 32] = torch.diff(run_[ends], dim=0, prepend=run_[:1])
        res["grad_table"] = total * st["scale"]
    return res


def _exact_route(case, st):
    k, top = case["k"], case["top"]
    x = st["logits"].double()
    open_ = torch.isfinite(x)
    if case["score"] == "softmax":
        s = torch.exp(torch.log_softmax(x, dim=1))
    else:
        s = torch.sigmoid(x)
    s = torch.where(open_, torch.nan_to_num(s), 0.0)
    rank = torch.where(open_, s + (0.0 if st["bias"] is None else st["bias"].double()), -math.inf)
    if case["groups"] > 1:
        per = k // case["groups"]
        best = torch.topk(rank.view(-1, case["groups"], per), case["group_top"], dim=2).values
        score = best.clamp(min=-1e300).sum(2)
        if case["group_top"] == 2:
            score = torch.where(torch.isinf(best[..., 1]), best[..., 0], score)
        floor = torch.topk(score, case["top_groups"], dim=1).values[:, -1:]
        rank = torch.where((score >= floor).repeat_interleave(per, dim=1), rank, -math.inf)
    if top == k:
        index = torch.arange(k, device=DEV).repeat(case["t"], 1)
    else:
        index = torch.topk(rank, top, dim=1).indices
    chosen = torch.zeros_like(s, dtype=torch.bool).scatter_(1, index, True)
    chosen &= torch.isfinite(rank)
    u = s * chosen
    z = u.sum(1, keepdim=True) if case["renorm"] else torch.ones_like(s[:, :1])
    z = torch.where(z > 0, z, math.inf)
    res = {"weights": torch.gather(u / z * st["scale"], 1, index), "index": None, "counts": None}
    if case["mode"] == "step":
        ga = torch.zeros_like(s).scatter_(1, index, st["grad"].double()) * chosen
        # through u / z, then through the scores
        if case["renorm"]:
            ga = ga - (ga * (u / z)).sum(1, keepdim=True)
        gu = ga / z * chosen * st["scale"]
        if case["score"] == "softmax":
            res["grad_logits"] = s * gu - s * (s * gu).sum(1, keepdim=True)
        else:
            res["grad_logits"] = gu * (s - s * s)
    return res


def _exact_mix(case, st):
    t, k, top, n = case["t"], case["k"], case["top"], case["n"]
    index = st["index"]
    if index is None:
        index = torch.arange(k, device=DEV).repeat(t, 1)
    index = index.long()
    w = st["weights"].double()
    out = torch.empty((t, n), dtype=torch.float64, device=DEV)
    ge = torch.zeros((k, n), dtype=torch.float64, device=DEV)
    gw = torch.zeros((t, top), dtype=torch.float64, device=DEV)
    for i in range(t):
        rows = st["experts"][index[i]].double()
        out[i] = (w[i, :, None] * rows).sum(0)
        if case["mode"] == "step":
            g = st["grad"][i].double()
            ge.index_add_(0, index[i], w[i, :, None] * g)
            gw[i] = rows.mul_(g).sum(1)
    return {"out": out, "grad_experts": ge, "grad_weights": gw} if case["mode"] == "step" else {
        "out": out}


def _exact_dropout(case, st):
    """The generator with the products' halves from 16-bit pieces, all else in 64 bits."""
    n, s, c = case["n"], case["s"], case["c"]
    if case["unit"] == "row":
        m = st["rows"].view(n, 1, 1)
    elif case["unit"] == "channel":
        m = torch.arange(n * c, device=DEV).view(n, 1, c)
    else:
        m = torch.arange(n * s * c, device=DEV).view(n, s, c)
    block, lane = torch.div(m, 4, rounding_mode="floor"), m % 4
    low = 2 ** 32 - 1

    def product(a, b):
        mid = (a & 65535) * b
        high = (a >> 16) * b + (mid >> 16)
        return high >> 16, ((high & 65535) << 16) | (mid & 65535)

    seed, offset = (int(v) for v in st["rng"].cpu())
    x = [block & low, block >> 32, torch.full_like(block, offset & low),
         torch.full_like(block, offset >> 32)]
    key = [seed & low, seed >> 32]
    for r in range(10):
        h0, l0 = product(x[0], 0xD2511F53)
        h1, l1 = product(x[2], 0xCD9E8D57)
        x = [h1 ^ x[1] ^ key[0], l1, h0 ^ x[3] ^ key[1], l0]
        key = [(key[0] + 0x9E3779B9) & low, (key[1] + 0xBB67AE85) & low]
    word = torch.where(lane < 2, torch.where(lane == 0, x[0], x[1]),
                       torch.where(lane == 2, x[2], x[3]))
    p = torch.tensor(case["p"], dtype=torch.float32).double().item()
    y = st["x"].double() / (1.0 - p) * (word.double() >= round(p * 2.0 ** 32))
    return {"out": y if st["residual"] is None else y + st["residual"].double()}
