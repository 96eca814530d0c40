"""Float64 definitions of the model operators beside the convolution: element
embedding, routing to experts, mixing of experts' weights, and dropout.

TEST INFRASTRUCTURE ONLY, like the rest of this package.  Written row by row
from the definitions, with numpy and Python integers; torch tensors of any
dtype go in, float64 tensors come out.
"""

import math

import numpy as np
import torch

F64 = torch.float64


# ---- element embedding --------------------------------------------------------
def embed_forward(ids, table, n_comp, scale, pad_id=None):
    """out [n, n_comp, C]; pad ids and ids outside the table give zero rows."""
    out = torch.zeros((len(ids), n_comp, table.shape[1]), dtype=F64)
    for i, v in enumerate(ids.tolist()):
        if v != pad_id and 0 <= v < table.shape[0]:
            out[i, 0] = table[v].to(F64) * scale
    return out


def embed_backward(ids, grad_rows, n_rows, scale, pad_id=None):
    """(grad_table [n_rows, C], the sums of magnitudes, the rows of each id)."""
    g = torch.zeros((n_rows, grad_rows.shape[1]), dtype=F64)
    mag, count = torch.zeros_like(g), torch.zeros(n_rows, dtype=F64)
    for i, v in enumerate(ids.tolist()):
        if v != pad_id and 0 <= v < n_rows:
            row = grad_rows[i].to(F64) * scale
            g[v] += row
            mag[v] += row.abs()
            count[v] += 1
    return g, mag, count


# ---- routing to experts ---------------------------------------------------------
def _scores(x, softmax):
    if not softmax:
        return [1.0 / (1.0 + math.exp(-v)) if v > -700 else 0.0 for v in x]
    m = max(x)
    if m == -math.inf:
        return [0.0] * len(x)
    e = [math.exp(v - m) for v in x]
    z = math.fsum(e)
    return [v / z for v in e]


def _rank(values):
    """Indices in falling order, NaN behind every number, ties by index."""
    low = [(1 if v != v else 0, 0.0 if v != v else -v, i) for i, v in enumerate(values)]
    return [i for _, _, i in sorted(low)]


def route_row(x, bias, top_k, softmax, n_groups=1, top_groups=1, group_top=1,
              renormalise=False, scale=1.0):
    """One row: (scores, chosen experts with -1 for unused slots, weights)."""
    K = len(x)
    clean = [-math.inf if v != v else v for v in x]
    s = _scores(clean, softmax)
    c = [s[i] + (bias[i] if bias is not None else 0.0) for i in range(K)]
    order = c if bias is not None else list(x)
    live = [x[i] != -math.inf and c[i] != -math.inf for i in range(K)]
    if n_groups > top_groups:
        per, ranks = K // n_groups, []
        for g in range(n_groups):
            member = [i for i in range(g * per, (g + 1) * per) if live[i]]
            by = order if group_top == 1 else c
            best = [member[i] for i in _rank([by[i] for i in member])][:group_top]
            ranks.append(sum(by[i] for i in best) if best else None)
        some = [g for g in range(n_groups) if ranks[g] is not None]
        stay = [some[i] for i in _rank([ranks[g] for g in some])][:top_groups]
        live = [live[i] and i // per in stay for i in range(K)]
    if top_k == K:
        chosen = [i if live[i] else -1 for i in range(K)]
    else:
        member = [i for i in range(K) if live[i]]
        chosen = [member[i] for i in _rank([order[i] for i in member])][:top_k]
        chosen += [-1] * (top_k - len(chosen))
    total = 1.0
    if renormalise:
        total = math.fsum(s[e] for e in chosen if e >= 0)
    w = [s[e] / total * scale if e >= 0 and total > 0 else 0.0 for e in chosen]
    return s, chosen, w


def route_forward(logits, bias=None, **kw):
    """(weights [n, k], index [n, k], counts [K]) in float64 / int64."""
    softmax = kw.pop("score", "softmax") == "softmax"
    b = None if bias is None else bias.double().tolist()
    rows = [route_row(x, b, softmax=softmax, **kw) for x in logits.double().tolist()]
    k = kw["top_k"]
    w = torch.tensor([r[2] for r in rows], dtype=F64).view(-1, k)
    index = torch.tensor([r[1] for r in rows], dtype=torch.int64).view(-1, k)
    counts = torch.bincount(index[index >= 0].flatten(), minlength=logits.shape[1])
    return w, index, counts


def route_backward(logits, index, grad_weights, score="softmax", renormalise=False, scale=1.0):
    """grad_logits [n, K]: row by row through the chain rule's Jacobians."""
    n, K = logits.shape
    out = torch.zeros((n, K), dtype=F64)
    for t in range(n):
        s = np.array(_scores(logits[t].double().tolist(), score == "softmax"))
        js = np.diag(s) - np.outer(s, s) if score == "softmax" else np.diag(s * (1.0 - s))
        g = np.zeros(K)
        slots = [(j, e) for j, e in enumerate(index[t].tolist()) if 0 <= e < K]
        gw = [float(v) for v in grad_weights[t].double().tolist()]
        total = sum(s[e] for _, e in slots)
        for j, e in slots:
            if not renormalise:
                g[e] += scale * gw[j]
            elif total > 0:
                g[e] += scale * gw[j] / total
                for _, f in slots:
                    g[f] -= scale * gw[j] * s[e] / total ** 2
        out[t] = torch.from_numpy(js @ g)
    return out


# ---- mixing of experts' weights -----------------------------------------------------
def mix_forward(experts, weights, index=None):
    """(out [T, n], the sums of magnitudes)."""
    T, k = weights.shape
    out = torch.zeros((T, experts.shape[1]), dtype=F64)
    mag = torch.zeros_like(out)
    for t in range(T):
        for j in range(k):
            e = j if index is None else int(index[t, j])
            if 0 <= e < experts.shape[0]:
                term = weights[t, j].to(F64) * experts[e].to(F64)
                out[t] += term
                mag[t] += term.abs()
    return out, mag


def mix_backward(experts, weights, grad_out, index=None):
    """((grad_experts, magnitudes), (grad_weights, magnitudes))."""
    T, k = weights.shape
    ge = torch.zeros((experts.shape[0], experts.shape[1]), dtype=F64)
    gw = torch.zeros((T, k), dtype=F64)
    me, mw = torch.zeros_like(ge), torch.zeros_like(gw)
    for t in range(T):
        g = grad_out[t].to(F64)
        for j in range(k):
            e = j if index is None else int(index[t, j])
            if 0 <= e < experts.shape[0]:
                term = weights[t, j].to(F64) * g
                ge[e] += term
                me[e] += term.abs()
                p = g * experts[e].to(F64)
                gw[t, j] = p.sum()
                mw[t, j] = p.abs().sum()
    return (ge, me), (gw, mw)


# ---- dropout ----------------------------------------------------------------------------
def philox(counter, key):
    """Philox-4x32-10 of a 128-bit counter and a 64-bit key, on Python integers."""
    low = (1 << 32) - 1
    x = [(counter >> (32 * i)) & low for i in range(4)]
    k = [key & low, (key >> 32) & low]
    for _ in range(10):
        a, b = x[0] * 0xD2511F53, x[2] * 0xCD9E8D57
        x = [(b >> 32) ^ x[1] ^ k[0], b & low, (a >> 32) ^ x[3] ^ k[1], a & low]
        k = [(k[0] + 0x9E3779B9) & low, (k[1] + 0xBB67AE85) & low]
    return x


def dropout_keep(shape, unit, p, seed, offset, rows=None):
    """The mask [n, n_comp, channels]; p is taken as its f32 value."""
    n, s, c = shape
    wrap = (1 << 64) - 1
    threshold = int(round(float(np.float32(p)) * 2.0 ** 32))
    cache, keep = {}, np.zeros(shape, dtype=bool)
    for i in range(n):
        for q in range(s):
            for d in range(c):
                if unit == "element":
                    m = (i * s + q) * c + d
                elif unit == "channel":
                    m = i * c + d
                else:
                    m = (i if rows is None else int(rows[i])) & wrap
                if m // 4 not in cache:
                    cache[m // 4] = philox((m // 4) | ((offset & wrap) << 64), seed & wrap)
                keep[i, q, d] = cache[m // 4][m % 4] >= threshold
    return torch.from_numpy(keep)


def dropout(x, keep, p, residual=None):
    p = float(np.float32(p))
    y = torch.zeros(x.shape, dtype=F64)
    if p < 1.0:
        y[keep] = x.to(F64)[keep] / (1.0 - p)
    return y if residual is None else y + residual.to(F64)
